"""Host-side checks of the decode-step entry points (no GPU: validation never
dereferences a pointer, so fake aligned addresses are enough)."""
import math

import pytest

import hadamard_rotated_activation_b200 as kq
from hadamard_rotated_activation_b200 import build as kqbuild

P, Q = 1 << 20, 2 << 20
LAUNCH_ERR = 701


@pytest.fixture(scope="module")
def L():
    kqbuild.build()
    return kq.lib()


def refused(L, call):
    """The call's status with a launch failure armed, so that nothing launches."""
    try:
        L.kq_diag_fail_next_launch(LAUNCH_ERR)
        return call()
    finally:
        L.kq_diag_fail_next_launch(0)


GEMV = dict(fmt=1, x=P, xt=1, m=2, codes=P, scales=P, zeros=P, t=None, n=100, k=256, group=128,
            y=Q, yt=1, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(), kq.KQ_ERR_CUDA), (dict(m=0, x=None, codes=None, scales=None, zeros=None, y=None), 0),
    (dict(m=-1), -1), (dict(n=0), -1), (dict(k=0), -1), (dict(x=None), -1), (dict(codes=None), -1),
    (dict(scales=None), -1), (dict(zeros=None), -1), (dict(y=None), -1), (dict(fmt=4), -1),
    (dict(fmt=-1), -1), (dict(fmt=2), -1), (dict(m=17), -2), (dict(xt=2), -2), (dict(yt=-1), -2),
    (dict(k=272), -2), (dict(k=160), -2), (dict(fmt=3, k=160), kq.KQ_ERR_CUDA),
    (dict(fmt=3, k=48), -2), (dict(group=64), -2), (dict(k=131072), kq.KQ_ERR_CUDA),
    (dict(k=131072 + 128), -2), (dict(n=1 << 31), -2), (dict(n=1), kq.KQ_ERR_CUDA),
    (dict(m=16), kq.KQ_ERR_CUDA), (dict(x=P + 8), -3), (dict(y=Q + 4), -3), (dict(codes=P + 8), -3),
    (dict(scales=P + 1), -3), (dict(zeros=P + 1), -3), (dict(scales=P + 2), kq.KQ_ERR_CUDA),
    (dict(fmt=0, scales=P + 2), -3), (dict(fmt=2, t=P, scales=P + 1), -3),
    (dict(fmt=2, t=P + 2), -3), (dict(fmt=2, t=P, scales=P + 2), kq.KQ_ERR_CUDA),
    (dict(fmt=3, scales=P + 1), kq.KQ_ERR_CUDA),
])
def test_gemv_validation(L, change, want):
    assert refused(L, lambda: L.kq_gemv(*{**GEMV, **change}.values())) == want


ATTN = dict(q=P, batch=2, qh=8, kh=2, ks=None, vs=None, kc=P, ksc=P, kz=P, vc=P, vsc=P, vz=P,
            slots=64, table=P, width=4, page=16, lens=P, window=0, sinks=0, scale=0.1, out=Q,
            ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(), kq.KQ_ERR_CUDA),
    (dict(batch=0, q=None, out=None, ws=None, ws_bytes=0, table=None, lens=None), 0),
    (dict(batch=-1), -1), (dict(slots=-1), -1), (dict(width=-1), -1), (dict(page=0), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(scale=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(lens=None), -1),
    (dict(table=None), -1), (dict(ws=None), -1), (dict(ws_bytes=8), -1), (dict(kc=None), -1),
    (dict(vz=None), -1), (dict(ksc=None), -1), (dict(kh=0), -2), (dict(kh=3), -2),
    (dict(kh=129, qh=129), -2), (dict(qh=258, kh=2), -2), (dict(batch=65536), -2),
    (dict(page=65537), -2), (dict(slots=1 << 31), -2), (dict(width=1 << 40), -2),
    (dict(width=1 << 39), -2), (dict(q=P + 8), -3), (dict(out=Q + 2), -3), (dict(ks=P + 8), -3),
    (dict(vs=P + 4), -3), (dict(kc=P + 8), -3), (dict(kz=P + 2), -3), (dict(vsc=P + 2), -3),
    (dict(ws=P + 8), -3), (dict(table=P + 2), -3), (dict(lens=P + 2), -3),
    (dict(qh=256), kq.KQ_ERR_CUDA), (dict(qh=128, kh=128), kq.KQ_ERR_CUDA),
    (dict(width=0, table=None), kq.KQ_ERR_CUDA),
])
def test_attn_validation(L, change, want):
    assert refused(L, lambda: L.kq_attn_decode_int4_kv(*{**ATTN, **change}.values())) == want


def test_attn_workspace_size(L):
    need = L.kq_attn_workspace_size(2, 8, 2)
    assert need > 0
    call = lambda n: refused(  # noqa: E731
        L, lambda: L.kq_attn_decode_int4_kv(*{**ATTN, "ws_bytes": n}.values()))
    assert call(need) == kq.KQ_ERR_CUDA and call(need - 1) == kq.KQ_ERR_INVALID_ARG
    for bad in ((-1, 8, 2), (2, 7, 2), (2, 8, 0), (2, 0, 2), (65536, 8, 2)):
        assert L.kq_attn_workspace_size(*bad) == 0
    assert kq.kq_attn_workspace_size(2, 8, 2) == need


COPY = dict(pairs=P, n=4, page=16, slots=64, layers=2, dim=256, kc=P, ks=P, kz=P, vc=P, vs=P,
            vz=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(), kq.KQ_ERR_CUDA), (dict(vc=None, vs=None, vz=None), kq.KQ_ERR_CUDA),
    (dict(n=0, pairs=None, kc=None, ks=None, kz=None), 0), (dict(slots=15), 0),
    (dict(n=-1), -1), (dict(page=0), -1), (dict(slots=-1), -1), (dict(layers=0), -1),
    (dict(dim=0), -1), (dict(pairs=None), -1), (dict(kc=None), -1), (dict(kz=None), -1),
    (dict(vc=None), -1), (dict(vs=None), -1), (dict(dim=192), -2), (dict(dim=16512), -2),
    (dict(page=65537), -2), (dict(n=1 << 30), -2), (dict(slots=1 << 39), -2),
    (dict(kc=P + 8), -3), (dict(vs=P + 2), -3), (dict(kz=P + 4), -3), (dict(pairs=P + 4), -3),
])
def test_copy_validation(L, change, want):
    assert refused(L, lambda: L.kq_kv_copy_pages(*{**COPY, **change}.values())) == want


def test_binding_refuses_what_the_kernels_could_not_bound(L):
    """Shapes, types and host tensors are refused before any call; the size
    checks need no GPU because they come before the device check fails."""
    import torch
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    codes = torch.zeros(8, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kq.kq_gemv(kq.KQ_FMT_MXFP4, x, codes, torch.zeros(8, 8, dtype=torch.uint8), None, None, 0,
                   torch.zeros(2, 8))
    with pytest.raises(ValueError):
        kq.kq_gemv(kq.KQ_FMT_MXFP4, x[0], codes, None, None, None, 0, torch.zeros(2, 8))
    with pytest.raises(ValueError):
        kq.KVCacheInt4(codes, codes, codes)
    with pytest.raises(ValueError):
        kq.KVCacheInt4(codes[:, :100], codes, codes)
    with pytest.raises(ValueError):
        kq.KVCacheInt4(codes[0], codes, codes)
