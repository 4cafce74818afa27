"""The marshalling module of the decode-step calls on the CPU: stand-ins for CUDA
tensors with made-up addresses, and a launch failure armed in the library, so
that a call that is passed on comes back with KQ_ERR_CUDA and launches nothing.
Whatever is wrong with an argument has to give None (nothing called)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from hadamard_rotated_activation_b200 import build as kqbuild

P = 1 << 20
BF, F32, F16, U8, I8, I32 = (torch.bfloat16, torch.float32, torch.float16, torch.uint8, torch.int8,
                             torch.int32)


class Tensor:
    """What the module asks of a tensor."""

    def __init__(self, dtype, *shape, at=0, contiguous=True, ptr=P):
        self.dtype, self.shape = dtype, torch.Size(shape)
        self._at, self._contiguous, self._ptr = at, contiguous, ptr

    def get_device(self):
        return self._at

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        if self._ptr is None:
            raise RuntimeError("no storage")
        return self._ptr


class Cache:
    def __init__(self, slots, dim, layers=0, at=0, view=None):
        lead = (layers, slots) if layers else (slots,)
        arrays = (Tensor(U8, *lead, dim // 2, at=at), Tensor(F16, *lead, dim // 128, at=at),
                  Tensor(F16, *lead, dim // 128, at=at))
        self._view = view if view is not None else \
            (*arrays, max(layers, 1), slots, dim, at, layers > 0)


class Stream:
    cuda_stream = 0


@pytest.fixture()
def call():
    """The module with device 0 current; the process's own state is put back."""
    kqbuild.build()
    L = kq.lib()
    mod = kq._native()
    entries = [ctypes.cast(f, ctypes.c_void_p).value
               for f in (L.kq_gemv, L.kq_attn_decode_int4_kv, L.kq_kv_copy_pages)]
    mod.init(BF, F32, F16, U8, I8, I32, lambda index: 0, lambda: 0, *entries)

    def armed(name, *args):
        L.kq_diag_fail_next_launch(701)
        try:
            return getattr(mod, name)(*args)
        finally:
            L.kq_diag_fail_next_launch(0)
    yield armed
    kq._call = None
    kq._native()


def gemv_args(base=1, /, m=2, n=100, k=256, xt=BF, yt=F32, **change):
    scales = {0: Tensor(F32, n), 1: Tensor(F16, n, k // 128), 2: Tensor(U8, n, k // 16),
              3: Tensor(U8, n, k // 32)}[base]
    a = dict(fmt=base, x=Tensor(xt, m, k), codes=Tensor(U8, n, k // 2), scales=scales,
             zeros=Tensor(F16, n, k // 128) if base == 1 else None,
             tensor_scale=Tensor(F32, 1) if base == 2 else None, group=128, y=Tensor(yt, m, n),
             stream=None)
    assert set(change) <= set(a)
    return {**a, **change}.values()


@pytest.mark.parametrize("fmt", range(4))
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_gemv_passes_on(call, fmt, xt, yt):
    for more in ({}, dict(stream=0), dict(stream=Stream()), dict(zeros=object())
                 if fmt != 1 else {}):
        assert call("gemv", *gemv_args(fmt, xt=xt, yt=yt, **more)) == kq.KQ_ERR_CUDA
    # what the C entry refuses comes back as its status
    assert call("gemv", *gemv_args(fmt, m=17, xt=xt, yt=yt)) == kq.KQ_ERR_UNSUPPORTED
    assert call("gemv", *gemv_args(fmt, xt=xt, yt=yt, group=64)) == \
        (kq.KQ_ERR_UNSUPPORTED if fmt == 1 else kq.KQ_ERR_CUDA)
    assert call("gemv", *gemv_args(fmt, m=0, xt=xt, yt=yt)) == kq.KQ_OK
    assert call("gemv", *gemv_args(fmt, x=Tensor(xt, 2, 256, ptr=P + 8))) == kq.KQ_ERR_MISALIGNED


@pytest.mark.parametrize("change", [
    dict(fmt=7), dict(fmt=-1), dict(fmt=None), dict(fmt=1 << 40), dict(group=1 << 32),
    dict(group=None), dict(x=Tensor(BF, 2, 128)), dict(x=Tensor(F16, 2, 256)), dict(x=None),
    dict(x=Tensor(BF, 256)), dict(x=Tensor(BF, 2, 256, at=1)), dict(x=Tensor(BF, 2, 256, at=-1)),
    dict(x=Tensor(BF, 2, 256, contiguous=False)), dict(x=Tensor(BF, 2, 256, ptr=None)),
    dict(codes=Tensor(I8, 100, 128)), dict(codes=Tensor(U8, 100, 64)),
    dict(codes=Tensor(U8, 99, 128)), dict(codes=Tensor(U8, 100, 128, at=1)),
    dict(codes=Tensor(U8, 100, 128, contiguous=False)), dict(codes=None),
    dict(scales=Tensor(F16, 100, 1)), dict(scales=Tensor(F32, 100, 2)), dict(scales=None),
    dict(zeros=Tensor(F16, 1, 100, 2)), dict(zeros=None), dict(y=Tensor(F32, 2, 99)),
    dict(y=Tensor(F32, 1, 100)), dict(y=Tensor(F16, 2, 100)), dict(y=Tensor(F32, 2, 100, at=1)),
    dict(y=Tensor(F32, 2, 100, contiguous=False)), dict(stream="s"), dict(stream=object()),
    dict(x=Tensor(BF, 0, (1 << 32) + 256), codes=Tensor(U8, 100, (1 << 31) + 128),
         scales=Tensor(F16, 100, (1 << 25) + 2), zeros=Tensor(F16, 100, (1 << 25) + 2)),
])
def test_gemv_leaves_alone(call, change):
    assert call("gemv", *gemv_args(**change)) is None


def test_gemv_other_formats_and_counts(call):
    assert call("gemv", *gemv_args(2, tensor_scale=None)) is None
    assert call("gemv", *gemv_args(2, tensor_scale=Tensor(F32, 2))) is None
    assert call("gemv", *gemv_args(0, scales=Tensor(F32, 99))) is None
    assert call("gemv", *gemv_args(3, scales=Tensor(U8, 100, 7))) is None
    assert call("gemv", *list(gemv_args())[:8]) is None


def attn_args(**change):
    a = dict(q=Tensor(BF, 3, 8, 128), k=Cache(64, 256), v=Cache(64, 256), ks=Tensor(I8, 256),
             vs=None, table=Tensor(I32, 3, 4), page=16, lens=Tensor(I32, 3), scale=0.1,
             out=Tensor(BF, 3, 8, 128, ptr=2 * P), ws=Tensor(U8, 1 << 26), window=0, sinks=0,
             stream=None)
    assert set(change) <= set(a)
    return {**a, **change}.values()


def test_attention_passes_on(call):
    for change in (dict(), dict(ks=None, vs=Tensor(I8, 256)), dict(window=7, sinks=2), dict(scale=1),
                   dict(stream=Stream()), dict(table=Tensor(I32, 3, 0))):
        assert call("attn", *attn_args(**change)) == kq.KQ_ERR_CUDA
    for change in (dict(page=0), dict(window=-1), dict(scale=float("inf")), dict(scale=1e300),
                   dict(ws=Tensor(U8, 8))):
        assert call("attn", *attn_args(**change)) == kq.KQ_ERR_INVALID_ARG
    assert call("attn", *attn_args(out=Tensor(BF, 3, 8, 128, ptr=P + 2))) == kq.KQ_ERR_MISALIGNED
    assert call("attn", *attn_args(q=Tensor(BF, 3, 7, 128), out=Tensor(BF, 3, 7, 128))) == \
        kq.KQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(q=Tensor(F32, 3, 8, 128)), dict(q=Tensor(BF, 3, 8, 64)), dict(q=Tensor(BF, 3, 1024)),
    dict(q=Tensor(BF, 3, 8, 128, at=1)), dict(q=Tensor(BF, 3, 8, 128, contiguous=False)),
    dict(q=None), dict(k=None), dict(k=Cache(64, 256, layers=2)), dict(v=Cache(32, 256)),
    dict(v=Cache(64, 128)), dict(v=Cache(64, 256, at=1)), dict(k=Cache(64, 256, view=(1, 2))),
    dict(k=Cache(64, 256, view=[0] * 8)), dict(k=Cache(64, 256, view=(0,) * 8)),
    dict(k=Cache(64, 256, at=-1), v=Cache(64, 256, at=-1)), dict(ks=Tensor(I8, 128)),
    dict(ks=Tensor(U8, 256)), dict(vs=Tensor(I8, 256, at=1)), dict(table=Tensor(I32, 2, 4)),
    dict(table=Tensor(torch.int64, 3, 4)), dict(table=Tensor(I32, 3)),
    dict(lens=Tensor(I32, 2)), dict(lens=Tensor(I32, 3, 1)), dict(lens=Tensor(F32, 3)),
    dict(lens=None), dict(page=1 << 32), dict(page=None), dict(window=1 << 31), dict(sinks=-1 << 32),
    dict(scale=None), dict(scale="x"), dict(out=Tensor(BF, 3, 8, 127)), dict(out=Tensor(F32, 3, 8, 128)),
    dict(out=Tensor(BF, 2, 8, 128)), dict(out=None), dict(ws=Tensor(F32, 1 << 24)),
    dict(ws=Tensor(U8, 1 << 20, 64)), dict(ws=Tensor(U8, 1 << 26, at=1)), dict(ws=None),
    dict(stream=b"s"),
])
def test_attention_leaves_alone(call, change):
    assert call("attn", *attn_args(**change)) is None


def test_copy(call):
    pairs, k, v = Tensor(I32, 2, 2), Cache(64, 256, 3), Cache(64, 256, 3)
    for args in ((pairs, 16, k, v, None), (pairs, 16, k, None, Stream()), (pairs, 64, k, v, 0)):
        assert call("copy", *args) == kq.KQ_ERR_CUDA
    assert call("copy", pairs, 65, k, v, None) == kq.KQ_OK            # no whole page
    assert call("copy", Tensor(I32, 0, 2), 16, k, v, None) == kq.KQ_OK
    assert call("copy", pairs, 0, k, v, None) == kq.KQ_ERR_INVALID_ARG
    assert call("copy", Tensor(I32, 2, 2, ptr=P + 4), 16, k, v, None) == kq.KQ_ERR_MISALIGNED
    for args in ((Tensor(I32, 2), 16, k, v, None), (Tensor(I32, 2, 3), 16, k, v, None),
                 (Tensor(F32, 2, 2), 16, k, v, None), (Tensor(I32, 2, 2, at=1), 16, k, v, None),
                 (Tensor(I32, 2, 2, contiguous=False), 16, k, v, None), (None, 16, k, v, None),
                 (pairs, 1 << 32, k, v, None), (pairs, 16, k, Cache(64, 256, 2), None),
                 (pairs, 16, k, Cache(64, 128, 3), None), (pairs, 16, k, Cache(32, 256, 3), None),
                 (pairs, 16, k, Cache(64, 256, 3, at=1), None), (pairs, 16, None, v, None),
                 (pairs, 16, k, v, "s"), (pairs, 16, k, v)):
        assert call("copy", *args) is None


def test_other_devices_and_faults_of_the_stream(call):
    """Another current device, or a torch that cannot name one, is left to the
    Python path."""
    L, mod = kq.lib(), kq._native()
    entries = [ctypes.cast(f, ctypes.c_void_p).value
               for f in (L.kq_gemv, L.kq_attn_decode_int4_kv, L.kq_kv_copy_pages)]

    def broken(*_):
        raise RuntimeError("no device")
    for stream, device in ((lambda i: 0, lambda: 1), (lambda i: 0, broken), (broken, lambda: 0),
                           (lambda i: None, lambda: 0), (lambda i: 0, lambda: "0")):
        mod.init(BF, F32, F16, U8, I8, I32, stream, device, *entries)
        assert call("gemv", *gemv_args()) is None
        assert call("attn", *attn_args()) is None
        assert call("copy", Tensor(I32, 2, 2), 16, Cache(64, 256), None, None) is None
    with pytest.raises(TypeError):
        mod.init(1, 2)


def test_nothing_is_kept_of_the_arguments(call):
    import sys
    args = list(attn_args())
    before = [sys.getrefcount(a) for a in args]
    for _ in range(50):
        call("attn", *args)
        call("attn", *args[:-1], "s")
    assert [sys.getrefcount(a) for a in args][:6] == before[:6]
    none = sys.getrefcount(BF)
    for _ in range(50):
        call("gemv", *gemv_args())
        call("gemv", *gemv_args(scales=None))
    assert abs(sys.getrefcount(BF) - none) < 5
