"""GPU: the join of the attention's partial sums, which finds them by what the first
kernel left in the workspace: many sequences, cut and whole units side by side, a
workspace of exactly the size asked for, and results of earlier calls in it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from test_gpu_decode import _case, _check_attn, _dev, _run_case, _upload

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _guarded(batch, q_heads, kv_heads, fill):
    need = kq.kq_attn_workspace_size(batch, q_heads, kv_heads)
    buf = torch.full((need + 8192,), fill, dtype=torch.uint8, device="cuda")
    return buf, buf[4096:4096 + need]


@pytest.mark.parametrize("batch,heads,group", [(900, 1, 1), (333, 8, 2), (150, 2, 9), (60, 4, 4),
                                               (41, 3, 17), (2500, 1, 2)])
def test_many_sequences(batch, heads, group):
    """More units than CTAs, a few of them long, some empty, some all holes."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 50, batch)
    lens[rng.integers(0, batch, 5)] = 1500
    lens[rng.integers(0, batch, batch // 9)] = 0
    q, k, v, ks, vs, table, lens = _case(batch, [int(n) for n in lens], heads, group, 16)
    table[rng.integers(0, batch, 3)] = -1
    buf, ws = _guarded(batch, heads * group, heads, 0xA5)
    out = _run_case(q, k, v, ks, vs, table, lens, 16, SCALE, ws=ws)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, lens, SCALE, 0, 0)
    assert (buf[:4096] == 0xA5).all() and (buf[-4096:] == 0xA5).all()


@pytest.mark.parametrize("fill", [0, 0x7F, 0xFF])
def test_what_the_workspace_holds_does_not_matter(fill):
    """Other lengths, other heads and other batches in one workspace, one behind the
    other."""
    buf, ws = _guarded(40, 64, 8, fill)
    for seed, (lens, heads, group) in enumerate([
            ([700 + i for i in range(40)], 8, 8), ([3000, 0, 5], 8, 4), ([0] * 40, 8, 8),
            ([9000], 2, 16), ([10, 600, 0, 2000], 4, 3), ([1] * 39 + [5000], 8, 8),
            ([20000], 1, 1)]):
        q, k, v, ks, vs, table, lens = _case(seed, lens, heads, group, 32, extra_width=20)
        out = _run_case(q, k, v, ks, vs, table, lens, 32, SCALE, ws=ws)
        _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 32, lens, SCALE, 0, 0)
    assert (buf[:4096] == fill).all() and (buf[-4096:] == fill).all()


def test_lengths_written_right_in_front_of_every_call():
    """Lengths that a kernel writes directly ahead of the call, changing how units are
    cut from call to call, with nothing waited for."""
    q, k, v, ks, vs, table, lens = _case(5, [2000, 1500, 900, 40], 8, 4, 16)
    args = q, _upload(k), _upload(v), _dev(ks), _dev(vs), _dev(table), 16
    rng = np.random.default_rng(5)
    all_lens = np.stack([lens] + [rng.integers(0, lens + 1) for _ in range(15)]).astype(np.int32)
    all_dev, now = _dev(all_lens), _dev(lens)
    ws = kq.empty_attn_workspace(4, 32, 8)
    want = []
    for i in range(16):
        out = torch.empty_like(q)
        now.copy_(all_dev[i])
        torch.cuda.synchronize()
        kq.kq_attn_decode_int4_kv(*args, now, SCALE, out, ws)
        torch.cuda.synchronize()
        want.append(out)
        if i < 3:
            _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, all_lens[i], SCALE,
                        0, 0)
    for _ in range(10):
        got = [torch.empty_like(q) for _ in range(16)]
        for i in range(16):
            torch.index_select(all_dev, 0, torch.tensor([i], device="cuda"), out=now.unsqueeze(0))
            kq.kq_attn_decode_int4_kv(*args, now, SCALE, got[i], ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
