"""GPU: the attention where a head's result rests on tokens whose value scales are
far below the largest one, which hardly counts.

Weights times value scale are held in fp16 times a power of two: with L the largest
value scale seen, L in [2^(e - 1), 2^e), as p s 2^(9 - e), p <= 1 the weight relative to
the largest.  Below 2^-14, that is for p s < 2^(e - 23) <= 2^-22 L, fp16 steps by 2^-24,
half a step is 2^-25, and p s is off by at most 2^(e - 34) <= 2^-33 L.  That much times
|u - z| of each token, over the sum of the weights, comes to the tolerance of
tests/test_gpu_decode.py.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
import oracle
from oracle import decode as od
from test_gpu_decode import _attn_tolerance, _case, _run_case

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _extra(q, k, v, ks, table, page, lens):
    batch, q_heads, _ = q.shape
    heads = k[1].shape[1]
    group, h, tol = q_heads // heads, oracle.sylvester(128) / math.sqrt(128), np.zeros(q.shape)
    for b in range(batch):
        rows = od.cache_rows(table[b], page, k[1].shape[0], np.arange(lens[b]))
        for i in range(heads):
            sl = slice(128 * i, 128 * i + 128)
            a = SCALE * ((q[b, i * group:(i + 1) * group] * ks[sl]) @ h) @ od.dequant_heads(k, rows, i).T
            total = np.exp(a - a.max(1, keepdims=True)).sum(1, keepdims=True)
            step = 2.0 ** -33 * v[1][rows, i].astype(np.float64).max()
            far = np.abs(v[0][rows, sl] - v[2][rows, i].astype(np.float64)[:, None]).sum()
            tol[b, i * group:(i + 1) * group] = step * far / total / math.sqrt(128)
    return tol


@pytest.mark.parametrize("heads,group", [(8, 4), (1, 4), (2, 3), (4, 2)])
@pytest.mark.parametrize("wide", [0, 60])
@pytest.mark.parametrize("down", [10, 18, 24])
def test_small_value_scales_beside_a_large_one(heads, group, wide, down):
    """The largest value scale belongs to tokens with next to no weight, in front of
    the others, among them and behind them."""
    q, k, v, ks, vs, table, lens = _case(heads, [200, 333, 64, 3], heads, group, 16, extra_width=wide)
    v[1][:] = (2.0 ** (10 - down) * np.random.default_rng(1).uniform(1, 1.9, v[1].shape)).astype(np.float16)
    k[2][:], k[1][:] = 8, 0.25                 # scores near each other
    h, q64 = oracle.sylvester(128) / math.sqrt(128), q.double().cpu().numpy()
    for b, at in ((0, 0), (1, 150), (2, 60), (3, 1)):
        row = od.cache_rows(table[b], 16, v[1].shape[0], np.array([at]))[0]
        for i in range(heads):
            sl = slice(128 * i, 128 * i + 128)
            mean = ((q64[b, i * group:(i + 1) * group] * ks[sl]) @ h).sum(0)
            k[0][row, sl] = np.where(mean > 0, 0, 15)          # against the queries' sum
            k[1][row, i] = 4
            v[1][row, i] = 1024
    args = q64, k, v, ks, vs, table, 16, lens, SCALE
    ref = od.attn_decode(*args)
    tol = _attn_tolerance(q64, k, v, ks, table, 16, lens, SCALE, 0, 0) + \
        _extra(q64, k, v, ks, table, 16, lens)
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    out = _run_case(q, k, v, ks, vs, table, lens, 16, SCALE)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max()} x tolerance"
    again = _run_case(q, k, v, ks, vs, table, lens, 16, SCALE)
    assert torch.equal(out, again)
