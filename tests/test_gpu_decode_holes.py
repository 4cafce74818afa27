"""GPU: attention over block tables with holes (entries outside the cache) in front
of visible tokens.  A hole hides whole tiles of a warp, of all warps, or the start
of a CTA's range; the tokens behind it carry value scales of zero or 2^-15, and
ordinary ones follow, so that a token whose weight were lost would change the
result by far more than the tolerance of tests/test_gpu_decode.py, which is used
unchanged.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from oracle import decode as od
from test_gpu_decode import _case, _check_attn, _run_case

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _quiet(v, table, seq, page, first, last, scale):
    """Value scale of the tokens first .. last - 1 of a sequence (where visible)."""
    rows = od.cache_rows(table[seq], page, v[1].shape[0], np.arange(first, last))
    v[1][rows[rows >= 0]] = np.float16(scale)


def _check(q, k, v, ks, vs, table, lens, page, window=0, sinks=0):
    out = _run_case(q, k, v, ks, vs, table, lens, page, SCALE, window, sinks)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, page, lens, SCALE, window, sinks)


@pytest.mark.parametrize("small", [0.0, 2.0 ** -15])
@pytest.mark.parametrize("heads", [1, 2, 4, 8])
@pytest.mark.parametrize("wide", [0, 64])
def test_hidden_first_tiles(heads, small, wide):
    """Sequences whose first 128 tokens are a hole: a unit a CTA (tables of 512
    tokens) and dealt (wider ones)."""
    page, lens = 16, [500, 385, 512, 140]
    q, k, v, ks, vs, table, lens = _case(heads, lens, heads, 4, page, extra_width=wide)
    for b in range(4):
        _quiet(v, table, b, page, 128, min(lens[b] - 8, 384), small)
        table[b, :8] = -1 if b % 2 else 2 ** 30
    _check(q, k, v, ks, vs, table, lens, page)


@pytest.mark.parametrize("heads", [1, 2, 4, 8])
def test_one_page_hides_a_warps_tile(heads):
    """384 tokens, two pages of the first 128 a hole, all value scales 2^-15 but those
    of the last 16 tokens."""
    page = 16
    for hole in range(0, 8, 2):
        q, k, v, ks, vs, table, lens = _case(hole + heads, [384], heads, 8, page)
        _quiet(v, table, 0, page, 0, 368, 2.0 ** -15)
        table[0, hole:hole + 2] = -1
        _check(q, k, v, ks, vs, table, lens, page)


@pytest.mark.parametrize("heads", [1, 2, 4, 8])
def test_ranges_that_begin_in_a_hole(heads):
    """One sequence cut into many ranges, half of its tiles (at random) holes,
    every value scale 2^-15 or zero but those of the last 200 tokens."""
    page = 32 if heads == 8 else 64 if heads == 4 else 128
    n = {8: 20000, 4: 20000, 2: 40000, 1: 80000}[heads]
    q, k, v, ks, vs, table, lens = _case(50 + heads, [n], heads, 2, page)
    rng = np.random.default_rng(heads)
    _quiet(v, table, 0, page, 0, n // 2, 2.0 ** -15)
    _quiet(v, table, 0, page, n // 2, n - 200, 0.0)
    hole = rng.random(table.shape[1]) < 0.5
    hole[-2:] = False
    table[0, hole] = -1
    _check(q, k, v, ks, vs, table, lens, page)


@pytest.mark.parametrize("heads", [1, 8])
def test_holes_behind_a_window_and_all_around_a_token(heads):
    """Holes inside the window and among the first tokens; a single visible token
    between holes; sequences that are nothing but holes stay zero."""
    page = 8
    q, k, v, ks, vs, table, lens = _case(70 + heads, [900, 900, 600, 700], heads, 4, page)
    table[0, 1:60] = -1
    _quiet(v, table, 0, page, 480, 890, 2.0 ** -15)
    one = table[2, 40]
    table[2, :] = -1
    table[2, 40] = one
    table[3, :] = 2 ** 31 - 1
    _check(q, k, v, ks, vs, table, lens, page)
    _check(q, k, v, ks, vs, table, lens, page, window=400, sinks=4)
    out = _run_case(q, k, v, ks, vs, table, lens, page, SCALE)
    assert not out[3].any()
