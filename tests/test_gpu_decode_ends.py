"""GPU: the attention at the ends of what it takes: the largest batch, the largest
pages, the most query heads to a cached one, the most cached heads."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from test_gpu_decode import _cache, _check_attn, _dev, _upload, _whole

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


@pytest.mark.parametrize("width", [20, 80])
def test_largest_batch(width):
    """65535 sequences of 0 to 40 tokens, some of 320 or 1280, over shared pages; so many
    units are dealt whatever the table allows."""
    batch, page, pages = 65535, 16, 500
    rng = np.random.default_rng(width)
    k, v = _cache(rng, pages * page, 1), _cache(rng, pages * page, 1)
    lens = rng.integers(0, 41, batch).astype(np.int32)
    long_ones = rng.integers(0, batch, 40)
    lens[long_ones] = width * page
    table = rng.integers(0, pages, (batch, width)).astype(np.int32)
    table[rng.integers(0, batch, 1000)] = -1
    q = torch.from_numpy(rng.standard_normal((batch, 1, 128)).astype(np.float32)).cuda().bfloat16()
    out = torch.full_like(q, float("nan"))
    ws = kq.empty_attn_workspace(batch, 1, 1)
    kq.kq_attn_decode_int4_kv(q, _upload(k), _upload(v), None, None, _dev(table), page, _dev(lens),
                              SCALE, out, ws)
    assert torch.isfinite(out).all()
    assert not out[_dev(lens) == 0].any()
    some = np.unique(np.concatenate([np.arange(40), rng.integers(0, batch, 200), long_ones,
                                     np.arange(batch - 40, batch)]))
    at = torch.from_numpy(some).cuda()
    _check_attn(out[at], q[at].double().cpu().numpy(), k, v, None, None, table[some], page,
                lens[some], SCALE, 0, 0)


@pytest.mark.parametrize("page", [65535, 65536, 32769])
def test_largest_pages(page):
    _whole(page, [page + 70, 5, page], 2, 2, page, spare=0)


@pytest.mark.parametrize("heads,group", [(1, 128), (128, 1), (127, 1), (2, 127), (120, 3)])
@pytest.mark.parametrize("wide", [0, 40])
def test_most_heads(heads, group, wide):
    _whole(heads, [100, 0, 333], heads, group, 16, extra_width=wide)
