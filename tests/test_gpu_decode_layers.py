"""GPU: every layer of a cache of several layers, written and attended to through
KVCacheInt4.layer, with numbers of slots that leave a layer's scales off the 16-byte
grid."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
import oracle
from test_gpu_decode import _attn, _check_attn, _dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


@pytest.mark.parametrize("heads", [1, 2, 3, 4, 6, 8, 12])
@pytest.mark.parametrize("wide", [False, True])
def test_layers_with_odd_numbers_of_slots(heads, wide):
    rng = np.random.default_rng(heads)
    page, slots, layers, dim = 7, 161, 3, heads * 128
    caches = [kq.empty_kv_cache(slots, dim, layers) for _ in range(2)]
    for c in caches:
        for a in (c.codes, c.scales, c.zeros):
            a.zero_()
    table = np.full((2, 100 if wide else 12), -1, dtype=np.int32)
    ids = rng.permutation(23)
    table[0, :11], table[1, :12] = ids[:11], ids[11:]
    lens = np.array([75, 84], dtype=np.int32)
    q = torch.from_numpy(rng.standard_normal((2, 2 * heads, 128))).cuda().bfloat16()
    slot = torch.arange(slots, device="cuda")
    for i in range(layers):
        at = [c.layer(i) for c in caches]
        for c in at:
            x = torch.from_numpy(rng.standard_normal((slots, dim))).cuda().bfloat16()
            kq.kq_rht_quant_int4_kv(x, None, slot, c.codes, c.scales, c.zeros)
    for i in range(layers):
        at = [c.layer(i) for c in caches]
        out = _attn(q, *at, None, None, _dev(table), page, _dev(lens), 128 ** -0.5)
        host = [(oracle.unpack_nibbles(c.codes.cpu().numpy()), c.scales.cpu().numpy(),
                 c.zeros.cpu().numpy()) for c in at]
        _check_attn(out, q.double().cpu().numpy(), *host, None, None, table, page, lens,
                    128 ** -0.5, 0, 0)
