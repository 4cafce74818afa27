"""Missing tensors and caches, and a format number past 32 bits, are refused with
ValueError (CPU; stand-ins for CUDA tensors, nothing is launched)."""
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from test_decode_cache import Array, armed, _cache  # noqa: F401
from test_decode_call import BF, F16, F32, I32, P, U8


def _gemv(**change):
    a = dict(fmt=kq.KQ_FMT_INT4_ASYM, x=Array(BF, 2, 256), codes=Array(U8, 100, 128),
             scales=Array(F16, 100, 2), zeros=Array(F16, 100, 2), tensor_scale=None, group=128,
             y=Array(F32, 2, 100), stream=0)
    kq.kq_gemv(**{**a, **change})


def _attn(**change):
    a = dict(q=Array(BF, 2, 4, 128), k_cache=_cache(), v_cache=_cache(), k_signs=None,
             v_signs=None, block_table=Array(I32, 2, 4), page_size=16, seq_lens=Array(I32, 2),
             softmax_scale=0.1, out=Array(BF, 2, 4, 128, ptr=2 * P), workspace=Array(U8, 1 << 26),
             stream=0)
    kq.kq_attn_decode_int4_kv(**{**a, **change})


@pytest.mark.parametrize("name", ["x", "codes", "scales", "zeros", "y"])
def test_gemv(armed, name):  # noqa: F811
    with pytest.raises(ValueError):
        _gemv(**{name: None})


@pytest.mark.parametrize("name", ["q", "k_cache", "v_cache", "block_table", "seq_lens", "out",
                                  "workspace"])
def test_attention(armed, name):  # noqa: F811
    with pytest.raises(ValueError):
        _attn(**{name: None})


def test_copy_and_cache(armed):  # noqa: F811
    for args in ((None, 16, _cache()), (Array(I32, 2, 2), 16, None)):
        with pytest.raises(ValueError):
            kq.kq_kv_copy_pages(*args, stream=0)
    with pytest.raises(ValueError):
        kq.KVCacheInt4(None, None, None)


@pytest.mark.parametrize("fmt", [2 ** 32 + 3, -2 ** 32 + 3, 2 ** 40 + 3])
def test_format_past_32_bits(armed, fmt):  # noqa: F811
    with pytest.raises(ValueError):
        _gemv(fmt=fmt, scales=Array(U8, 100, 8), zeros=None)
