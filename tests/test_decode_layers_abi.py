"""Alignment of the scales and zero points that the decode attention takes: that of
their rows, as layers of a larger cache have it (CPU: nothing is launched)."""
import pytest

import hadamard_rotated_activation_b200 as kq
from test_decode_abi import ATTN, L, P, refused  # noqa: F401


@pytest.mark.parametrize("heads,unit", [(1, 2), (2, 4), (3, 2), (4, 8), (6, 4), (8, 16), (12, 8),
                                        (16, 16), (5, 2), (32, 16)])
@pytest.mark.parametrize("name", ["ksc", "kz", "vsc", "vz"])
def test_scales_alignment(L, heads, unit, name):  # noqa: F811
    def call(at):
        return refused(L, lambda: L.kq_attn_decode_int4_kv(
            *{**ATTN, "kh": heads, "qh": 2 * heads, name: at}.values()))
    assert call(P + unit) == kq.KQ_ERR_CUDA           # passed on to the launch
    assert call(P + unit // 2) == kq.KQ_ERR_MISALIGNED
    assert call(P + 1) == kq.KQ_ERR_MISALIGNED
