"""GPU: kq_gemv where x, the weights' scales or both are near the ends of fp32's
range, against the float64 oracle with the tolerance of tests/test_gpu_decode.py
(nothing is required where the magnitudes that are added reach 2^127).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from test_gpu_decode import KIND, _check_gemv, _gemv, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _tokens(rng, m, k, powers, xt):
    """m rows, row i scaled by the i-th power of two (in turn)."""
    x = rng.standard_normal((m, k)) * np.exp2(np.resize(powers, m).astype(float))[:, None]
    return torch.from_numpy(x).cuda().to(KIND[xt])


def _run(fmt, x, w, yt="f32"):
    y = torch.full((x.shape[0], w[0].shape[0]), float("nan"), dtype=KIND[yt], device="cuda")
    _gemv(fmt, x, *w, y)
    _check_gemv(fmt, x.double().cpu().numpy(), w, y)
    return y


@pytest.mark.parametrize("xt,m", [("bf16", 4), ("bf16", 12), ("f32", 3), ("f32", 7), ("f32", 12)])
def test_mxfp4_scales_from_end_to_end(xt, m):
    """Block exponents 0 to 254 beside tokens of 2^-118 to 2^122."""
    rng = np.random.default_rng(m)
    codes, scales, _, _ = _weights(rng, "mxfp4", 70, 640)
    scales[:60] = np.array([254, 252, 246, 240, 233, 232, 231, 192, 191, 190, 128, 127, 64, 63, 62,
                            20, 2, 1, 0, 112])[np.arange(60) % 20, None]
    scales[60:66] = rng.integers(0, 6, (6, 20)) + np.array([189, 61, 249, 0, 229, 28])[:, None]
    for powers in ([-60, -118, 0, 60], [122, -100, 90, -3]):
        _run("mxfp4", _tokens(rng, m, 640, powers, xt), (codes, scales, None, None))


@pytest.mark.parametrize("xt,m", [("bf16", 1), ("bf16", 8), ("f32", 4)])
def test_mxfp4_blocks_far_apart_in_a_group(xt, m):
    """A block of weight 2^127 beside blocks of 2^-127, where x is zero at the one or
    the codes are."""
    rng = np.random.default_rng(m)
    codes, scales, _, _ = _weights(rng, "mxfp4", 33, 256)
    scales[:, 0::4], scales[:, 1::4], scales[:, 2::4] = 254, 0, 130
    x = rng.standard_normal((m, 8, 32)) * 2.0 ** 30
    x[:, 0::4] = 0
    x = torch.from_numpy(x.reshape(m, 256)).cuda().to(KIND[xt])
    _run("mxfp4", x, (codes, scales, None, None))
    x = _tokens(rng, m, 256, [30], xt)
    codes = codes.reshape(33, 8, 32).copy()
    codes[:, 0::4] = rng.integers(0, 2, (33, 2, 32)) * 8            # 0 and -0
    _run("mxfp4", x, (codes.reshape(33, 256), scales, None, None))
