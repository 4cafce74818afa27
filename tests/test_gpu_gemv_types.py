"""GPU: kq_gemv with x and y of different types, against the float64 oracle.

The tolerance is that of tests/test_gpu_decode.py, and for INT4 with a bf16 result what
its operands cost besides.  They are masked codes, u or 16 u times 2^-24, which
the tensor core lines up with the others as if they began at 2^-14: a sum of 16 such
products keeps 25 bits from the largest exponent on, so each of them loses less than
2^-24 2^-14 of the group's largest |x|, in units of 2^-24 of the result (for the upper
codes x is divided by 16 first): 2^-14 X a column, 128 2^-14 X s a group.  As the losses
of a group are not aligned, the whole is asked to be within one bf16 step as well.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from oracle import decode as od
from test_gpu_decode import FMT, KIND, _gemv, _magnitude, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _check(fmt, x, w, y):
    codes, scales, zeros, t = w
    n, k = codes.shape
    ref = od.gemv(x, od.weights(fmt, codes, scales, zeros, t))
    tol = (2.0 ** -18 + (k / 128 + 16) * 2.0 ** -23) * _magnitude(fmt, x, codes, scales, zeros, t)
    if y.dtype == torch.bfloat16:
        if fmt.startswith("int4"):
            for g in range(-(-k // 128)):
                top = np.abs(x[:, 128 * g:128 * g + 128]).max(1)
                s = (scales if fmt == "int4_sym" else scales[:, g]).astype(np.float64)
                tol = tol + 128 * 2.0 ** -14 * top[:, None] * s[None, :]
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max()} x tolerance"
    if y.dtype == torch.bfloat16:
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(ref)


@pytest.mark.parametrize("fmt", sorted(FMT))
@pytest.mark.parametrize("n,k,m", [(1, 128, 1), (7, 128, 16), (16, 256, 2), (129, 384, 5),
                                   (64, 1152, 8), (300, 4096, 1), (250, 12288, 4), (40, 2176, 9),
                                   (513, 1024, 13), (333, 1536, 16)])
@pytest.mark.parametrize("xt,yt", [("f32", "bf16"), ("bf16", "f32")])
def test_types_differ(fmt, n, k, m, xt, yt):
    rng = np.random.default_rng(n * k + m)
    w = _weights(rng, fmt, n, k)
    x = torch.from_numpy(rng.standard_normal((m, k))).cuda().to(KIND[xt])
    y = torch.full((m, n), float("nan"), dtype=KIND[yt], device="cuda")
    _gemv(fmt, x, *w, y)
    _check(fmt, x.double().cpu().numpy(), w, y)


@pytest.mark.parametrize("fmt", ["int4_asym", "int4_sym"])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_every_number_of_tokens_to_bf16(fmt, xt):
    """128 columns: one rank, 1536: two, 4096: four; sums travel two tokens or one a
    store."""
    rng = np.random.default_rng(4)
    for k in (128, 1536, 4096):
        w = _weights(rng, fmt, 333, k)
        for m in range(1, 17):
            x = torch.from_numpy(rng.standard_normal((m, k))).cuda().to(KIND[xt])
            buf = torch.full((m * 333 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
            y = buf[32:32 + m * 333].view(m, 333)
            _gemv(fmt, x, *w, y)
            _check(fmt, x.double().cpu().numpy(), w, y)
            assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


@pytest.mark.parametrize("fmt", ["int4_sym", "int4_asym"])
@pytest.mark.parametrize("n,k,m", [(33000, 896, 16), (60011, 128, 16), (100, 32768, 16),
                                   (12000, 2048, 11)])
def test_fp32_tokens_to_bf16_in_rounds_and_segments(fmt, n, k, m):
    rng = np.random.default_rng(n + k)
    codes, scales, zeros, t = _weights(rng, fmt, n, k)
    x = torch.from_numpy(rng.standard_normal((m, k))).cuda().float()
    y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    _gemv(fmt, x, codes, scales, zeros, t, y)
    assert torch.isfinite(y).all()
    rows = np.unique(np.concatenate([np.arange(min(n, 20)), rng.integers(0, n, 100),
                                     np.arange(n - 40, n)]))
    part = codes[rows], scales[rows], None if zeros is None else zeros[rows], t
    _check(fmt, x.double().cpu().numpy(), part, y[:, torch.from_numpy(rows).cuda()])
