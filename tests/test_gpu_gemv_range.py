"""GPU: kq_gemv where x, the weights' scales or both are near the ends of fp32's
range, against the float64 oracle with the tolerance of tests/test_gpu_decode.py
(nothing is required where the magnitudes that are added reach 2^127).

To it comes what holding x in fp16 may take from elements far below their group's
largest, as include/kq.h states it.  A group (a token's 128 columns) is held times a
power of two that puts its largest element T in [2^14, 2^15).  fp16 steps by 2^-24
below 2^-14, so an element is off by at most 2^-25 there, which is 2^-39 T; by 16
times that, 2^-35 T, for INT4 with a bf16 result, where it is halved four times
before it is rounded.  (Where fp32 elements are two parts, the second is 2^11 times
what the first left, rounded the same way: 2^-50 T.)  Each weight w of the group takes
|w| times as much into the result.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from oracle import decode as od
from test_gpu_decode import KIND, _gemv, _magnitude, _weights

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
    x64, k = x.double().cpu().numpy(), x.shape[1]
    matrix = od.weights(fmt, *w)
    ref, mag = od.gemv(x64, matrix), _magnitude(fmt, x64, *w)
    tol = (2.0 ** -18 + (k / 128 + 16) * 2.0 ** -23) * mag + k * 2.0 ** -149
    step = 2.0 ** -35 if fmt.startswith("int4") and yt == "bf16" else \
        2.0 ** -39 if x.dtype == torch.bfloat16 else 2.0 ** -50
    for at in range(0, k, 128):
        top = np.abs(x64[:, at:at + 128]).max(1, keepdims=True)
        tol += step * top * np.abs(matrix[:, at:at + 128]).sum(1)
    if yt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    ok = (err <= tol) | (mag >= 2.0 ** 127)
    assert ok.all(), f"worst {(err / tol)[~ok].max()} x tolerance, {(~ok).sum()} outputs"
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


def _e2m1_weights(rng, fmt, n, k):
    """Small weights: products with 2^127 stay below 2^127."""
    codes, scales, _, t = _weights(rng, fmt, n, k)
    scales[:] = rng.integers(1, 9, scales.shape) if fmt == "nvfp4" else \
        rng.integers(80, 100, scales.shape)
    return codes, scales, None, t


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("xt,m", [("bf16", 3), ("bf16", 12), ("f32", 2), ("f32", 5), ("f32", 15)])
def test_e2m1_largest_tokens(fmt, xt, m):
    """Elements of 2^127 and of the type's largest value, one a token."""
    rng = np.random.default_rng(m)
    w = _e2m1_weights(rng, fmt, 50, 384)
    x = torch.from_numpy(rng.standard_normal((m, 384))).cuda().to(KIND[xt])
    for i in range(m):
        x[i, 29 * i % 384] = (2.0 ** 127, -torch.finfo(KIND[xt]).max, -2.0 ** 127, 2.0 ** 126)[i % 4]
    _run(fmt, x, w)
    _run(fmt, x, w, "bf16")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [3, 12])
@pytest.mark.parametrize("power", [15, 18, 24])
def test_e2m1_small_elements_beside_a_large_one(fmt, m, power):
    """bf16 elements of 8 significant bits beside one of 2^power that meets zero
    weights: they are 2^-power of it, and exact."""
    rng = np.random.default_rng(power)
    codes, scales, _, t = _weights(rng, fmt, 40, 256)
    codes[:, [0, 130]] = 0
    x = torch.full((m, 256), 1 + 2.0 ** -7, device="cuda")
    x[:, [0, 130]] = 2.0 ** power
    _run(fmt, x.bfloat16(), (codes, scales, None, t))


@pytest.mark.parametrize("fmt", ["int4_asym", "int4_sym", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("m", [3, 12])
def test_infinities_and_nan_stay_in_their_token(fmt, xt, yt, m):
    """A token with an infinity or a NaN has no finite result; the others have theirs,
    bit by bit."""
    rng = np.random.default_rng(m)
    w = _weights(rng, fmt, 37, 512)
    x = torch.from_numpy(rng.standard_normal((m, 512))).cuda().to(KIND[xt])
    want = _run(fmt, x, w, yt)
    bad = {0: float("inf"), 2: float("nan"), m - 1: -float("inf")}
    for token, value in bad.items():
        x[token, 100 * token % 512] = value
    got = torch.zeros_like(want)
    _gemv(fmt, x, *w, got)
    for i in range(m):
        if i in bad:
            assert not torch.isfinite(got[i]).any()
        else:
            assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [2, 12])
def test_e2m1_infinities_have_their_sign(fmt, m):
    """bf16 x of one infinity, weights that are not zero there."""
    rng = np.random.default_rng(m)
    codes, scales, _, t = _weights(rng, fmt, 37, 256)
    scales[scales == 0] = 1
    codes[:, 77] = rng.integers(1, 8, 37) + 8 * rng.integers(0, 2, 37)
    scales[:, 77 // (16 if fmt == "nvfp4" else 32)] = scales.max(1)
    x = torch.zeros((m, 256), dtype=torch.bfloat16, device="cuda")
    x[0, 77], x[1, 77] = float("inf"), -float("inf")
    y = torch.zeros((m, 37), device="cuda")
    _gemv(fmt, x, codes, scales, None, t, y)
    sign = torch.from_numpy(np.where(codes[:, 77] < 8, np.inf, -np.inf)).float().cuda()
    assert torch.equal(y[0], sign) and torch.equal(y[1], -sign) and not y[2:].any()


@pytest.mark.parametrize("fmt", ["int4_asym", "int4_sym", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("xt,m,yt", [("bf16", 4, "f32"), ("bf16", 4, "bf16"), ("bf16", 12, "f32"),
                                     ("bf16", 12, "bf16"), ("f32", 4, "f32"), ("f32", 6, "bf16"),
                                     ("f32", 13, "f32"), ("f32", 13, "bf16")])
def test_tokens_over_the_range_that_is_stated(fmt, xt, m, yt):
    """Group maxima up to 2^97 and down to 2^-100, beside scales that take the result
    the other way (and beside ordinary ones)."""
    rng = np.random.default_rng(m)
    for power, down in ([94, -60], [94, -14], [94, 0], [60, -90], [-60, 90], [-99, 60], [-99, 14],
                        [-99, 0], [0, 100], [0, -100]):
        codes, scales, zeros, t = _weights(rng, fmt, 60, 640)
        if fmt == "int4_asym":
            scales = np.ldexp(rng.uniform(0.5, 1, scales.shape),
                              np.clip(down, -14, 15)).astype(np.float16)
        elif fmt == "int4_sym":
            scales = np.ldexp(rng.uniform(0.5, 1, 60),
                              down + rng.integers(-9, 9, 60)).astype(np.float32)
        elif fmt == "nvfp4":
            t = np.float32(np.ldexp(0.7, down - 8))
        else:
            scales = (127 + down + rng.integers(-5, 5, scales.shape)).astype(np.uint8)
        _run(fmt, _tokens(rng, m, 640, [power, power], xt).clamp(-2.0 ** 97, 2.0 ** 97),
             (codes, scales, zeros, t), yt)


@pytest.mark.parametrize("fmt", ["int4_asym", "int4_sym", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("n,k,m,xt", [(70, 4096, 5, "bf16"), (70, 2560, 11, "f32"),
                                      (100, 32768, 16, "f32"), (40, 131072, 3, "bf16"),
                                      (12007, 2048, 16, "bf16")])
def test_far_groups_beside_near_ones(fmt, n, k, m, xt):
    """Tokens whose groups are near 1, 2^80 and 2^-80 in turn along k: split over the
    CTAs of a cluster, over segments of x and over rounds of rows."""
    if fmt != "nvfp4":
        n = min(n, 4000)
    rng = np.random.default_rng(k)
    w = _weights(rng, fmt, n, k)
    x = rng.standard_normal((m, k // 512, 512))
    for i in range(m):
        x[i] *= np.exp2(rng.choice([0, 80, -80] if i % 3 == 0 else [0, -80] if i % 3 == 1 else [0],
                                   k // 512))[:, None]
    _run(fmt, torch.from_numpy(x.reshape(m, k)).cuda().to(KIND[xt]), w)


@pytest.mark.parametrize("fmt", ["int4_sym", "nvfp4"])
def test_zero_and_infinite_scales(fmt):
    """A row's or the tensor's scale of zero, infinity or NaN reaches that row (all rows)
    and no other."""
    rng = np.random.default_rng(1)
    codes, scales, _, t = _weights(rng, fmt, 40, 256)
    x = _tokens(rng, 3, 256, [0, 90, -90], "bf16")
    if fmt == "int4_sym":
        scales[3], scales[17], scales[39] = 0, np.inf, np.nan
        y = torch.empty((3, 40), device="cuda")
        _gemv(fmt, x, codes, scales, None, t, y)
        assert not y[:, 3].any() and y[:, 39].isnan().all() and not torch.isfinite(y[:, 17]).any()
        scales[17] = scales[39] = 1
        _run(fmt, x, (codes, scales, None, t))
    else:
        assert not _run(fmt, x, (codes, scales, None, np.float32(0))).any()
