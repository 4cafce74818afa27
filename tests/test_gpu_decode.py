"""GPU: the decode-step operators against the float64 oracle.

Tolerance of kq_gemv.  fp32 rows are held as two fp16 parts (22 significant
bits, 2^-22 relative), bf16 rows exactly.  Weights are exact.  Let A be the sum
of the magnitudes that are added: |x| s (u + |z|) for the asymmetric format
(the zero point is subtracted as a separate sum), |x| s (q + 16) for the
symmetric one (offset codes), |x w| for the others.  An accumulation inside a
128-wide group takes at most 8 tensor-core steps, each losing under 2^-21 of
the magnitudes so far; groups and warps are joined in fp32, at most K / 128 + 16
further roundings of 2^-23 in all (scale products included).  So
  |y - y_ref| <= (2^-18 + (K / 128 + 16) 2^-23) A,  bf16 output + 2^-8 |y|,
inside fp32's range (see _check_gemv).

Tolerance of the attention.  The rotated query is rounded to fp16 (2^-11
relative per element) and so are the softmax weights times the value scale;
scores and sums add in fp32 with under 2^-17 of their magnitudes lost (steps of
the kind above, then subtraction of the zero point's part).  With
  d_t = scale sk_t sum_d |q'_d| (2^-11 |u - z| + 2^-17 (u + |z|))
the weights are off by at most e^{2 max d} - 1 + 2^-11, the value of dimension d
by sum_t w_t sv_t ((e^{2 max d} - 1 + 2^-11) |u - z| + 2^-17 (u + |z|)), and the
inverse rotation adds 128 such errors with weight 1 / sqrt(128).  bf16 output
adds 2^-8 of the value.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
import oracle
from oracle import decode as od

pytestmark = pytest.mark.gpu

FMT = {"int4_sym": kq.KQ_FMT_INT4_SYM, "int4_asym": kq.KQ_FMT_INT4_ASYM,
       "nvfp4": kq.KQ_FMT_NVFP4, "mxfp4": kq.KQ_FMT_MXFP4}
KIND = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------- gemv
def _weights(rng, fmt, n, k):
    codes = rng.integers(0, 16, (n, k))
    if fmt == "int4_sym":
        return codes, rng.lognormal(-3, 1, n).astype(np.float32), None, None
    if fmt == "int4_asym":
        return (codes, rng.lognormal(-3, 1, (n, k // 128)).astype(np.float16),
                np.rint(rng.uniform(-2, 17, (n, k // 128))).astype(np.float16), None)
    if fmt == "nvfp4":
        return codes, rng.integers(0, 0x7F, (n, k // 16)).astype(np.uint8), None, \
            np.float32(1.37e-3)
    return codes, rng.integers(112, 132, (n, k // 32)).astype(np.uint8), None, None


def _magnitude(fmt, x, codes, scales, zeros, t):
    n, k = codes.shape
    if fmt == "int4_asym":
        s = scales.astype(np.float64)[..., None]
        w = ((codes.reshape(n, k // 128, 128) + np.abs(zeros.astype(np.float64))[..., None]) *
             s).reshape(n, k)
    elif fmt == "int4_sym":
        w = (np.where(codes >= 8, 16 - codes, codes) + 16) * scales.astype(np.float64)[:, None]
    else:
        w = np.abs(od.weights(fmt, codes, scales, zeros, t))
    return np.abs(x) @ w.T


def _gemv(fmt, x, codes, scales, zeros, t, y, stream=None):
    kq.kq_gemv(FMT[fmt], x, _dev(oracle.pack_nibbles(codes)), _dev(scales),
               None if zeros is None else _dev(zeros),
               None if t is None else torch.tensor([float(t)], device="cuda"),
               128 if fmt == "int4_asym" else 0, y, stream=stream)


def _check_gemv(fmt, x, w, y):
    codes, scales, zeros, t = w
    ref = od.gemv(x, od.weights(fmt, codes, scales, zeros, t))
    mag = _magnitude(fmt, x, codes, scales, zeros, t)
    tol = (2.0 ** -18 + (codes.shape[1] / 128 + 16) * 2.0 ** -23) * mag
    # fp32's range: each of the k products and joins may lose one subnormal step
    # (2^-149), and where the magnitudes add up to 2^127 or more a partial sum
    # need not be representable, so nothing is required of the result there
    tol = np.where(mag < 2.0 ** 127, tol + codes.shape[1] * 2.0 ** -149, np.inf)
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    ok = (err <= tol) | np.isinf(tol)
    assert ok.all(), f"worst {(err / tol)[~ok].max()} x tolerance, {(~ok).sum()} outputs"


@pytest.mark.parametrize("fmt", sorted(FMT))
@pytest.mark.parametrize("n,k,m", [(1, 128, 1), (7, 128, 16), (16, 256, 2), (17, 512, 3),
                                   (129, 384, 5), (64, 1152, 8), (300, 4096, 1), (250, 12288, 4),
                                   (40, 2176, 9), (513, 1024, 13)])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32")])
def test_gemv(fmt, n, k, m, xt, yt):
    rng = np.random.default_rng(n * k + m)
    w = _weights(rng, fmt, n, k)
    x = torch.from_numpy(rng.standard_normal((m, k))).cuda()
    x[:, rng.integers(0, k, 3)] *= 40
    x = x.to(KIND[xt])
    y = torch.full((m, n), float("nan"), dtype=KIND[yt], device="cuda")
    _gemv(fmt, x, *w, y)
    _check_gemv(fmt, x.double().cpu().numpy(), w, y)


@pytest.mark.parametrize("fmt", ["int4_sym", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("k", [32, 64, 96, 160, 416, 1056])
def test_gemv_rows_that_end_inside_a_group(fmt, k):
    rng = np.random.default_rng(k)
    w = _weights(rng, fmt, 37, k)
    x = torch.from_numpy(rng.standard_normal((6, k))).cuda().float()
    y = torch.empty((6, 37), device="cuda")
    _gemv(fmt, x, *w, y)
    _check_gemv(fmt, x.double().cpu().numpy(), w, y)


def test_gemv_extremes():
    """A zero row of x, magnitudes far apart in one row and between rows, zero
    scales, the largest block scales."""
    rng = np.random.default_rng(5)
    for fmt in sorted(FMT):
        codes, scales, zeros, t = _weights(rng, fmt, 33, 512)
        scales = scales.copy()
        scales[3] = 0
        if fmt == "nvfp4":
            scales[4] = 0x7E
            scales[5] = 1
        if fmt == "mxfp4":
            scales[4], scales[5] = 190, 60
        x = rng.standard_normal((4, 512))
        x[0] = 0
        x[1] *= 2.0 ** 60
        x[2] *= 2.0 ** -60
        x[3, ::2] *= 2.0 ** -12
        x = torch.from_numpy(x).cuda().float()
        y = torch.empty((4, 33), device="cuda")
        _gemv(fmt, x, codes, scales, zeros, t, y)
        _check_gemv(fmt, x.double().cpu().numpy(), (codes, scales, zeros, t), y)
        assert not y[0].any()


def test_gemv_is_reproducible_and_stays_in_its_output():
    rng = np.random.default_rng(6)
    for fmt in sorted(FMT):
        w = _weights(rng, fmt, 131, 768)
        x = torch.from_numpy(rng.standard_normal((3, 768))).cuda().bfloat16()
        buf = torch.full((3 * 131 + 256,), 7.0, device="cuda")
        y = buf[128:128 + 3 * 131].view(3, 131)
        _gemv(fmt, x, *w, y)
        first = y.clone()
        _gemv(fmt, x, *w, y)
        assert torch.equal(first, y)
        assert (buf[:128] == 7).all() and (buf[-128:] == 7).all()
        # a token's result does not depend on the tokens beside it
        one = torch.empty((1, 131), device="cuda")
        _gemv(fmt, x[1:2].contiguous(), *w, one)
        assert torch.equal(one[0], y[1])


# -------------------------------------------------------------- attention
def _cache(rng, slots, heads):
    codes = rng.integers(0, 16, (slots, heads * 128))
    scales = rng.lognormal(-2, 0.7, (slots, heads)).astype(np.float16)
    zeros = np.rint(rng.uniform(3, 12, (slots, heads))).astype(np.float16)
    return codes, scales, zeros


def _upload(cache):
    codes, scales, zeros = cache
    return kq.KVCacheInt4(_dev(oracle.pack_nibbles(codes)), _dev(scales), _dev(zeros))


def _table(rng, lens, page, pool, width):
    ids = rng.permutation(pool)
    table, at = np.full((len(lens), width), -1, dtype=np.int32), 0
    for b, v in enumerate(lens):
        n = -(-max(0, v) // page)
        table[b, :n] = ids[at:at + n]
        at += n
    assert at <= pool
    return table


def _attn_tolerance(q, k, v, ks, table, page, lens, scale, window, sinks):
    batch, q_heads, _ = q.shape
    slots, heads = k[1].shape
    group = q_heads // heads
    h = oracle.sylvester(128) / math.sqrt(128)
    tol = np.zeros_like(q)
    for b in range(batch):
        rows = od.cache_rows(table[b], page, slots,
                             od.visible(min(int(lens[b]), table.shape[1] * page), window, sinks))
        rows = rows[rows >= 0]
        if not rows.size:
            continue
        for i in range(heads):
            sl = slice(i * 128, (i + 1) * 128)
            sg = np.ones(128) if ks is None else ks[sl].astype(np.float64)
            qr = (q[b, i * group:(i + 1) * group] * sg) @ h
            parts = []
            for codes, s, z in (k, v):
                u = codes[rows, sl].astype(np.float64)
                z64 = z[rows, i].astype(np.float64)[:, None]
                s64 = s[rows, i].astype(np.float64)[:, None]
                parts.append((s64 * np.abs(u - z64), s64 * (u + np.abs(z64)), s64 * (u - z64)))
            (kd, km, kk), (vd, vm, _) = parts
            d = abs(scale) * (np.abs(qr) @ (2.0 ** -11 * kd + 2.0 ** -17 * km).T)
            a = scale * (qr @ kk.T)
            p = np.exp(a - a.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            rel = np.exp(2 * d.max(1, keepdims=True)) - 1 + 2.0 ** -11
            e = rel * (p @ vd) + 2.0 ** -17 * (p @ vm)
            tol[b, i * group:(i + 1) * group] = e.sum(1, keepdims=True) / math.sqrt(128)
    return tol


def _check_attn(out, q, k, v, ks, vs, table, page, lens, scale, window, sinks):
    ref = od.attn_decode(q, k, v, ks, vs, table, page, lens, scale, window, sinks)
    tol = _attn_tolerance(q, k, v, ks, table, page, lens, scale, window, sinks)
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = out.double().cpu().numpy()
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    ok = err <= tol
    assert ok.all(), f"worst {(err / tol)[~ok].max()} x tolerance, {(~ok).sum()} outputs"
    # the bound above adds worst cases; on these inputs the errors are far from
    # aligned, and the whole is within a bf16 step
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(err) <= 2.0 ** -7 * norm


def _attn(q, kc, vc, ks, vs, table, page, lens, scale, window=0, sinks=0, ws=None, out=None,
          stream=None):
    out = torch.full_like(q, float("nan")) if out is None else out
    ws = ws if ws is not None else kq.empty_attn_workspace(q.shape[0], q.shape[1], kc.dim // 128)
    kq.kq_attn_decode_int4_kv(q, kc, vc, ks, vs, table, page, lens, scale, out, ws, window=window,
                              sinks=sinks, stream=stream)
    return out


def _case(seed, lens, heads, group, page, window=0, sinks=0, signs=True, spare=5, extra_width=0):
    rng = np.random.default_rng(seed)
    pool = sum(-(-max(0, v) // page) for v in lens) + spare
    width = max(1, max(-(-max(0, v) // page) for v in lens) + extra_width)
    k, v = _cache(rng, pool * page, heads), _cache(rng, pool * page, heads)
    table = _table(rng, lens, page, pool, width)
    q = torch.from_numpy(rng.standard_normal((len(lens), heads * group, 128))).cuda().bfloat16()
    ks, vs = ((rng.integers(0, 2, heads * 128) * 2 - 1).astype(np.int8) if signs else None
              for _ in range(2))
    return q, k, v, ks, vs, table, np.array(lens, dtype=np.int32)


def _run_case(q, k, v, ks, vs, table, lens, page, scale, window=0, sinks=0, **kw):
    return _attn(q, _upload(k), _upload(v), None if ks is None else _dev(ks),
                 None if vs is None else _dev(vs), _dev(table), page, _dev(lens), scale, window,
                 sinks, **kw)


def _whole(seed, lens, heads, group, page, window=0, sinks=0, scale=128 ** -0.5, **kw):
    q, k, v, ks, vs, table, lens = _case(seed, lens, heads, group, page, window, sinks, **kw)
    out = _run_case(q, k, v, ks, vs, table, lens, page, scale, window, sinks)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, page, lens, scale, window,
                sinks)


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 8), (2, 3), (3, 2), (4, 4), (5, 5), (6, 1),
                                         (8, 1), (8, 4), (8, 8), (12, 2), (16, 2), (2, 16), (1, 20),
                                         (32, 1)])
def test_attention_head_layouts(heads, group):
    _whole(heads * 100 + group, [1, 33, 150, 0, 17], heads, group, 16)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 32, 50, 64, 128, 1000])
def test_attention_pages(page):
    _whole(page, [200, 1, 31, 32, 33, 129, 63, 64, 65], 8, 2, page)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [32], [33], [127], [128],
                                  [129], [255], [256], [257], [1000], [0], [0, 0, 3]])
def test_attention_lengths(lens):
    _whole(sum(lens), lens, 2, 4, 16)
    _whole(sum(lens) + 1, lens, 8, 4, 16)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 4), (64, 0), (100, 1),
                                          (40, 17), (500, 4), (3, 1000), (0, 9)])
def test_attention_window_and_sinks(window, sinks):
    _whole(window + sinks, [1, 5, 40, 64, 200, 0, 333, 104], 8, 4, 16, window, sinks)
    _whole(window + sinks, [1, 5, 40, 64, 200, 0, 333, 104], 1, 3, 7, window, sinks)


@pytest.mark.parametrize("batch,heads,group", [(1, 8, 4), (3, 2, 8), (130, 8, 1), (70, 1, 2)])
def test_attention_many_and_long(batch, heads, group):
    """One sequence over every multiprocessor, and more sequences than those."""
    rng = np.random.default_rng(batch)
    lens = [9000] if batch == 1 else [int(v) for v in np.exp(rng.uniform(0, 6, batch))] + [2500]
    _whole(batch, lens, heads, group, 32)


def test_attention_without_signs_and_other_scales():
    _whole(1, [70, 9], 8, 2, 16, signs=False)
    _whole(2, [70, 9], 8, 2, 16, scale=0.0)
    _whole(3, [70, 9], 8, 2, 16, scale=-0.05)


def test_attention_peaked_and_flat_weights():
    """A first token with most of the weight and a small value scale, and many
    tokens far below it that carry the values between them."""
    for down in (4.0, 9.0):
        q, k, v, ks, vs, table, lens = _case(7, [3000], 2, 2, 16)
        h = oracle.sylvester(128) / math.sqrt(128)
        row0 = int(table[0, 0]) * 16
        qr = (q[0, 0].double().cpu().numpy() * ks[:128]) @ h
        codes, scales, zeros = k
        codes[row0, :128] = np.clip(np.rint(qr * 3) + 8, 0, 15)
        zeros[row0, 0] = 8
        a0 = qr @ (codes[row0, :128] - 8.0) / math.sqrt(128)
        scales[row0, 0] = np.float16(down / a0)
        v[1][row0, 0] = np.float16(2.0 ** -14)
        out = _run_case(q, k, v, ks, vs, table, lens, 16, 128 ** -0.5)
        _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, lens, 128 ** -0.5, 0,
                    0)


def test_attention_value_scales_far_apart():
    rng = np.random.default_rng(8)
    q, k, v, ks, vs, table, lens = _case(8, [400, 90], 8, 4, 16)
    v[1][:] = np.exp2(rng.integers(-14, 12, v[1].shape)).astype(np.float16)
    v[1][::5] = 0
    out = _run_case(q, k, v, ks, vs, table, lens, 16, 128 ** -0.5)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, lens, 128 ** -0.5, 0, 0)
    v[1][:] = 0                     # every value is zero
    out = _run_case(q, k, v, ks, vs, table, lens, 16, 128 ** -0.5)
    assert not out.any()


def test_attention_flat_rows_and_far_zero_points():
    """Rows the writer makes of constant heads: scale 0, or a zero point far
    outside the codes."""
    q, k, v, ks, vs, table, lens = _case(9, [130, 40], 8, 2, 16)
    k[1][::3] = 0
    for c in (k, v):
        c[1][1::3] = np.float16(2.0 ** -7)
        c[2][1::3] = -600
    out = _run_case(q, k, v, ks, vs, table, lens, 16, 128 ** -0.5)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, lens, 128 ** -0.5, 0, 0)


@pytest.mark.parametrize("heads,group", [(8, 4), (1, 4), (2, 16)])
def test_attention_ignores_what_is_not_visible(heads, group):
    """NaN and infinities in rows behind the last token, in unused pages, in
    tokens the window hides; lengths and table entries out of range."""
    page, window, sinks = 16, 40, 3
    q, k, v, ks, vs, table, lens = _case(10, [5, 100, 333, 64, 20], heads, group, page,
                                         extra_width=2)
    want = _run_case(q, k, v, ks, vs, table, lens, page, 0.1, window, sinks)
    _check_attn(want, q.double().cpu().numpy(), k, v, ks, vs, table, page, lens, 0.1, window,
                sinks)
    seen = np.zeros(k[1].shape[0], dtype=bool)
    for b in range(len(lens)):
        seen[od.cache_rows(table[b], page, len(seen), od.visible(lens[b], window, sinks))] = True
    dirty = []
    for codes, scales, zeros in (k, v):
        codes, scales, zeros = codes.copy(), scales.copy(), zeros.copy()
        codes[~seen] = 15
        scales[~seen] = np.nan
        zeros[~seen] = np.inf
        dirty.append((codes, scales, zeros))
    hidden = table.copy()
    for b in range(len(lens)):
        for p in range(hidden.shape[1]):
            if not np.intersect1d(od.visible(lens[b], window, sinks),
                                  np.arange(p * page, (p + 1) * page)).size:
                hidden[b, p] = 2 ** 30 if p % 2 else -7
    got = _run_case(q, *dirty, ks, vs, hidden, lens, page, 0.1, window, sinks)
    assert torch.equal(got, want)


def test_attention_bad_pages_and_lengths():
    page = 8
    q, k, v, ks, vs, table, lens = _case(11, [100, 40, 24, 9], 8, 2, page)
    slots = k[1].shape[0]
    table[0, 3], table[0, 5] = -1, slots // page          # one page before, one behind the cache
    table[1, :] = 2 ** 31 - 1                             # nothing there
    table[3, :] = -2 ** 31
    lens = np.array([100, 40, 2 ** 31 - 1, -5], dtype=np.int32)
    out = _run_case(q, k, v, ks, vs, table, lens, page, 0.1)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, page, lens, 0.1, 0, 0)
    assert not out[1].any() and not out[3].any()
    # num_slots that ends inside a page: the rows behind it are not visible
    q, k, v, ks, vs, table, lens = _case(12, [64, 30], 2, 2, 16)
    k, v = (tuple(a[:-83] for a in c) for c in (k, v))
    out = _run_case(q, k, v, ks, vs, table, lens, 16, 0.1)
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, lens, 0.1, 0, 0)


def test_attention_workspace_streams_and_graph():
    """The result does not depend on what the workspace holds, on the stream, or
    on replaying a graph after lengths, pages and the cache changed in place."""
    page = 16
    q, k, v, ks, vs, table, lens = _case(13, [500, 3, 77, 2000], 8, 4, page)
    want = _run_case(q, k, v, ks, vs, table, lens, page, 0.1)
    kc, vc, ksd, vsd, td, ld = _upload(k), _upload(v), _dev(ks), _dev(vs), _dev(table), _dev(lens)
    ws = kq.empty_attn_workspace(4, 32, 8)
    for fill in (0, 255, 0x7F):
        ws.fill_(fill)
        assert torch.equal(_attn(q, kc, vc, ksd, vsd, td, page, ld, 0.1, ws=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    _attn(q, kc, vc, ksd, vsd, td, page, ld, 0.1, ws=ws, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _attn(q, kc, vc, ksd, vsd, td, page, ld, 0.1, ws=ws, out=out)
    for new in ([500, 3, 77, 2000], [1, 0, 50, 1999], [33, 3, 0, 0], [500, 2, 77, 64]):
        ld.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        new = np.array(new, dtype=np.int32)
        _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, page, new, 0.1, 0, 0)


def test_attention_output_stays_in_place():
    q, k, v, ks, vs, table, lens = _case(14, [50, 9, 300], 8, 3, 16)
    buf = torch.full((256 + q.numel() + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[256:256 + q.numel()].view(q.shape)
    need = kq.kq_attn_workspace_size(3, 24, 8)
    wbuf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    _run_case(q, k, v, ks, vs, table, lens, 16, 0.1, out=out, ws=wbuf[4096:4096 + need])
    assert (buf[:256] == 7).all() and (buf[-256:] == 7).all()
    assert (wbuf[:4096] == 0x5A).all() and (wbuf[-4096:] == 0x5A).all()


# ------------------------------------------------------------- page copies
@pytest.mark.parametrize("layers,page,heads,pages", [(1, 1, 1, 9), (2, 16, 8, 40), (3, 7, 3, 21),
                                                     (1, 128, 32, 6), (4, 5, 5, 33)])
@pytest.mark.parametrize("tail", [0, 1])
@pytest.mark.parametrize("values", [True, False])
def test_copy_pages(layers, page, heads, pages, tail, values):
    rng = np.random.default_rng(pages + tail)
    slots = pages * page + (page // 2 if tail else 0)      # a last page that is not whole
    caches = [kq.empty_kv_cache(slots, heads * 128, layers) for _ in range(2)]
    before = []
    for c in caches:
        for a in (c.codes, c.scales, c.zeros):
            a.view(torch.uint8).copy_(torch.from_numpy(
                rng.integers(0, 256, a.view(torch.uint8).shape, dtype=np.uint8)))
            before.append(a.view(torch.uint8).cpu().numpy())
    ids = rng.permutation(pages)
    n = pages // 2 - 1
    pairs = [(ids[i], ids[n + i]) for i in range(n)]
    pairs += [(-1, ids[-1]), (ids[0], pages), (ids[0], -5), (2 ** 31 - 1, ids[-1]), (ids[-1],) * 2]
    pairs = np.array(pairs, dtype=np.int32)
    kq.kq_kv_copy_pages(_dev(pairs), page, caches[0], caches[1] if values else None)
    after = [a.view(torch.uint8).cpu().numpy() for c in caches for a in (c.codes, c.scales, c.zeros)]
    for i, (x, y) in enumerate(zip(before, after)):
        assert np.array_equal(y, od.copy_pages(x, pairs, page) if values or i < 3 else x), i


def test_copy_pages_nothing_to_do():
    c = kq.empty_kv_cache(64, 256)
    c.codes.zero_()
    kq.kq_kv_copy_pages(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 16, c)
    kq.kq_kv_copy_pages(torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), 128, c)
    assert not c.codes.any()


# ------------------------------------------------------ refused by the binding
def test_binding_refuses_wrong_tensors():
    rng = np.random.default_rng(0)
    w = _weights(rng, "int4_asym", 8, 256)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(2, 8, device="cuda")
    codes, s, z = _dev(oracle.pack_nibbles(w[0])), _dev(w[1]), _dev(w[2])
    bad = [(x[:, ::2], codes, s, z, y), (x, codes[:, :64], s, z, y), (x, codes, s[:4], z, y),
           (x, codes, s, s.float(), y), (x, codes, s, z, y.t()), (x, codes, s, z, y[:1]),
           (x.half(), codes, s, z, y), (x, codes, s.cpu(), z, y)]
    for args in bad:
        with pytest.raises(ValueError):
            kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, *args[:4], None, 128, args[4])
    q, k, v, ks, vs, table, lens = _case(1, [20, 3], 2, 2, 16)
    kc, vc, ksd, vsd, t, n = _upload(k), _upload(v), _dev(ks), _dev(vs), _dev(table), _dev(lens)
    ok = dict(q=q, k_cache=kc, v_cache=vc, k_signs=ksd, v_signs=vsd, block_table=t, page_size=16,
              seq_lens=n, softmax_scale=0.1, out=torch.empty_like(q),
              workspace=kq.empty_attn_workspace(2, 4, 2))
    kq.kq_attn_decode_int4_kv(**ok)
    small = kq.KVCacheInt4(kc.codes[:16], kc.scales[:16], kc.zeros[:16])
    for change in (dict(q=q.float()), dict(q=q[:, :3].contiguous()), dict(out=ok["out"][:1]),
                   dict(block_table=t.long()), dict(block_table=t[:1]), dict(seq_lens=n[:1]),
                   dict(seq_lens=n.long()), dict(v_cache=small), dict(k_signs=ksd[:128]),
                   dict(v_signs=vsd.float())):
        with pytest.raises((ValueError, kq.KQError)):
            kq.kq_attn_decode_int4_kv(**{**ok, **change})
    with pytest.raises(kq.KQError):
        kq.kq_attn_decode_int4_kv(**{**ok, "workspace": ok["workspace"][:8]})
    layered = kq.empty_kv_cache(32, 256, 2)
    with pytest.raises(ValueError):
        kq.kq_attn_decode_int4_kv(**{**ok, "k_cache": layered})
    with pytest.raises(ValueError):
        kq.kq_kv_copy_pages(torch.zeros(2, 2, device="cuda"), 16, kc)
    with pytest.raises(ValueError):
        kq.kq_kv_copy_pages(torch.zeros(2, 2, dtype=torch.int32, device="cuda"), 16, kc, small)


# --------------------------------------------------------- used together
def test_decode_step_together():
    """Prompts written into pages by the library's writer, one of them forked by
    a page copy, a new token appended to each, attention over the cache, and an
    output projection on the rotated result -- against the oracle on the same
    cache contents, and against attention of the unquantized heads."""
    rng = np.random.default_rng(21)
    heads, group, page, layers = 8, 2, 16, 2
    dim, layer = heads * 128, 1
    signs = [torch.from_numpy((rng.integers(0, 2, dim) * 2 - 1).astype(np.int8)).cuda()
             for _ in range(2)]
    lens = [41, 90]
    pool = 16
    caches = [kq.empty_kv_cache(pool * page, dim, layers) for _ in range(2)]
    for c in caches:
        for a in (c.codes, c.scales, c.zeros):
            a.zero_()
    ids = [int(v) for v in rng.permutation(pool)]
    table = np.full((3, 6), -1, dtype=np.int32)
    table[0, :3], table[1, :6] = ids[:3], ids[3:9]
    raw = [[torch.from_numpy(rng.standard_normal((n, dim))).cuda().bfloat16() for n in lens]
           for _ in range(2)]

    def write(seq, x, first):
        pos = np.arange(first, first + x[0].shape[0])
        slots = _dev(table[seq, pos // page].astype(np.int64) * page + pos % page)
        for c, s, rows in zip(caches, signs, x):
            at = c.layer(layer)
            kq.kq_rht_quant_int4_kv(rows, s, slots, at.codes, at.scales, at.zeros)
    for seq in range(2):
        write(seq, [raw[0][seq], raw[1][seq]], 0)
    # sequence 2 is a fork of sequence 0: whole pages shared, the last one copied
    table[2, :3] = table[0, 0], table[0, 1], ids[9]
    kq.kq_kv_copy_pages(_dev(np.array([[table[0, 2], ids[9]]], dtype=np.int32)), page, *caches)
    new = [torch.from_numpy(rng.standard_normal((3, dim))).cuda().bfloat16() for _ in range(2)]
    length = [41, 90, 41]
    for seq in range(3):
        write(seq, [new[0][seq:seq + 1], new[1][seq:seq + 1]], length[seq])
    length = np.array(length, dtype=np.int32) + 1
    q = torch.from_numpy(rng.standard_normal((3, heads * group, 128))).cuda().bfloat16()
    kc, vc = caches[0].layer(layer), caches[1].layer(layer)
    out = _attn(q, kc, vc, *signs, _dev(table), page, _dev(length), 128 ** -0.5)
    host = [(oracle.unpack_nibbles(c.codes.cpu().numpy()), c.scales.cpu().numpy(),
             c.zeros.cpu().numpy()) for c in (kc, vc)]
    sg = [s.cpu().numpy() for s in signs]
    _check_attn(out, q.double().cpu().numpy(), *host, *sg, table, page, length, 128 ** -0.5, 0, 0)
    # the quantizer's error bound: half a step of 4 bits over a head's range
    for seq, (src, n) in enumerate([(0, 41), (1, 90), (0, 41)]):
        keys, vals = (torch.cat([raw[i][src], new[i][seq:seq + 1]]).double().view(-1, heads, 128)
                      for i in range(2))
        qq = q[seq].double().view(heads, group, 128)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", qq, keys) * 128 ** -0.5, -1)
        ideal = torch.einsum("hgn,nhd->hgd", p, vals).reshape(heads * group, 128)
        assert (out[seq].double() - ideal).norm() < 0.5 * ideal.norm()
    # the untouched layer stayed as it was
    assert not caches[0].codes[0].any() and not caches[1].scales[0].any()
    # output projection: attention result -> rotation -> 4-bit weights
    k, n = heads * group * 128, 300
    s2 = torch.from_numpy((rng.integers(0, 2, k) * 2 - 1).astype(np.int8)).cuda()
    rot = torch.empty((3, k), device="cuda")
    kq.kq_rht(out.view(3, k), 0, s2, rot)
    w = _weights(rng, "int4_asym", n, k)
    y = torch.empty((3, n), device="cuda")
    _gemv("int4_asym", rot, *w, y)
    _check_gemv("int4_asym", rot.double().cpu().numpy(), w, y)


# ------------------------------------------- where the kernels change their ways
def _check_some_rows(fmt, x, w, y, rows):
    codes, scales, zeros, t = w
    part = (codes[rows], scales[rows], None if zeros is None else zeros[rows], t)
    _check_gemv(fmt, x, part, y[:, torch.from_numpy(rows).cuda()])


@pytest.mark.parametrize("fmt,n,k,m,xt,yt", [
    # more tiles than a round's sums have room for: one CTA a cluster, four of them
    ("int4_asym", 60011, 128, 16, "bf16", "f32"), ("int4_sym", 52001, 256, 8, "bf16", "bf16"),
    ("nvfp4", 12007, 2048, 16, "bf16", "bf16"), ("mxfp4", 11003, 2048, 16, "f32", "f32"),
    # x in several segments, and rounds on top of them
    ("int4_sym", 4801, 13312, 16, "f32", "f32"), ("int4_asym", 100, 32768, 16, "f32", "f32"),
    ("mxfp4", 33, 131072, 3, "bf16", "f32"), ("nvfp4", 70, 65536 + 160, 9, "bf16", "f32"),
])
def test_gemv_rounds_and_segments(fmt, n, k, m, xt, yt):
    rng = np.random.default_rng(n + k)
    w = _weights(rng, fmt, n, k)
    x = torch.from_numpy(rng.standard_normal((m, k))).cuda().to(KIND[xt])
    y = torch.full((m, n), float("nan"), dtype=KIND[yt], device="cuda")
    _gemv(fmt, x, *w, y)
    rows = np.unique(np.concatenate([np.arange(min(n, 20)), rng.integers(0, n, 200),
                                     np.arange(max(0, n - 40), n)]))
    _check_some_rows(fmt, x.double().cpu().numpy(), w, y, rows)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("fmt", ["int4_asym", "nvfp4", "mxfp4"])
def test_gemv_scales_at_other_alignments(fmt):
    """Scales that begin off the 16-byte grid, as a layer's slice of a larger tensor
    may: the result is that of aligned copies."""
    rng = np.random.default_rng(3)
    codes, scales, zeros, t = _weights(rng, fmt, 65, 1024)
    x = torch.from_numpy(rng.standard_normal((2, 1024))).cuda().bfloat16()
    want = torch.empty((2, 65), device="cuda")
    _gemv(fmt, x, codes, scales, zeros, t, want)

    def moved(a, by):
        flat = torch.zeros(a.size + by, dtype=torch.from_numpy(a).dtype, device="cuda")
        flat[by:] = _dev(a).view(-1)
        return flat[by:].view(a.shape)
    for by in (1, 2, 3) if fmt != "nvfp4" else (2, 4, 6):
        y = torch.empty((2, 65), device="cuda")
        kq.kq_gemv(FMT[fmt], x, _dev(oracle.pack_nibbles(codes)), moved(scales, by),
                   None if zeros is None else moved(zeros, by),
                   None if t is None else torch.tensor([float(t)], device="cuda"),
                   128 if zeros is not None else 0, y)
        assert torch.equal(y, want)


def test_gemv_streams_and_graph():
    rng = np.random.default_rng(4)
    w = _weights(rng, "int4_asym", 300, 1024)
    codes, s, z = _dev(oracle.pack_nibbles(w[0])), _dev(w[1]), _dev(w[2])
    xs = [torch.from_numpy(rng.standard_normal((4, 1024))).cuda().bfloat16() for _ in range(2)]
    want = [torch.empty((4, 300), device="cuda") for _ in range(2)]
    for x, y in zip(xs, want):
        kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, x, codes, s, z, None, 128, y)
    torch.cuda.synchronize()
    # two calls at once, on streams of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty((4, 300), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, y, st in zip(xs, got, streams):
            kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, x, codes, s, z, None, 128, y, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # captured, then replayed on an input changed in place
    x, y = xs[0].clone(), torch.empty((4, 300), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, x, codes, s, z, None, 128, y)
    x.copy_(xs[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[1])


def test_attention_calls_at_once():
    """Two streams, a workspace each: neither sees the other."""
    page = 16
    cases = [_case(30 + i, lens, 8, 4, page) for i, lens in enumerate([[3000], [5, 700, 40]])]
    args = []
    for q, k, v, ks, vs, table, lens in cases:
        args.append((q, _upload(k), _upload(v), _dev(ks), _dev(vs), _dev(table), page, _dev(lens), 0.1))
    want = [_attn(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    ws = [kq.empty_attn_workspace(a[0].shape[0], 32, 8) for a in args]
    out = [torch.empty_like(a[0]) for a in args]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, w, o, st in zip(args, ws, out, streams):
            _attn(*a, ws=w, out=o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_attention_joins_many_rows_and_few():
    """The three ways partial sums are joined (by the number of rows), every
    sequence split over several CTAs."""
    _whole(40, [2000, 1990], 8, 8, 16)                       # 128 rows
    _whole(41, [700 + i for i in range(24)], 8, 4, 16)       # 768 rows
    _whole(42, [400 + i for i in range(40)], 8, 5, 16)       # 1600 rows
    _whole(43, [3000, 10, 0], 1, 3, 16)


def test_cache_offsets_past_32_bits():
    """Rows whose codes begin behind 2^32 bytes: attention and page copies."""
    heads, page = 32, 16
    slots = (1 << 32) // (heads * 64) + 4 * page
    rng = np.random.default_rng(50)
    caches = [kq.empty_kv_cache(slots, heads * 128) for _ in range(2)]
    pages = slots // page
    table = np.array([[pages - 1, 3, pages - 2]], dtype=np.int32)
    small = []
    for c in caches:
        codes, scales, zeros = _cache(rng, 3 * page, heads)
        for i, p in enumerate(table[0]):
            at, here = slice(int(p) * page, int(p) * page + page), slice(i * page, i * page + page)
            c.codes[at] = _dev(oracle.pack_nibbles(codes[here]))
            c.scales[at], c.zeros[at] = _dev(scales[here]), _dev(zeros[here])
        small.append((codes, scales, zeros))
    q = torch.from_numpy(rng.standard_normal((1, heads, 128))).cuda().bfloat16()
    lens = np.array([45], dtype=np.int32)
    out = _attn(q, *caches, None, None, _dev(table), page, _dev(lens), 0.1)
    _check_attn(out, q.double().cpu().numpy(), *small, None, None,
                np.array([[0, 1, 2]]), page, lens, 0.1, 0, 0)
    kq.kq_kv_copy_pages(_dev(np.array([[pages - 1, pages - 4], [3, pages - 3]], dtype=np.int32)),
                        page, *caches)
    for c in caches:
        for a in (c.codes, c.scales, c.zeros):
            a = a.view(torch.uint8).view(slots, -1)
            for s, d in ((pages - 1, pages - 4), (3, pages - 3)):
                assert torch.equal(a[s * page:(s + 1) * page], a[d * page:(d + 1) * page])


@pytest.mark.parametrize("batch", [2, 20, 40])
def test_attention_nan_query_stays_in_its_head(batch):
    """A NaN in one head's query reaches all of that head's result and nothing
    else, whichever way the partial sums are joined (by the number of rows)."""
    q, k, v, ks, vs, table, lens = _case(33, [9, 700] + [650] * (batch - 2), 8, 4, 16)
    bad = q.clone()
    for b, h in ((0, 3), (1, 5), (batch - 1, 31)):
        q[b, h, 7] = 0
        bad[b, h, 7] = float("nan")
    clean = _run_case(q, k, v, ks, vs, table, lens, 16, 128 ** -0.5)
    out = _run_case(bad, k, v, ks, vs, table, lens, 16, 128 ** -0.5)
    for b, h in ((0, 3), (1, 5), (batch - 1, 31)):
        assert out[b, h].isnan().all()
        out[b, h] = clean[b, h]
    _check_attn(out, q.double().cpu().numpy(), k, v, ks, vs, table, 16, lens, 128 ** -0.5, 0, 0)


def test_binding_refuses_sizes_past_32_bits_and_missing_tensors():
    """Sizes that the C entries' 32 bits would cut are refused, not cut; so are
    tensors that a format needs and does not get, and other ranks."""
    q, k, v, ks, vs, table, lens = _case(1, [20, 3], 2, 2, 16)
    kc, vc, t, n = _upload(k), _upload(v), _dev(table), _dev(lens)
    ok = dict(q=q, k_cache=kc, v_cache=vc, k_signs=None, v_signs=None, block_table=t, page_size=16,
              seq_lens=n, softmax_scale=0.1, out=torch.empty_like(q),
              workspace=kq.empty_attn_workspace(2, 4, 2))
    for change in (dict(page_size=2 ** 32 + 16), dict(window=2 ** 32 + 5), dict(sinks=2 ** 32),
                   dict(window=2 ** 31), dict(window=-2 ** 32 + 5), dict(block_table=t[0]),
                   dict(q=q[0]), dict(seq_lens=None), dict(workspace=ok["workspace"].cpu())):
        with pytest.raises(ValueError):
            kq.kq_attn_decode_int4_kv(**{**ok, **change})
    kq.kq_attn_decode_int4_kv(**{**ok, "window": 2 ** 31 - 1, "sinks": 2 ** 31 - 1})
    pairs = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for args in ((pairs, 2 ** 32 + 16, kc), (pairs[0], 16, kc)):
        with pytest.raises(ValueError):
            kq.kq_kv_copy_pages(*args)
    with pytest.raises(AttributeError):
        kc.codes = vc.codes[:4]
    rng = np.random.default_rng(0)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(2, 8, device="cuda")
    for fmt in sorted(FMT):
        codes, s, z, _ = _weights(rng, fmt, 8, 256)
        codes, s = _dev(oracle.pack_nibbles(codes)), _dev(s)
        with pytest.raises(ValueError):
            kq.kq_gemv(FMT[fmt], x, codes, None, None, None, 128, y)
        if fmt in ("int4_asym", "nvfp4"):
            with pytest.raises(ValueError):
                kq.kq_gemv(FMT[fmt], x, codes, s, None, None, 128, y)
        else:
            with pytest.raises(ValueError):
                kq.kq_gemv(FMT[fmt], x, codes, s, None, None, 2 ** 32 + 128, y)
    wide = 2 ** 32 + 128
    with pytest.raises(ValueError):
        kq.kq_gemv(kq.KQ_FMT_MXFP4, x.new_empty(0, wide),
                   torch.empty(0, wide // 2, dtype=torch.uint8, device="cuda"),
                   torch.empty(0, wide // 32, dtype=torch.uint8, device="cuda"), None, None, 128,
                   y.new_empty(0, 0))


# Short tables take the units of a batch one by one; the sizes above once more behind
# tables wide enough (more than 512 tokens) that the same lengths are dealt and joined.
def _dealt(page):
    return dict(extra_width=512 // page + 1)


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 8), (2, 3), (3, 2), (4, 4), (5, 5), (6, 1),
                                         (8, 1), (8, 4), (8, 8), (12, 2), (16, 2), (2, 16), (1, 20),
                                         (32, 1)])
def test_attention_head_layouts_dealt(heads, group):
    _whole(heads * 100 + group, [1, 33, 150, 0, 17], heads, group, 16, **_dealt(16))


@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 32, 50, 64, 128])
def test_attention_pages_dealt(page):
    _whole(page, [200, 1, 31, 32, 33, 129, 63, 64, 65], 8, 2, page, **_dealt(page))


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [32], [33], [127], [128],
                                  [129], [255], [256], [257], [0], [0, 0, 3]])
def test_attention_lengths_dealt(lens):
    _whole(sum(lens), lens, 2, 4, 16, **_dealt(16))
    _whole(sum(lens) + 1, lens, 8, 4, 16, **_dealt(16))


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (64, 0), (100, 1), (256, 256), (256, 257),
                                          (512, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("heads,group", [(8, 4), (2, 9)])
def test_attention_windows_on_long_tables(heads, group, window, sinks):
    """A window of few tokens on a long table is short too; on either side of 512."""
    _whole(window + sinks, [1, 5, 40, 600, 2000, 0, 333, 513], heads, group, 16, window, sinks)


@pytest.mark.parametrize("batch", [18, 19, 36, 37, 38, 74, 75])
def test_attention_short_units_around_the_ctas(batch):
    """Numbers of (sequence, head) units around one and two CTAs a multiprocessor."""
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(0, 513, batch)]
    for heads, group in ((8, 2), (4, 9)):
        _whole(batch, lens, heads, group, 32, **(dict(extra_width=16 - max(-(-n // 32) for n in lens))))


# ----------------------------------- calls right behind what makes their inputs
def test_decode_calls_right_behind_their_inputs():
    """The kernels may be brought in while the one in front of them ends: inputs
    written by it (kernels, copies and sets, on the same or another stream, in
    captured graphs too) are the ones that are read, and what comes behind a call
    sees its result."""
    rng = np.random.default_rng(8)
    heads, group, page = 8, 4, 16
    q, k, v, ks, vs, table, lens = _case(41, [900, 70, 1300, 5], heads, group, page)
    kc, vc, ksd, vsd = _upload(k), _upload(v), _dev(ks), _dev(vs)
    w = _weights(rng, "int4_asym", 500, 2048)
    codes, sc, z = _dev(oracle.pack_nibbles(w[0])), _dev(w[1]), _dev(w[2])
    # two sets of inputs, and results of calls that had all the time they want
    qs = [q, q.flip(0).contiguous()]
    ls = [_dev(lens), _dev(lens // 2)]
    xs = [torch.from_numpy(rng.standard_normal((3, 2048))).cuda().bfloat16() for _ in range(2)]
    tab, ws = _dev(table), kq.empty_attn_workspace(4, heads * group, heads)
    want = []
    for i in range(2):
        y = torch.empty(3, 500, device="cuda")
        kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, xs[i], codes, sc, z, None, 128, y)
        torch.cuda.synchronize()
        want.append((_attn(qs[i], kc, vc, ksd, vsd, tab, page, ls[i], 0.1), y))
        torch.cuda.synchronize()
    which = torch.zeros((), dtype=torch.int64, device="cuda")
    qb, lb, xb = torch.empty_like(q), torch.empty_like(ls[0]), torch.empty_like(xs[0])
    out, yb = torch.empty_like(q), torch.empty(3, 500, device="cuda")
    res, yres = torch.empty_like(out), torch.empty_like(yb)
    allq, alll, allx = torch.stack(qs), torch.stack(ls), torch.stack(xs)
    busy = torch.zeros(1 << 24, device="cuda")
    other = torch.cuda.Stream()
    pinned = [n.cpu().pin_memory() for n in ls]

    def kernels(i):
        busy.add_(1.0)                       # keeps the multiprocessors while the call is issued
        torch.index_select(allq, 0, which.view(1), out=qb.unsqueeze(0))
        torch.index_select(alll, 0, which.view(1), out=lb.unsqueeze(0))

    def copies(i):
        qb.copy_(qs[i])
        lb.copy_(pinned[i], non_blocking=True)

    def across(i):
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        with torch.cuda.stream(other):
            kernels(i)
        busy.mul_(0.5)
        main.wait_stream(other)

    def step(i, before):
        before(i)
        kq.kq_attn_decode_int4_kv(qb, kc, vc, ksd, vsd, tab, page, lb, 0.1, out, ws)
        res.copy_(out)
        torch.index_select(allx, 0, which.view(1), out=xb.unsqueeze(0))
        yb.zero_()
        kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, xb, codes, sc, z, None, 128, yb)
        yres.copy_(yb)

    def check(i):
        torch.cuda.synchronize()
        assert torch.equal(res, want[i][0]) and torch.equal(yres, want[i][1])
    for before in (kernels, copies, across):
        for turn in range(12):
            which.fill_(turn & 1)
            for a in (qb, out, res):
                a.fill_(float("nan"))
            step(turn & 1, before)
            check(turn & 1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs = []
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(i, before)
            graphs.append(g)
        for turn in range(12):
            which.fill_(turn & 1)
            for a in (qb, out, res, yb, yres):
                a.fill_(float("nan"))
            graphs[turn & 1].replay()
            check(turn & 1)


def test_decode_calls_in_a_chain():
    """Page copies, attention and products one behind the other with nothing in
    between, each reading what the one in front wrote, against the same calls with a
    synchronization behind each."""
    heads, group, page = 8, 2, 16
    q, k, v, ks, vs, table, lens = _case(43, [333, 48, 700], heads, group, page, spare=12)
    rng = np.random.default_rng(9)
    n = heads * group * 128
    w = [_weights(rng, f, n, n) for f in ("int4_asym", "mxfp4")]
    w = [(_dev(oracle.pack_nibbles(c)), _dev(s * 0.02 if i == 0 else s),
          None if zz is None else _dev(zz)) for i, (c, s, zz, _) in enumerate(w)]
    pages = k[0].shape[0] // page
    spare = [p for p in range(pages) if p not in set(table.ravel().tolist())]
    pairs = _dev(np.array([[table[0, 0], spare[0]], [table[1, 1], spare[1]]], dtype=np.int32))
    table2 = table.copy()
    table2[0, 0], table2[1, 1] = spare[0], spare[1]
    tab, ln, ws = _dev(table2), _dev(lens), kq.empty_attn_workspace(3, heads * group, heads)

    def run(wait):
        def then():
            if wait:
                torch.cuda.synchronize()
        kc, vc = _upload(k), _upload(v)
        torch.cuda.synchronize()
        x, results = q.clone(), []
        for turn in range(4):
            kq.kq_kv_copy_pages(pairs, page, kc, vc)
            then()
            out = torch.empty_like(q)
            kq.kq_attn_decode_int4_kv(x, kc, vc, None, None, tab, page, ln, 0.02, out, ws)
            then()
            y = torch.empty(3, n, dtype=torch.bfloat16, device="cuda")
            kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, out.view(3, n), *w[0], None, 128, y)
            then()
            y2 = torch.empty(3, n, dtype=torch.bfloat16, device="cuda")
            kq.kq_gemv(kq.KQ_FMT_MXFP4, y, w[1][0], w[1][1], None, None, 128, y2)
            then()
            x = (y2 / 64).clamp(-4, 4).view_as(q)
            results += [out, y, y2]
        torch.cuda.synchronize()
        return results
    for _ in range(5):
        for a, b in zip(run(True), run(False)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("fmt", sorted(FMT))
@pytest.mark.parametrize("n,k,m,xt", [
    # one rank; two with steps of 2 and 1, 3 and 2; four with a short last step; none whole
    (4800, 1536, 1, "bf16"), (500, 1536, 8, "bf16"), (500, 2560, 4, "f32"), (90, 2176, 8, "bf16"),
    (90, 2688, 8, "bf16"), (70, 5504, 7, "f32"), (70, 640, 16, "f32"), (40000, 1536, 8, "bf16"),
    (33000, 2048, 16, "bf16"), (33000, 896, 16, "f32"), (50, 12800, 16, "bf16")])
def test_gemv_splits_of_k(fmt, n, k, m, xt):
    """Numbers of 128-wide groups that the ranks of a cluster and the steps of a
    warp do and do not divide, with few rows and with many."""
    rng = np.random.default_rng(n + k + m)
    w = _weights(rng, fmt, n, k)
    x = torch.from_numpy(rng.standard_normal((m, k))).cuda().to(KIND[xt])
    y = torch.empty((m, n), device="cuda")
    _gemv(fmt, x, *w, y)
    rows = np.unique(np.concatenate([np.arange(min(n, 40)), rng.integers(0, n, 60), [n - 1]]))
    _check_some_rows(fmt, x.double().cpu().numpy(), w, y, rows)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["int4_asym", "mxfp4"])
def test_gemv_every_number_of_tokens(fmt, xt):
    """Sums travel between the CTAs of a cluster four, two or one at a time by
    the number of tokens; 1536: two ranks, 4096: four, 128: one."""
    rng = np.random.default_rng(3)
    for k in (128, 1536, 4096):
        w = _weights(rng, fmt, 333, k)
        for m in range(1, 17):
            x = torch.from_numpy(rng.standard_normal((m, k))).cuda().to(KIND[xt])
            buf = torch.full((m * 333 + 64,), 7.0, device="cuda")
            y = buf[32:32 + m * 333].view(m, 333)
            _gemv(fmt, x, *w, y)
            _check_gemv(fmt, x.double().cpu().numpy(), w, y)
            assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()
