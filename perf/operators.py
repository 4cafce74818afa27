"""Serving operators over rotated 4-bit tensors, as they are measured.

Three operators that stand between the quantizers and the tokens of a decode
step:
  * gemv  -- y = x W^T with the weights W in one of the library's 4-bit
             formats and a few tokens x;
  * attn  -- attention of one new token per sequence over the paged INT4
             key-value cache that kq_rht_quant_int4_kv writes, with an optional
             sliding window and first tokens that stay visible;
  * copy  -- pages of that cache copied to other pages (a forked sequence's
             last page, a compacted pool).

`run` computes each either in its plain form (elementary torch operations in
32 bits) or, with `own` set, through the library's entry points; `exact`
computes it once more from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD = 128                      # head width = Hadamard block = quantization group
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the query projection of a 4096-wide layer
        dict(name="gemv_asym_4096x4096_m1", op="gemv", fmt="int4_asym", n=4096, k=4096, m=1,
             x="bf16", y="bf16"),
        # eight sequences through the up projection (4096 -> 12288)
        dict(name="gemv_asym_12288x4096_m8", op="gemv", fmt="int4_asym", n=12288, k=4096, m=8,
             x="bf16", y="bf16"),
        # the down projection on the fp32 rows the 12288-wide rotation returns
        dict(name="gemv_nvfp4_4096x12288_m2", op="gemv", fmt="nvfp4", n=4096, k=12288, m=2,
             x="f32", y="f32"),
        # a vocabulary-sized head with an odd number of rows
        dict(name="gemv_mxfp4_32003x4096_m4", op="gemv", fmt="mxfp4", n=32003, k=4096, m=4,
             x="bf16", y="f32"),
        # a full decode batch on per-row scales
        dict(name="gemv_sym_4096x4096_m16", op="gemv", fmt="int4_sym", n=4096, k=4096, m=16,
             x="f32", y="f32"),
        # a few sequences just begun, one of them still empty
        dict(name="attn_short", op="attn", batch=4, min_len=1, max_len=200, kv_heads=8, group=4,
             page=16, window=0, sinks=0, empty=True),
        # a serving batch of ragged lengths, four query heads to a cached one
        dict(name="attn_batch32", op="attn", batch=32, min_len=300, max_len=4096, kv_heads=8,
             group=4, page=16, window=0, sinks=0, empty=False),
        # one long document
        dict(name="attn_long_131072", op="attn", batch=1, min_len=131071, max_len=131071,
             kv_heads=8, group=8, page=64, window=0, sinks=0, empty=False),
        # 32 heads of their own, the head layout of a 4096-wide cache row
        dict(name="attn_mha32", op="attn", batch=5, min_len=1000, max_len=8192, kv_heads=32,
             group=1, page=32, window=0, sinks=0, empty=False),
        # long streams behind a window, four first tokens kept
        dict(name="attn_window", op="attn", batch=64, min_len=500, max_len=32768, kv_heads=8,
             group=4, page=16, window=1024, sinks=4, empty=False),
        # a forked sequence's last pages, over the layers of one cache
        dict(name="copy_fork", op="copy", pages=3, total=512, layers=4, page=16, kv_heads=8),
        # a pool compacted: many pages, and the rows that pad the list
        dict(name="copy_compact", op="copy", pages=1500, total=4096, layers=4, page=16,
             kv_heads=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "attn", "attn", "copy"])
    if op == "gemv":
        while True:
            n, k = _log(rng, 64, 32768), 128 * _log(rng, 1, 96)
            if n * k <= 32003 * 4096:
                break
        return dict(op=op, fmt=rng.choice(["int4_asym", "int4_sym", "nvfp4", "mxfp4"]), n=n, k=k,
                    m=_log(rng, 1, 16), x=rng.choice(["bf16", "f32"]),
                    y=rng.choice(["bf16", "f32"]))
    if op == "attn":
        while True:
            batch, most = _log(rng, 1, 64), _log(rng, 1, 131072)
            kv, group = rng.choice([1, 2, 3, 4, 5, 8, 16, 32]), rng.choice([1, 2, 3, 4, 5, 8, 16])
            if batch * most * kv * max(8, group) <= 131071 * 8 * 8:
                break
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        return dict(op=op, batch=batch, min_len=_log(rng, 1, most), max_len=most, kv_heads=kv,
                    group=group, page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                    window=window, sinks=rng.choice([0, 1, 4, 17]) if window else 0,
                    empty=rng.random() < 0.3)
    pages = _log(rng, 1, 1500)
    return dict(op=op, pages=pages, total=2 * pages + rng.randint(2, 1000),
                layers=rng.randint(1, 4), page=rng.choice([1, 8, 16, 24]),
                kv_heads=rng.choice([1, 2, 3, 5, 8]))


def _lengths(case):
    """The sequences' lengths, spread evenly over the logarithm (in some order)."""
    b, lo, hi = case["batch"], case["min_len"], case["max_len"]
    lens = [int(round(lo * (hi / lo) ** (i / max(1, b - 1)))) for i in range(b)]
    lens[-1] = hi
    if case["empty"] and b > 1:
        lens[0] = 0
    return lens


def _visible(case, length):
    return min(length, case["window"] + case["sinks"]) if case["window"] else length


def _scale_bytes(fmt, n, k):
    return {"int4_asym": 4 * n * (k // HEAD), "int4_sym": 4 * n, "nvfp4": n * (k // 16) + 4,
            "mxfp4": n * (k // 32)}[fmt]


def work(case):
    if case["op"] == "gemv":
        n, k, m = case["n"], case["k"], case["m"]
        size = {"bf16": 2, "f32": 4}
        return {"bytes": n * k // 2 + _scale_bytes(case["fmt"], n, k) + m * k * size[case["x"]] +
                m * n * size[case["y"]], "flops": 2 * n * k * m}
    if case["op"] == "attn":
        lens = _lengths(case)
        vis = sum(_visible(case, v) for v in lens)
        heads = case["kv_heads"] * case["group"]
        row = case["kv_heads"] * (HEAD // 2 + 4)          # codes, scale and zero point
        return {"bytes": 2 * vis * row + 2 * 2 * case["batch"] * heads * HEAD,
                "flops": 4 * vis * heads * HEAD}
    row = case["kv_heads"] * (HEAD // 2 + 4)
    return {"bytes": 2 * 2 * case["pages"] * case["layers"] * case["page"] * row, "flops": 0}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _hadamard(dtype=torch.float32):
    """Sylvester's matrix of 128 rows, natural order, normalized."""
    i = torch.arange(HEAD, device="cuda")
    both = i[:, None] & i[None, :]
    odd = torch.zeros_like(both)
    for bit in range(7):
        odd = odd ^ (both >> bit & 1)
    return (1 - 2 * odd).to(dtype) / math.sqrt(HEAD)


def _pack(codes):
    c = codes.to(torch.uint8)
    return (c[..., 0::2] | c[..., 1::2] << 4).contiguous()


def _quant_asym(y):
    """[..., groups, 128] -> codes, fp16 scale and zero point."""
    hi, lo = y.amax(-1), y.amin(-1)
    s = ((hi - lo) / 15).half()
    z = torch.where(s > 0, torch.round(-lo / s.float()), 0.0).half()
    u = (torch.round(y / s.float()[..., None]) + z.float()[..., None]).clamp(0, 15)
    return torch.where(s[..., None] > 0, u, 0.0), s, z


def _quant_e2m1(v):
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return torch.bucketize(v.abs(), edges) + 8 * (v < 0)


def _weights(fmt, n, k, g):
    """A weight matrix [n, k] in the format: codes, scales, zeros, tensor scale."""
    w = torch.randn(n, k, generator=g, device="cuda")
    w *= 0.02 * torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
    if fmt == "int4_asym":
        u, s, z = _quant_asym(w.view(n, k // HEAD, HEAD))
        return _pack(u.view(n, k)), s, z, None
    if fmt == "int4_sym":
        s = w.abs().amax(1) / 7
        q = torch.round(w / s[:, None]).clamp(-8, 7).to(torch.int32) & 15
        return _pack(q), s, None, None
    if fmt == "nvfp4":
        t = (w.abs().amax() / 2688).reshape(1)
        s = (w.view(n, k // 16, 16).abs().amax(-1) / (6 * t)).clamp(max=448).to(torch.float8_e4m3fn)
        d = (s.float() * t)[..., None]
        v = torch.where(d > 0, w.view(n, k // 16, 16) / d, 0.0)
        return _pack(_quant_e2m1(v).view(n, k)), s.view(torch.uint8), None, t
    e = (torch.floor(torch.log2(w.view(n, k // 32, 32).abs().amax(-1))) - 2).clamp(-127, 127)
    v = w.view(n, k // 32, 32) / torch.exp2(e)[..., None]
    return _pack(_quant_e2m1(v).view(n, k)), (e + 127).to(torch.uint8), None, None


def _cache(rows, heads, h, signs, g):
    """A cache of `rows` rows: activations with heads of different size and two
    outlier channels a head, rotated and quantized head by head."""
    size = torch.exp(torch.randn(heads, 1, generator=g, device="cuda") * 0.5)
    size = size.expand(heads, HEAD).clone()
    size[:, [5, 77]] *= 8
    codes = torch.empty(rows, heads * HEAD // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, heads, dtype=torch.float16, device="cuda")
    zeros = torch.empty(rows, heads, dtype=torch.float16, device="cuda")
    step = max(1, (1 << 26) // (heads * HEAD))
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = torch.randn(b - a, heads, HEAD, generator=g, device="cuda") * size
        u, s, z = _quant_asym((x.bfloat16().float() * signs.view(heads, HEAD)) @ h)
        codes[a:b], scales[a:b], zeros[a:b] = _pack(u.view(b - a, heads * HEAD)), s, z
    return codes, scales, zeros


def _signs(n, g):
    return (torch.randint(0, 2, (n,), generator=g, device="cuda") * 2 - 1).to(torch.int8)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "gemv":
        n, k, m = case["n"], case["k"], case["m"]
        codes, scales, zeros, t = _weights(case["fmt"], n, k, g)
        x = torch.randn(m, k, generator=g, device="cuda")
        x[:, torch.randint(0, k, (max(1, k // 512),), generator=g, device="cuda")] *= 20
        kind = {"bf16": torch.bfloat16, "f32": torch.float32}
        return dict(case=case, x=x.to(kind[case["x"]]), codes=codes, scales=scales, zeros=zeros,
                    tensor_scale=t, y=torch.empty(m, n, dtype=kind[case["y"]], device="cuda"))
    if case["op"] == "attn":
        rng = random.Random(seed)
        lens = _lengths(case)
        rng.shuffle(lens)
        batch, page, heads = case["batch"], case["page"], case["kv_heads"]
        width = -(-case["max_len"] // page)
        used = [-(-v // page) for v in lens]
        pool = sum(used) + 7
        ids = list(range(pool))
        rng.shuffle(ids)
        table = np.full((batch, width), -1, dtype=np.int32)
        for b, v in enumerate(lens):
            for p in range(used[b]):
                at = ids.pop()
                # pages that the window has left behind were given back to the pool
                if _visible(case, v) < v and p * page >= case["sinks"] and \
                        (p + 1) * page <= v - case["window"]:
                    continue
                table[b, p] = at
        h, dim = _hadamard(), heads * HEAD
        k_signs, v_signs = _signs(dim, g), _signs(dim, g)
        rows = pool * page
        q = torch.randn(batch, heads * case["group"], HEAD, generator=g, device="cuda") * 1.5
        return dict(case=case, q=q.bfloat16(), k_signs=k_signs, v_signs=v_signs,
                    k=_cache(rows, heads, h, k_signs, g), v=_cache(rows, heads, h, v_signs, g),
                    table=torch.from_numpy(table).cuda(),
                    lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                    most=max(_visible(case, v) for v in lens), hadamard=h,
                    out=torch.empty_like(q, dtype=torch.bfloat16))
    rng = random.Random(seed)
    layers, rows, heads = case["layers"], case["total"] * case["page"], case["kv_heads"]
    pages = list(range(1, case["total"]))                # page 0 belongs to nobody
    rng.shuffle(pages)
    n = case["pages"]
    pairs = [(pages[i], pages[n + i]) for i in range(n)] + [(-1, -1)] * (n // 8)
    rng.shuffle(pairs)

    def some(shape, kind):
        top = 256 if kind == torch.uint8 else 15000
        return torch.randint(0, top, shape, generator=g, device="cuda", dtype=torch.int16) \
            .to(torch.uint8) if kind == torch.uint8 else \
            torch.randint(1, top, shape, generator=g, device="cuda", dtype=torch.int16)
    kv = [[some((layers, rows, heads * HEAD // 2), torch.uint8),
           some((layers, rows, heads), torch.int16), some((layers, rows, heads), torch.int16)]
          for _ in range(2)]
    return dict(case=case, k=kv[0], v=kv[1],
                pairs=torch.tensor(pairs, dtype=torch.int32, device="cuda").reshape(-1, 2))


# -------------------------------------------------------------- plain form
def _nibbles(packed):
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def _plain_weights(s):
    fmt, n, k = s["case"]["fmt"], s["case"]["n"], s["case"]["k"]
    c = _nibbles(s["codes"])
    if fmt == "int4_asym":
        w = (c.float().view(n, k // HEAD, HEAD) - s["zeros"].float()[..., None])
        return (w * s["scales"].float()[..., None]).view(n, k)
    if fmt == "int4_sym":
        return (c.float() - 16 * (c >= 8)) * s["scales"][:, None]
    v = torch.tensor(E2M1 + tuple(-a for a in E2M1), device="cuda")[c.int()]
    if fmt == "nvfp4":
        d = s["scales"].view(torch.float8_e4m3fn).float() * s["tensor_scale"]
        return (v.view(n, k // 16, 16) * d[..., None]).view(n, k)
    return (v.view(n, k // 32, 32) * torch.exp2(s["scales"].float() - 127)[..., None]).view(n, k)


def _plain_gemv(s):
    return (s["x"].float() @ _plain_weights(s).t()).to(s["y"].dtype)


def _plain_rows(cache, slots, heads):
    """Dequantized rows [..., heads, 128] of the slots."""
    codes, scales, zeros = (t[slots] for t in cache)
    u = _nibbles(codes).view(*slots.shape, heads, HEAD).float()
    return (u - zeros.float()[..., None]) * scales.float()[..., None]


def _plain_attn(s):
    c = s["case"]
    heads, group, page = c["kv_heads"], c["group"], c["page"]
    lens = s["lens"].long()[:, None]
    seen = torch.arange(s["most"], device="cuda")[None, :]
    if c["window"]:
        left = (lens - c["window"] - c["sinks"]).clamp(min=0)
        pos = torch.where(seen < c["sinks"], seen, seen + left)
    else:
        pos = seen.expand(c["batch"], -1)
    there = pos < lens
    at = torch.where(there, pos, 0)
    pages = s["table"].long().gather(1, at // page)
    slots = torch.where(there, pages * page + at % page, 0)
    h = s["hadamard"]
    q = s["q"].float().view(c["batch"], heads, group, HEAD)
    q = (q * s["k_signs"].float().view(heads, 1, HEAD)) @ h
    score = torch.einsum("bhgd,bnhd->bhgn", q, _plain_rows(s["k"], slots, heads))
    score = (score / math.sqrt(HEAD)).masked_fill(~there[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgn,bnhd->bhgd", p, _plain_rows(s["v"], slots, heads))
    o = torch.where(total > 0, o / total, 0.0)
    o = (o @ h) * s["v_signs"].float().view(heads, 1, HEAD)
    return o.view(c["batch"], heads * group, HEAD).bfloat16()


def _plain_copy(s):
    c = s["case"]
    pairs = s["pairs"].long()
    src, dst = torch.where(pairs >= 0, pairs, 0).unbind(1)
    kv = s["k"] + s["v"]
    pages = [t.view(c["layers"], c["total"], -1) for t in kv]
    for t in pages:
        t[:, dst] = t[:, src]
    return kv


# ----------------------------------------------------- the library's calls
def _own_gemv(kq, s):
    fmt = {"int4_sym": kq.KQ_FMT_INT4_SYM, "int4_asym": kq.KQ_FMT_INT4_ASYM,
           "nvfp4": kq.KQ_FMT_NVFP4, "mxfp4": kq.KQ_FMT_MXFP4}[s["case"]["fmt"]]
    kq.kq_gemv(fmt, s["x"], s["codes"], s["scales"], s["zeros"], s["tensor_scale"],
               HEAD if s["zeros"] is not None else 0, s["y"])
    return s["y"]


def _own_attn(kq, s):
    c = s["case"]
    if "cache" not in s:
        s["cache"] = kq.KVCacheInt4(*s["k"]), kq.KVCacheInt4(*s["v"])
        s["workspace"] = kq.empty_attn_workspace(c["batch"], c["kv_heads"] * c["group"],
                                                 c["kv_heads"])
    k, v = s["cache"]
    kq.kq_attn_decode_int4_kv(s["q"], k, v, s["k_signs"], s["v_signs"], s["table"], c["page"],
                              s["lens"], 1 / math.sqrt(HEAD), s["out"], s["workspace"],
                              window=c["window"], sinks=c["sinks"])
    return s["out"]


def _own_copy(kq, s):
    if "cache" not in s:
        s["cache"] = [kq.KVCacheInt4(t[0], t[1].view(torch.float16), t[2].view(torch.float16))
                      for t in (s["k"], s["v"])]
    kq.kq_kv_copy_pages(s["pairs"], s["case"]["page"], *s["cache"])
    return s["k"] + s["v"]


def run(state):
    op = state["case"]["op"]
    if own:
        import hadamard_rotated_activation_b200 as kq
        return {"gemv": _own_gemv, "attn": _own_attn, "copy": _own_copy}[op](kq, state)
    return {"gemv": _plain_gemv, "attn": _plain_attn, "copy": _plain_copy}[op](state)


# --------------------------------------------------------------- 64 bits
def _exact_gemv(s):
    case = s["case"]
    n, k, fmt = case["n"], case["k"], case["fmt"]
    y = torch.zeros(case["m"], n, dtype=torch.float64, device="cuda")
    table = [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]
    if fmt == "int4_asym":
        table = list(range(16))
    elif fmt == "int4_sym":
        table = [(i + 8) % 16 - 8 for i in range(16)]
    table = torch.tensor(table, dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for a in range(0, n, 2048):
        b = min(n, a + 2048)
        packed = s["codes"][a:b].int()
        w = torch.empty(b - a, k, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = table[packed % 16], table[packed // 16]
        if fmt == "int4_sym":
            w *= s["scales"][a:b, None].double()
        elif fmt == "int4_asym":
            w -= s["zeros"][a:b].double().repeat_interleave(HEAD, 1)
            w *= s["scales"][a:b].double().repeat_interleave(HEAD, 1)
        elif fmt == "nvfp4":
            byte = s["scales"][a:b].int()
            e, f = byte // 8, (byte % 8).double()
            d = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f / 512)
            w *= d.repeat_interleave(16, 1) * s["tensor_scale"].double()
        else:
            w *= torch.exp2(s["scales"][a:b].double() - 127).repeat_interleave(32, 1)
        y[:, a:b] = x @ w.T
    return y


def _exact_attn(s):
    case = s["case"]
    heads, group, page = case["kv_heads"], case["group"], case["page"]
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    for _ in range(7):
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    out = torch.zeros(case["batch"], heads, group, HEAD, dtype=torch.float64, device="cuda")
    root = math.sqrt(HEAD)
    for b, length in enumerate(s["lens"].tolist()):
        keep = [p for p in range(length) if not case["window"] or p < case["sinks"] or
                p >= length - case["window"]]
        if not keep:
            continue
        pos = torch.tensor(keep, device="cuda")
        row = s["table"][b].long()[pos // page] * page + pos % page
        for head in range(heads):
            at = slice(head * HEAD, (head + 1) * HEAD)
            kv = []
            for codes, scales, zeros in (s["k"], s["v"]):
                packed = codes[row, head * HEAD // 2:(head + 1) * HEAD // 2].int()
                u = torch.empty(len(keep), HEAD, dtype=torch.float64, device="cuda")
                u[:, 0::2], u[:, 1::2] = (packed % 16).double(), (packed // 16).double()
                u -= zeros[row, head].double()[:, None]
                # the values as the model has them: the rotation undone
                kv.append(u * scales[row, head].double()[:, None] @ h / root)
            keys = kv[0] * s["k_signs"][at].double()
            values = kv[1] * s["v_signs"][at].double()
            q = s["q"][b, head * group:(head + 1) * group].double()
            out[b, head] = torch.softmax(q @ keys.T / root, 1) @ values
    return out.view(case["batch"], heads * group, HEAD)


def exact(case, seed):
    if case["op"] == "copy":
        return None
    s = prepare(case, seed)
    return _exact_gemv(s) if case["op"] == "gemv" else _exact_attn(s)
