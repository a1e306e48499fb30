"""What is measured of the int8 linear and the int4 cache operators.

Four operators of one decoder layer that runs on rotated activations:

  norm    hadq_rmsnorm_quant   residual addition, root-mean-square norm, int8 codes with a scale per token
  matmul  hadq_matmul_int8     int8 codes x int8 weights, scales per token and per output channel
  append  hadq_kv4_append      K rotated per head, K and V to int4 in the pages of a cache
  attend  hadq_kv4_attention   the newest tokens' attention over those pages

With ``own`` false, ``run`` computes them from elementary torch operations; with ``own`` true it makes the library's
calls.  Codes are whole numbers (int4 codes in the bytes of the cache, as stored), so both sides agree on each of them.
"""

import math

import torch

own = False

DEV = "cuda"
NAMES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's norm: one token of hidden size 4096, where only latency counts
        dict(name="norm 1x4096", op="norm", rows=1, n=4096, dtype="bf16", residual=True),
        # a prefill batch's norm on the residual stream
        dict(name="norm 16384x8192", op="norm", rows=16384, n=8192, dtype="bf16", residual=True),
        # fp32 rows without a residual, odd count, a width that is no power of 2
        dict(name="norm 777x1000 f32", op="norm", rows=777, n=1000, dtype="f32", residual=False),
        # a decode step's down projection, one token
        dict(name="matmul 1x4096x14336", op="matmul", m=1, n=4096, k=14336, out="bf16", bias=False),
        # decode with a batch of sequences
        dict(name="matmul 48x14336x4096", op="matmul", m=48, n=14336, k=4096, out="bf16", bias=False),
        # ragged in every size, with a bias, fp32 out
        dict(name="matmul 333x1001x4112 f32", op="matmul", m=333, n=1001, k=4112, out="f32", bias=True),
        # a prefill batch's down projection
        dict(name="matmul 8192x4096x14336", op="matmul", m=8192, n=4096, k=14336, out="bf16", bias=False),
        # a decode step's cache write: one token for each of 16 sequences
        dict(name="append 16x8x128", op="append", tokens=16, kv_heads=8, d=128, group=128, page=64, rotate=True),
        # a prefill batch's cache write
        dict(name="append 32768x8x128", op="append", tokens=32768, kv_heads=8, d=128, group=128, page=64, rotate=True),
        # one sequence's decode step over a long context
        dict(name="attend 1x32k", op="attend", batch=1, q_len=1, kv_heads=8, ratio=4, d=128, group=128, page=64,
             context=32768, rotate=True),
        # every head with its own K and V: batch 16, 32 heads, 4096 positions
        dict(name="attend 16x32 heads x4k", op="attend", batch=16, q_len=1, kv_heads=32, ratio=1, d=128, group=128,
             page=64, context=4096, rotate=True),
        # four drafted tokens a sequence, grouped heads, finer scales, lengths from zero to the whole context
        dict(name="attend 64x4 drafted", op="attend", batch=64, q_len=4, kv_heads=8, ratio=4, d=128, group=32, page=16,
             context=6000, rotate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "append", "attend"])
    if op == "norm":
        n = 8 * _log(rng, 8, 1792)
        rows = _log(rng, 1, min(16384, 16384 * 8192 // n))
        return dict(op=op, rows=rows, n=n, dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.7)
    if op == "matmul":
        k, n = 16 * _log(rng, 4, 1024), _log(rng, 16, 16384)
        m = _log(rng, 1, min(8192, 8192 * 4096 * 14336 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.3)
    d = rng.choice([64, 128, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    page = rng.choice([16, 32, 64, 128, 48])
    heads = rng.choice([1, 2, 4, 8, 16, 32])
    if op == "append":
        tokens = _log(rng, 1, 32768 * 8 // heads)
        return dict(op=op, tokens=tokens, kv_heads=heads, d=d, group=group, page=page, rotate=rng.random() < 0.8)
    context = _log(rng, 1, 32768)
    batch = _log(rng, 1, max(1, min(128, 16 * 32 * 4096 // (heads * context))))
    return dict(op=op, batch=batch, q_len=rng.choice([1, 1, 1, 2, 5, 8]), kv_heads=heads,
                ratio=rng.choice([1, 2, 4, 5, 8]), d=d, group=group, page=page, context=context,
                rotate=rng.random() < 0.8)


def work(case):
    c = case
    if c["op"] == "norm":
        size = 2 if c["dtype"] == "bf16" else 4
        e = c["rows"] * c["n"]
        return {"bytes": e * (size * (3 if c["residual"] else 1) + 1) + c["n"] * size + 4 * c["rows"], "flops": 6 * e}
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        out = (2 if c["out"] == "bf16" else 4) * m * n + (4 * n if c["bias"] else 0)
        return {"bytes": m * k + n * k + 4 * (m + n) + out, "flops": 2 * m * n * k}
    row = c["d"] // 2 + 2 * (c["d"] // c["group"])           # bytes of one cached row of codes and scales
    if c["op"] == "append":
        rows = 2 * c["tokens"] * c["kv_heads"]
        return {"bytes": rows * (2 * c["d"] + row) + 8 * c["tokens"], "flops": rows * c["d"] * 8}
    rows = sum(_lengths(c)) * c["kv_heads"]
    q = c["batch"] * c["q_len"] * c["kv_heads"] * c["ratio"] * c["d"]
    return {"bytes": 2 * rows * row + 4 * q, "flops": 4 * rows * c["ratio"] * c["q_len"] * c["d"]}


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """Sequence lengths of a batch: the whole context for one sequence, else spread over it, an empty one among them."""
    b, n = c["batch"], c["context"]
    if b == 1:
        return [n]
    if c["q_len"] == 1 and b <= 16:
        return [n - (i * n) // (8 * b) for i in range(b)]
    return [(n * i) // (b - 1) for i in range(b)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _codes8(g, rows, n):
    """Codes of a per-token quantizer: normal values against the largest of a row."""
    return (_randn(g, (rows, n)) * 32.0).round_().clamp_(-127, 127).to(torch.int8)


def _cache(g, pages, c):
    """One cache tensor pair: packed codes of normal values, and scales that differ from row to row."""
    shape = (pages, c["kv_heads"], c["page"])
    # 65536 byte values, two normal codes each, drawn from by index
    nib = (_randn(g, (2, 65536)) * 2.6).round_().clamp_(-7, 7).to(torch.int32) & 15
    table = (nib[0] | (nib[1] << 4)).to(torch.uint8)
    codes = table[torch.randint(65536, shape + (c["d"] // 2,), generator=g, device=DEV, dtype=torch.int32)]
    scales = (0.38 * torch.exp(0.25 * _randn(g, shape + (c["d"] // c["group"],)))).to(torch.float16)
    return codes, scales


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "norm":
        dt = NAMES[c["dtype"]]
        # a residual stream: normal entries, a few channels far larger, as rotated models have before the rotation
        spread = torch.where(torch.rand(c["n"], generator=g, device=DEV) < 0.01, 20.0, 1.0)
        s["x"] = _randn(g, (c["rows"], c["n"]), dt)
        s["residual"] = (_randn(g, (c["rows"], c["n"])) * spread).to(dt) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * _randn(g, (c["n"],))).to(dt)
        s["eps"] = 1e-6
    elif c["op"] == "matmul":
        s["a"], s["w"] = _codes8(g, c["m"], c["k"]), _codes8(g, c["n"], c["k"])
        s["a_scales"] = 0.01 + 0.05 * torch.rand(c["m"], generator=g, device=DEV)
        s["w_scales"] = (0.5 + torch.rand(c["n"], generator=g, device=DEV)) * (0.001 / math.sqrt(c["k"]))
        s["bias"] = _randn(g, (c["n"],)) if c["bias"] else None
    elif c["op"] == "append":
        # K and V are column slices of one fused projection's output, as a layer has them
        width = c["kv_heads"] * c["d"]
        qkv = _randn(g, (c["tokens"], 2 * width), torch.bfloat16)
        qkv[:, 3::c["d"]] *= 20.0                                  # an outlier dimension in each head
        s["k"] = qkv[:, :width].unflatten(1, (c["kv_heads"], c["d"]))
        s["v"] = qkv[:, width:].unflatten(1, (c["kv_heads"], c["d"]))
        pages = -(-c["tokens"] // c["page"]) + 1
        # the cache holds other sequences' rows, which stay as they are
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device=DEV)[: c["tokens"]]
        s["cache"] = _cache(g, pages, c) + _cache(g, pages, c)
    else:
        lengths = _lengths(c)
        most = -(-max(max(lengths), 1) // c["page"])
        pages = c["batch"] * most + 3
        heads = c["kv_heads"] * c["ratio"]
        s["q"] = _randn(g, (c["batch"], c["q_len"], heads, c["d"]), torch.bfloat16)
        s["cache"] = _cache(g, pages, c) + _cache(g, pages, c)
        table = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
        s["table"] = table[: c["batch"] * most].view(c["batch"], most)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(c["d"])
    return s


# --------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "matmul": _matmul, "append": _append, "attend": _attend}[state["case"]["op"]](state)


def _run_own(s):
    from hadamard_rotation_bit_b200 import hadq as H
    c = s["case"]
    if c["op"] == "norm":
        codes, scales, stream = H.hadq_rmsnorm_quant(s["x"], s["weight"], s["eps"], residual=s["residual"])
        return {"codes": codes, "scales": scales, "residual": stream}
    if c["op"] == "matmul":
        return H.hadq_matmul_int8(s["a"], s["a_scales"], s["w"], s["w_scales"], bias=s["bias"],
                                  out_dtype=NAMES[c["out"]])
    block = 0 if c["rotate"] else 1
    if c["op"] == "append":
        H.hadq_kv4_append(s["k"], s["v"], s["slots"], *s["cache"], block=block)
        return list(s["cache"])
    return H.hadq_kv4_attention(s["q"], *s["cache"], s["table"], s["lengths"], scale=s["scale"], block=block)


def _norm(s):
    x, w = s["x"], s["weight"].float()
    h = x.float()
    stream = None
    if s["residual"] is not None:
        stream = (h + s["residual"].float()).to(x.dtype)
        h = stream.float()
    t = h * w
    top = t.abs().amax(-1, keepdim=True)
    # 64 bits: a code is the nearest whole number, and near a half 32 bits would pick the wrong one
    q = torch.where(top > 0, (127.0 * t.double() / top.double()).round(), 0.0).to(torch.int8)
    scales = top[:, 0] * torch.rsqrt((h * h).mean(-1) + s["eps"]) / 127.0
    return {"codes": q, "scales": scales, "residual": stream}


def _matmul(s):
    acc = s["a"].float() @ s["w"].float().t()
    y = acc * s["a_scales"][:, None] * s["w_scales"][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(NAMES[s["case"]["out"]])


def _hadamard(z):
    """z H_d along the last axis, index bit by index bit from the lowest: sums and differences in 32 bits."""
    d, step = z.shape[-1], 1
    while step < d:
        z = z.unflatten(-1, (d // (2 * step), 2, step))
        a, b = z[..., 0, :], z[..., 1, :]
        z = torch.stack((a + b, a - b), dim=-2).flatten(-3)
        step *= 2
    return z


def _int4(x, group, rotate):
    """Packed codes and fp16 scales of rows x."""
    d = x.shape[-1]
    z, norm = x.float(), 1.0
    if rotate:
        z = _hadamard(z)
        norm = torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32).item()
    z = z.unflatten(-1, (d // group, group))
    top = z.abs().amax(-1) * norm
    scales = (top.double() / 7.0).float().clamp(max=65504.0).to(torch.float16)
    f = torch.where(scales > 0, (norm / scales.double()).float(), 0.0)
    q = (z.double() * f.double()[..., None]).round().clamp(-7, 7).to(torch.int32).flatten(-2) & 15
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), scales


def _append(s):
    c = s["case"]
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    k_codes, k_scales, v_codes, v_scales = s["cache"]
    k_codes[page, :, at], k_scales[page, :, at] = _int4(s["k"], c["group"], c["rotate"])
    v_codes[page, :, at], v_scales[page, :, at] = _int4(s["v"], c["group"], False)
    return list(s["cache"])


def _values(codes, scales, table, most):
    """Cached rows of each sequence, [batch, kv_heads, most, d], in 32 bits."""
    x = codes[table].transpose(1, 2).flatten(2, 3)[:, :, :most]
    x = torch.stack((x << 4, x & 0xF0), dim=-1).view(torch.int8).flatten(-2) >> 4     # signed nibbles, low first
    sc = scales[table].transpose(1, 2).flatten(2, 3)[:, :, :most].float()
    return (x.float().unflatten(-1, (sc.shape[-1], -1)) * sc[..., None]).flatten(-2)


def _attend(s):
    c = s["case"]
    q, table, most = s["q"].float(), s["table"].long(), max(c["context"], 1)
    if c["rotate"]:
        q = _hadamard(q) * torch.tensor(1.0 / math.sqrt(c["d"]), dtype=torch.float32).item()
    k_codes, k_scales, v_codes, v_scales = s["cache"]
    # [batch, kv_heads, rows of the group, d], rows = q_len x ratio
    q = q.unflatten(2, (c["kv_heads"], c["ratio"])).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = s["scale"] * (q @ _values(k_codes, k_scales, table, most).transpose(-1, -2))
    # the newest position that each query sees
    last = s["lengths"][:, None] - c["q_len"] + torch.arange(c["q_len"], device=DEV)
    seen = torch.arange(most, device=DEV) <= last.repeat_interleave(c["ratio"], 1)[:, None, :, None]
    top = torch.where(seen, scores, -math.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(scores - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    out = (p @ _values(v_codes, v_scales, table, most)) / torch.where(total > 0, total, 1.0)
    out = out.unflatten(2, (c["q_len"], c["ratio"])).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return out.to(torch.bfloat16)


# ------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        h, stream = s["x"].double(), None
        if s["residual"] is not None:
            stream = h + s["residual"].double()
            h = stream.to(s["x"].dtype).double()        # the norm is of the stored stream
        weighted = h * s["weight"].double()
        biggest = weighted.abs().max(-1).values
        rms = (h.pow(2).sum(-1) / c["n"] + s["eps"]).sqrt()
        return {"codes": None, "scales": biggest / rms / 127.0, "residual": stream}
    if c["op"] == "matmul":
        y = torch.einsum("mk,nk->mn", s["a"].double(), s["w"].double())
        y *= torch.outer(s["a_scales"].double(), s["w_scales"].double())
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "append":
        # the codes are whole numbers that both sides share; the scales have a value in 64 bits
        out = []
        for x, rotate, scales in ((s["k"], c["rotate"], s["cache"][1]), (s["v"], False, s["cache"][3])):
            y = x.double()
            if rotate:
                y = y @ _sylvester(c["d"])
            full = scales.double()
            flat = full.transpose(1, 2).flatten(0, 1)                               # [slots, kv_heads, groups]
            flat[s["slots"]] = y.reshape(y.shape[0], y.shape[1], -1, c["group"]).abs().max(-1).values / 7.0
            out += [None, flat.unflatten(0, (-1, c["page"])).transpose(1, 2)]
        return out
    return _exact_attention(s, c)


def _sylvester(d):
    i = torch.arange(d, device=DEV)
    bits = (i[:, None] & i[None, :])
    sign = torch.ones((d, d), dtype=torch.float64, device=DEV)
    for b in range(d.bit_length()):
        sign = torch.where((bits >> b) & 1 == 1, -sign, sign)
    return sign / math.sqrt(d)


def _exact_attention(s, c):
    lengths = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    rot = _sylvester(c["d"]) if c["rotate"] else None
    for b in range(c["batch"]):
        n = lengths[b]
        if n == 0:
            continue
        pos = torch.arange(n, device=DEV)
        page, at = s["table"][b].long()[pos // c["page"]], pos % c["page"]
        kv = []
        for codes, scales in (s["cache"][:2], s["cache"][2:]):
            raw = codes[page, :, at].to(torch.int64)                                # [n, kv_heads, d / 2]
            nib = torch.stack((raw % 16, raw // 16), -1).reshape(n, c["kv_heads"], c["d"])
            val = torch.where(nib > 7, nib - 16, nib).double()
            kv.append(val * scales[page, :, at].double().repeat_interleave(c["group"], -1))
        for i in range(c["q_len"]):
            m = n - c["q_len"] + i + 1
            if m <= 0:
                continue
            q = s["q"][b, i].double()
            if rot is not None:
                q = q @ rot
            k = kv[0][:m].repeat_interleave(c["ratio"], 1)
            v = kv[1][:m].repeat_interleave(c["ratio"], 1)
            p = torch.softmax(s["scale"] * torch.einsum("hd,mhd->hm", q, k), -1)
            out[b, i] = torch.einsum("hm,mhd->hd", p, v)
    return out
