"""Plain 64-bit implementations of the int8 linear and int4 cache operators,
written from their formulas, and the error bounds their tests use."""

import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative


def norm(x, weight, eps, residual=None):
    """(codes, scales, stream) of the norm: exact codes of the fp32 products, scales in 64 bits."""
    stream = None
    h = x
    if residual is not None:
        stream = (x.float() + residual.float()).to(x.dtype)
        h = stream
    t = (h.float() * weight.float()).double()
    top = t.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, torch.round(127.0 * t / torch.where(top > 0, top, 1.0)), 0.0).to(torch.int8)
    scales = torch.where(top[..., 0] > 0, top[..., 0] / (127.0 * torch.sqrt((h.double() ** 2).mean(-1) + eps)), 0.0)
    return codes, scales, stream


def matmul(a, a_scales, w, w_scales, bias=None):
    y = (a.double() @ w.double().t()) * a_scales.double()[..., None] * w_scales.double()
    return y if bias is None else y + bias.double()


def hadamard(d):
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h


def int4_rows(x, group, rotate):
    """(codes, scales) of rows x [..., d] (numpy float32), bit for bit: fp32
    butterfly stages in ascending order, then one rounding to the integer grid."""
    z = x.astype(np.float32)
    d = z.shape[-1]
    c = np.float32(1.0)
    if rotate:
        c = np.float32(1.0 / math.sqrt(d))
        for bit in range(int(math.log2(d))):
            i = np.arange(d)
            other = z[..., i ^ (1 << bit)]
            z = np.where((i >> bit) & 1, other - z, z + other)
    z = z.reshape(*z.shape[:-1], d // group, group)
    m = np.abs(z).max(-1) * c
    scales = np.minimum(m / np.float32(7.0), np.float32(65504.0)).astype(np.float16)
    s32 = scales.astype(np.float32)
    f = np.where(s32 > 0, c / np.where(s32 > 0, s32, np.float32(1.0)), np.float32(0.0)).astype(np.float32)
    q = np.clip(np.rint(z.astype(np.float64) * f[..., None].astype(np.float64)), -7, 7)
    return q.reshape(*q.shape[:-2], d).astype(np.int8), scales


def pack(q):
    q = q.astype(np.int32) & 15
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    lo, hi = (codes & 15).to(torch.int16), (codes >> 4).to(torch.int16)
    q = torch.stack((lo, hi), -1).flatten(-2)
    return torch.where(q > 7, q - 16, q)


def cached_rows(codes, scales, pages, n):
    """The first n positions of a sequence, [kv_heads, n, d], in 64 bits."""
    group = 2 * codes.shape[-1] // scales.shape[-1]
    c = codes[pages].transpose(0, 1).flatten(1, 2)[:, :n]
    s = scales[pages].transpose(0, 1).flatten(1, 2)[:, :n].double()
    return unpack(c).double() * s.repeat_interleave(group, -1)


def attention(q, cache, table, lengths, scale, rotate):
    """(out, tolerance) in 64 bits: q [batch, q_len, heads, d].

    The bound: the rotated q is rounded to 2^-15 of its row's largest value
    where a cached row has one scale, so a score is off by at most scale 2^-15 max|q| sum |k_d|; with
    more scales to fp16, off by 2^-11 per value, scale 2^-11 sum |q_d k_d|.
    The fp32 rotation and sums of at most 128 products add less than 2^-16 of
    sum |q_d k_d|, taken as 2^-15 of it.  With e the whole, p is off by a factor
    exp(+-e) in numerator and denominator each; P is rounded to fp16 (2^-11)
    or, below 2^-14, by at most 2^-25 per position against codes of at most 8
    in units of the scale of the position that leads the running maximum; exp2
    and the fp32 sums take another 2^-14; the result is rounded to bf16.
    Where e is so large that exp(2 e) says nothing (it is infinite from e = 355
    on), a second bound holds as well: whatever the p are, both results are
    means of the same values with weights that sum to 1, so they lie between
    the smallest and the largest of them and differ by at most their distance,
    next to the roundings above, which are relative to the values.
    """
    k_codes, k_scales, v_codes, v_scales = cache
    page = k_codes.shape[2]
    batch, q_len, heads, d = q.shape
    kv_heads = k_codes.shape[1]
    ratio = heads // kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    one_scale = k_scales.shape[3] == 1
    rot = torch.from_numpy(hadamard(d) / math.sqrt(d)).to(q.device)
    for b in range(batch):
        n = int(lengths[b])
        pages = table[b, : -(-n // page)].long()
        if n == 0:
            continue
        k = cached_rows(k_codes, k_scales, pages, n).repeat_interleave(ratio, 0)      # [heads, n, d]
        v = cached_rows(v_codes, v_scales, pages, n).repeat_interleave(ratio, 0)
        rows = q[b].double() @ rot if rotate else q[b].double()                      # [q_len, heads, d]
        sv = v_scales[pages].transpose(0, 1).flatten(1, 2)[:, :n].double().abs().amax((1, 2)).repeat_interleave(ratio, 0)
        for i in range(q_len):
            m = n - q_len + i + 1
            if m <= 0:
                continue
            row = rows[i]
            p = torch.softmax(scale * torch.einsum("hd,hmd->hm", row, k[:, :m]), -1)
            y = torch.einsum("hm,hmd->hd", p, v[:, :m])
            products = torch.einsum("hd,hmd->hm", row.abs(), k[:, :m].abs())
            if one_scale:
                e = 2.0 ** -15 * (products + row.abs().amax(1, keepdim=True) * k[:, :m].abs().sum(-1))
            else:
                e = (2.0 ** -15 + 2.0 ** -11) * products
            e = abs(scale) * e.amax(-1)
            spread = torch.einsum("hm,hmd->hd", p, v[:, :m].abs())
            out[b, i] = y
            rounding = (2.0 ** -11 + 2.0 ** -14) * (1 + HALF[torch.bfloat16])
            factor = (1 + HALF[torch.bfloat16]) * torch.expm1(2 * e)[:, None]
            near = (y.abs() * HALF[torch.bfloat16] + spread * rounding
                    + torch.where(spread > 0, spread * factor, 0.0) + (m * 2.0 ** -22 * sv)[:, None])
            low, high = v[:, :m].amin(1), v[:, :m].amax(1)
            hull = (high - low) + torch.maximum(low.abs(), high.abs()) * (HALF[torch.bfloat16] + rounding) \
                + (m * 2.0 ** -22 * sv)[:, None]
            tol[b, i] = torch.where(torch.isinf(factor), hull, near)
    return out, tol
