"""GPU: the int8 norm and matrix product, and the int4 cache (append and
attention), against the plain 64-bit implementations of tests/layer_reference.py."""

import math

import numpy as np
import pytest
import torch

from hadamard_rotation_bit_b200 import hadq as H
from tests import layer_reference as R

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _clean():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.load_library()
    yield
    torch.cuda.synchronize()
    assert H.hadq_device_faults(clear=True) == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def untouched(t):
    """The same tensor in the middle of a larger buffer of known bytes, and a check that only it was written."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    inner = buf[256:256 + n].view(t.dtype).view(t.shape)
    inner.copy_(t)

    def check():
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n:] == 0xA5).all())
    return inner, check


# --------------------------------------------------------------------- norm

def check_norm(x, w, eps, residual, codes, scales, stream):
    c, s, h = R.norm(x, w, eps, residual)
    assert torch.equal(codes, c)
    # at most 42 roundings in the sum of squares (halved by the root) and 5 after it
    assert bool(((scales.double() - s).abs() <= 32 * 2.0 ** -24 * s).all())
    if residual is not None:
        assert torch.equal(stream, h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 16), (130, 72), (5, 248), (7, 256), (9, 264), (33, 512), (3, 520),
                                    (777, 1000), (2, 1024), (3, 1032), (5, 2048), (3, 2056), (300, 4096), (1, 4096),
                                    (3, 4104), (4099, 2064), (5000, 4096), (1001, 4104), (1500, 8192), (1000, 14336),
                                    (1203, 16384), (2, 8192), (3, 8200), (2, 14336), (2, 16384), (3, 16392), (2, 32768)])
def test_norm(rows, n, dtype, res):
    g, dt = gen(rows + n), DTYPES[dtype]
    x = randn(g, rows, n, dtype=dt)
    r = (randn(g, rows, n) * 3).to(dt) if res else None
    w = (1 + 0.3 * randn(g, n)).to(dt)
    if rows > 2:
        x[1] = 0
        if res:
            r[1] = 0
    codes, check_c = untouched(torch.zeros((rows, n), dtype=torch.int8, device="cuda"))
    scales, check_s = untouched(torch.zeros(rows, device="cuda"))
    _, _, stream = H.hadq_rmsnorm_quant(x, w, 1e-5, residual=r, codes=codes, scales=scales)
    check_norm(x, w, 1e-5, r, codes, scales, stream)
    check_c(), check_s()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_codes_at_halves(dtype):
    """Quotients exactly on and next to k + 1/2: ties to even, neighbours to their side."""
    dt = DTYPES[dtype]
    n, rows = 256, 64
    x = torch.zeros((rows, n), device="cuda")
    x[:, 0] = 254.0 * (2.0 ** torch.arange(rows, device="cuda").float().sub(32))        # m: 127 t / m = t / 2^(i - 31)
    k = torch.arange(127, device="cuda").float()
    x[:, 1:128] = (2 * k + 1) * (2.0 ** torch.arange(rows, device="cuda").float().sub(32))[:, None]
    near = x[:, 1:128].clone()
    if dtype == "f32":
        near = torch.nextafter(near, torch.full_like(near, math.inf))
    x[:, 128:255] = -near
    x = x.to(dt)
    w = torch.ones(n, dtype=dt, device="cuda")
    codes, scales, _ = H.hadq_rmsnorm_quant(x, w, 1e-6)
    check_norm(x, w, 1e-6, None, codes, scales, None)
    if dtype == "bf16":
        assert codes[3, 1:6].tolist() == [0, 2, 2, 4, 4]


@pytest.mark.parametrize("size", [1e-42, 1e-38, 3e-31, 1e17])
def test_norm_small_and_large_rows(size):
    x = randn(gen(3), 5, 512) * size
    w = torch.ones(512, device="cuda")
    codes, scales, _ = H.hadq_rmsnorm_quant(x, w, 1e-6)
    c, s, _ = R.norm(x, w, 1e-6)
    assert torch.equal(codes, c)
    # a subnormal scale is a multiple of 2^-149
    assert bool(((scales.double() - s).abs() <= 32 * 2.0 ** -24 * s + 2.0 ** -149).all())


@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("rows,n", [(64, 4096), (5000, 4096), (1100, 14336)])
def test_norm_in_place(rows, n, target):
    g = gen(5)
    x, r = randn(g, rows, n, dtype=torch.bfloat16), randn(g, rows, n, dtype=torch.bfloat16)
    w = randn(g, n, dtype=torch.bfloat16)
    x0, r0 = x.clone(), r.clone()
    codes, scales, stream = H.hadq_rmsnorm_quant(x, w, residual=r, residual_out=x if target == "x" else r)
    assert stream.data_ptr() == (x if target == "x" else r).data_ptr()
    check_norm(x0, w, 1e-6, r0, codes, scales, stream)
    assert torch.equal(r if target == "x" else x, r0 if target == "x" else x0)


@pytest.mark.parametrize("rows,n", [(3, 256), (5000, 4096)])
def test_norm_zero_rows_without_eps(rows, n):
    x, w = torch.zeros((rows, n), device="cuda"), torch.ones(n, device="cuda")
    x[1] = 1.0
    codes, scales, _ = H.hadq_rmsnorm_quant(x, w, 0.0)
    check_norm(x, w, 0.0, None, codes, scales, None)
    assert float(scales[0]) == 0.0 and int(codes[1, 5]) == 127


@pytest.mark.parametrize("rows,n", [(3, 256), (5000, 4096)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_norm_shows_rows_that_are_no_numbers(rows, n, bad):
    x, w = randn(gen(5), rows, n), torch.ones(n, device="cuda")
    codes, scales, _ = H.hadq_rmsnorm_quant(x, w, 1e-6)
    x[1, 7] = bad
    x[2] = math.nan
    codes_, scales_, _ = H.hadq_rmsnorm_quant(x, w, 1e-6)
    assert bool(scales_[1:3].isnan().all())
    keep = [i for i in range(rows) if i not in (1, 2)]
    assert torch.equal(codes[keep], codes_[keep]) and torch.equal(scales[keep], scales_[keep])


def test_norm_leading_dimensions_and_empty():
    g = gen(6)
    x, w = randn(g, 2, 3, 128), randn(g, 128)
    codes, scales, none = H.hadq_rmsnorm_quant(x, w)
    assert codes.shape == (2, 3, 128) and scales.shape == (2, 3) and none is None
    check_norm(x, w, 1e-6, None, codes, scales, None)
    codes, scales, _ = H.hadq_rmsnorm_quant(x[:, :0].contiguous(), w)
    assert codes.shape == (2, 0, 128) and scales.shape == (2, 0)


# ------------------------------------------------------------------- matmul

def check_matmul(out, a, sa, w, sw, bias):
    y = R.matmul(a, sa, w, sw)
    z = y if bias is None else y + bias.double()
    # the sum to fp32 and two products, the bias, and the output's rounding
    tol = y.abs() * 3.01 * 2.0 ** -24 + z.abs() * (1.01 * 2.0 ** -24 + R.HALF[out.dtype] * (out.dtype != torch.float32))
    err = (out.double() - z).abs()
    assert bool((err <= tol).all()), f"{float((err - tol).max())} over"


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 128, 4096), (4, 131, 14336), (3, 515, 4096), (2, 40, 16), (1, 4096, 14336), (2, 129, 48), (3, 7, 144), (5, 333, 112),
                                   (8, 4096, 512), (5, 9001, 80), (8, 8200, 4112), (13, 8193, 1040), (7, 33, 16), (16, 4096, 14336), (9, 200, 1040), (16, 1000, 4112), (17, 256, 128), (32, 512, 272),
                                   (33, 130, 96), (48, 1433, 4096), (64, 384, 1040), (65, 96, 208), (127, 255, 256),
                                   (128, 256, 64), (129, 257, 80), (200, 1024, 4096), (256, 128, 2048), (257, 511, 640),
                                   (333, 1001, 4112), (512, 4096, 1024), (1025, 520, 384), (2000, 24, 256),
                                   (40, 20000, 64), (300, 8, 16), (1300, 2100, 208), (300, 5201, 4112), (200, 10250, 64),
                                   (10300, 40, 96), (2048, 2048, 1024), (2817, 1032, 272),
                                   (70, 19201, 80), (128, 20000, 144), (64, 19300, 272), (50, 19000, 1040), (20, 4100, 8192), (65, 129, 4096),
                                   (90, 8200, 8192), (200, 2047, 14336), (333, 4100, 4112), (130, 500, 65536), (200, 6101, 4112)])
def test_matmul(m, n, k, out):
    g = gen(m + n + k)
    a = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(m, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda") * 1e-3
    bias = randn(g, n) if (m + n) % 2 else None
    buf, check = untouched(torch.zeros((m, n), dtype=DTYPES[out], device="cuda"))
    H.hadq_matmul_int8(a, sa, w, sw, bias=bias, out=buf)
    check_matmul(buf, a, sa, w, sw, bias)
    check()


@pytest.mark.parametrize("k", [16, 32, 48, 80])
@pytest.mark.parametrize("m", [5, 8, 11, 16])
def test_matmul_rows_shorter_than_a_round(m, k):
    """The bytes beside the last row hold no part of the result: the same in a buffer of its own and between others."""
    g = gen(m + k)
    wide = torch.randint(-127, 128, (m + 2, k), generator=g, device="cuda", dtype=torch.int8)
    a, w = wide[1:-1], torch.randint(-127, 128, (33, k), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(m, generator=g, device="cuda"), torch.rand(33, generator=g, device="cuda")
    out = H.hadq_matmul_int8(a, sa, w, sw, out_dtype=torch.float32)
    check_matmul(out, a, sa, w, sw, None)
    wide[0], wide[-1] = 127, -128
    assert torch.equal(out, H.hadq_matmul_int8(a.clone(), sa, w, sw, out_dtype=torch.float32))
    assert torch.equal(out, H.hadq_matmul_int8(a, sa, w, sw, out_dtype=torch.float32))


@pytest.mark.parametrize("m,n", [(1, 130), (3, 33), (9, 40), (17, 65), (200, 300)])
def test_matmul_largest_sums(m, n):
    """-128 x -128 over the longest k: 2147221504, just inside 32 bits."""
    k = 131056
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    out = H.hadq_matmul_int8(a, one_m, w, one_n, out_dtype=torch.float32)
    want = torch.tensor([128.0 * 128 * k, -128.0 * 127 * k], device="cuda").repeat(n // 2 + 1)[:n]
    assert bool((out == want.float()).all())


def test_matmul_leading_dimensions_zero_scales_and_empty():
    g = gen(9)
    a = torch.randint(-127, 128, (2, 5, 64), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (40, 64), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.zeros((2, 5), device="cuda"), torch.ones(40, device="cuda")
    out = H.hadq_matmul_int8(a, sa, w, sw)
    assert out.shape == (2, 5, 40) and not bool(out.any())
    assert H.hadq_matmul_int8(a[:, :0].contiguous(), sa[:, :0].contiguous(), w, sw).shape == (2, 0, 40)
    assert H.hadq_matmul_int8(a, sa, w[:0], sw[:0]).shape == (2, 5, 0)


def test_matmul_same_result_every_time():
    g = gen(10)
    for m in (1, 4, 12, 24, 300):
        a = torch.randint(-127, 128, (m, 14336), generator=g, device="cuda", dtype=torch.int8)
        w = torch.randint(-127, 128, (1024, 14336), generator=g, device="cuda", dtype=torch.int8)
        sa, sw = torch.rand(m, device="cuda"), torch.rand(1024, device="cuda")
        first = H.hadq_matmul_int8(a, sa, w, sw)
        for _ in range(5):
            assert torch.equal(first, H.hadq_matmul_int8(a, sa, w, sw))


# --------------------------------------------------------------- int4 cache

def new_cache(g, pages, heads, page, d, group):
    """Four tensors with random finite content: other sequences' rows."""
    out = []
    for _ in range(2):
        out.append(torch.randint(0, 256, (pages, heads, page, d // 2), generator=g, device="cuda", dtype=torch.uint8))
        out.append((0.02 + 0.5 * torch.rand((pages, heads, page, d // group), generator=g, device="cuda")).half())
    return out


def expect_append(cache, k, v, slots, rotate):
    """The cache after an append, from the bitwise definition."""
    page, d = cache[0].shape[2], 2 * cache[0].shape[3]
    group = d // cache[1].shape[3]
    want = [t.clone() for t in cache]
    keep = slots >= 0
    at = slots[keep]
    for x, rot, codes, scales in ((k, rotate, want[0], want[1]), (v, False, want[2], want[3])):
        q, s = R.int4_rows(x[keep].float().cpu().numpy(), group, rot)
        codes[at // page, :, at % page] = torch.from_numpy(R.pack(q)).cuda()
        scales[at // page, :, at % page] = torch.from_numpy(s).cuda()
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("tokens,heads,d,group,page", [(1, 1, 128, 128, 16), (1, 8, 128, 128, 64), (3, 2, 64, 64, 16),
                                                       (17, 3, 128, 32, 48), (100, 5, 64, 32, 32), (33, 4, 128, 64, 80),
                                                       (500, 8, 128, 128, 128), (257, 1, 64, 32, 16)])
def test_append(tokens, heads, d, group, page, rotate, dtype):
    g, dt = gen(tokens + heads + d), DTYPES[dtype]
    pages = tokens // page + 3
    cache = new_cache(g, pages, heads, page, d, group)
    qkv = randn(g, tokens, 3, heads, d)
    qkv[..., 5] *= 30
    if tokens > 2:
        qkv[1] = 0
        qkv[2] *= 1e-9                               # scales that round to zero,
    if tokens > 8:
        qkv[5:9] *= torch.tensor([2e-7, 4e-7, 1e-6, 1e-4], device="cuda").view(4, 1, 1, 1)     # and subnormal ones
    qkv = qkv.to(dt)
    k, v = qkv[:, 1], qkv[:, 2]                      # slices of a fused projection
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    if tokens > 4:
        slots[3] = -1
        slots[4] = -(2 ** 40)
    want = expect_append(cache, k, v, slots, rotate)
    H.hadq_kv4_append(k, v, slots, *cache, block=0 if rotate else 1)
    for got, w in zip(cache, want):
        assert torch.equal(got, w)


def test_append_agrees_with_rotate_quant():
    """The same codes as the library's R3 quantizer, up to its own parity rule."""
    g = gen(21)
    k = randn(g, 64, 8, 128, dtype=torch.bfloat16)
    cache = new_cache(g, 4, 8, 16, 128, 128)
    H.hadq_kv4_append(k, k, torch.arange(64, device="cuda"), *cache)
    codes, scales = H.hadq_rotate_quant(k, 128, "int4", 128)
    mine = cache[0].transpose(1, 2).reshape(64 * 8, 64)
    smine = cache[1].transpose(1, 2).reshape(64 * 8, 1)
    # scales within one fp16 step; where they agree, codes within one step and nearly always equal
    codes, scales = codes.reshape(512, 64), scales.reshape(512, 1)
    assert bool(((smine.double() - scales.double()).abs() <= 2.0 ** -10 * scales.double()).all())
    same = (smine == scales).expand(-1, 128)
    diff = (R.unpack(mine) - R.unpack(codes)).abs()[same]
    assert int(diff.max()) <= 1 and float((diff > 0).float().mean()) < 1e-3


@pytest.mark.parametrize("size,saturates", [(1e5, False), (3e6, True), (1e38, True)])
def test_append_huge_rows_saturate(size, saturates):
    g = gen(22)
    x = (randn(g, 4, 1, 128) * size).clamp(-3e38, 3e38)
    cache = new_cache(g, 2, 1, 16, 128, 128)
    slots = torch.arange(4, device="cuda")
    want = expect_append(cache, x, x, slots, False)
    H.hadq_kv4_append(x, x, slots, *cache, block=1)
    for got, w in zip(cache, want):
        assert torch.equal(got, w)
    assert bool(torch.isfinite(cache[3].float()).all())
    assert (float(cache[3].float().max()) == 65504.0) == saturates


def test_append_shows_rows_that_are_no_numbers():
    k = randn(gen(24), 3, 2, 128)
    k[1, 0, 9] = math.nan
    cache = new_cache(gen(25), 1, 2, 16, 128, 32)
    H.hadq_kv4_append(k, k, torch.arange(3, device="cuda"), *cache)
    assert bool(cache[1][0, 0, 1].isnan().all()) and int(cache[1][0, :, :3].isnan().sum()) == 4
    assert not bool(cache[3].isnan().any())


def test_append_slots_outside_the_cache_are_recorded():
    g = gen(23)
    k = randn(g, 5, 2, 64, dtype=torch.bfloat16)
    cache = new_cache(g, 3, 2, 16, 64, 64)
    slots = torch.tensor([0, 48, 47, 2 ** 33 + 5, -7], device="cuda")
    inside = torch.where(slots < 48, slots, -1)
    want = expect_append(cache, k, k, inside, True)
    H.hadq_kv4_append(k, k, slots, *cache)
    torch.cuda.synchronize()
    assert H.hadq_device_faults(clear=True) == 64
    for got, w in zip(cache, want):
        assert torch.equal(got, w)


def attention_case(seed, batch, q_len, kv_heads, ratio, d, group, page, lengths, spread=0.0):
    g = gen(seed)
    most = max(1, -(-max(lengths) // page))
    pages = batch * most + 2
    cache = new_cache(g, pages, kv_heads, page, d, group)
    if spread:                                       # scales over many binades, zeros among them
        for i in (1, 3):
            s = torch.exp2(torch.randint(-10, 3, cache[i].shape, generator=g, device="cuda").float() * spread)
            s[torch.rand(cache[i].shape, generator=g, device="cuda") < 0.1] = 0
            cache[i] = (0.1 * s).half()
    q = randn(g, batch, q_len, kv_heads * ratio, d, dtype=torch.bfloat16)
    table = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)[: batch * most].view(batch, most)
    return q, cache, table.contiguous(), torch.tensor(lengths, dtype=torch.int32, device="cuda")


def check_attention(out, q, cache, table, lengths, scale, rotate):
    want, tol = R.attention(q, cache, table, lengths, scale, rotate)
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol.clamp_min(1e-30)).max())} of the bound"


@pytest.mark.parametrize("q_len,kv_heads,ratio,d,group,page,lengths", [
    (1, 1, 1, 128, 128, 16, [1]), (1, 1, 1, 64, 64, 16, [1]), (1, 2, 1, 128, 128, 16, [15, 16, 17, 0]),
    (1, 2, 4, 128, 128, 64, [64, 63, 65, 200]), (1, 8, 4, 128, 128, 64, [1000, 1]), (1, 3, 5, 64, 32, 48, [47, 48, 49, 333]),
    (1, 2, 8, 128, 32, 32, [100, 31, 0, 513]), (1, 1, 16, 128, 64, 16, [257]), (1, 2, 11, 64, 64, 16, [129, 5]),
    (2, 2, 4, 128, 128, 16, [1, 2, 0, 50]), (3, 1, 8, 128, 32, 16, [2, 3, 4, 100]), (4, 2, 4, 128, 64, 32, [4, 3, 1, 97]),
    (5, 1, 7, 64, 32, 16, [40, 6]), (8, 2, 8, 128, 128, 128, [300, 7]), (16, 1, 3, 64, 64, 16, [16, 15, 33]),
    (64, 1, 2, 128, 128, 16, [70, 64, 63]), (1, 1, 1, 128, 128, 16, [5000]), (1, 4, 2, 64, 32, 64, [3001, 64, 2999]),
    (1, 40, 1, 128, 128, 16, [33, 12]), (1, 1, 64, 128, 32, 16, [77])])
@pytest.mark.parametrize("rotate", [True, False])
def test_attention(q_len, kv_heads, ratio, d, group, page, lengths, rotate):
    q, cache, table, ln = attention_case(q_len + ratio + sum(lengths), len(lengths), q_len, kv_heads, ratio, d, group, page, lengths)
    scale = 1 / math.sqrt(d)
    out, check = untouched(torch.zeros_like(q))
    H.hadq_kv4_attention(q, *cache, table, ln, block=0 if rotate else 1, out=out)
    check_attention(out, q, cache, table, ln, scale, rotate)
    check()


@pytest.mark.parametrize("d,group", [(128, 128), (128, 64), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("scale", [0.0, 0.02, 1.0, -0.3])
def test_attention_scales_of_many_sizes(d, group, scale):
    """Flat and peaked probabilities, V's scales (zeros too) over 2^26: what fp16 products could lose."""
    q, cache, table, ln = attention_case(7, 3, 2, 2, 3, d, group, 32, [700, 33, 1], spread=2.0)
    out = H.hadq_kv4_attention(q, *cache, table, ln, scale=scale)
    check_attention(out, q, cache, table, ln, scale, True)


def test_attention_large_and_tiny_queries():
    q, cache, table, ln = attention_case(8, 4, 1, 2, 2, 128, 128, 16, [50, 51, 52, 53])
    size = torch.tensor([1e-30, 1e4, 0.0, 1e-3], device="cuda").view(4, 1, 1, 1)
    q = (q.float() * size).to(torch.bfloat16)
    out = H.hadq_kv4_attention(q, *cache, table, ln, scale=1e-3)
    check_attention(out, q, cache, table, ln, 1e-3, True)


@pytest.mark.parametrize("group", [128, 32])
def test_attention_rows_of_one_tile_do_not_disturb_each_other(group):
    """Heads that share a K/V head, 2^40 apart in size, one of them infinite: every other row is what it is alone."""
    q, cache, table, ln = attention_case(14, 1, 2, 2, 4, 128, group, 16, [45])
    size = torch.tensor([1.0, 2.0 ** 20, 2.0 ** -20, 1.0, 1.0, 1.0, 3.0, 1.0], device="cuda").view(1, 1, 8, 1)
    q = (q.float() * size).to(torch.bfloat16)
    out = H.hadq_kv4_attention(q, *cache, table, ln, scale=0.05)
    check_attention(out, q, cache, table, ln, 0.05, True)
    bad = q.clone()
    bad[0, 0, 3], bad[0, 1, 5, 7] = math.inf, math.nan
    got = H.hadq_kv4_attention(bad, *cache, table, ln, scale=0.05)
    keep = torch.ones((1, 2, 8), dtype=torch.bool, device="cuda")
    keep[0, 0, 3] = keep[0, 1, 5] = False
    assert torch.equal(got[keep], out[keep])
    assert bool(got[~keep].isnan().all())


@pytest.mark.parametrize("d,group,n", [(128, 128, 45), (128, 32, 45), (64, 64, 2100), (128, 128, 9000)])
@pytest.mark.parametrize("which", [1, 3])
def test_attention_shows_scales_that_are_no_numbers(d, group, n, which):
    """A NaN or an infinity as the scale of a position: the K/V head's rows that see it are no numbers, the others are untouched."""
    q, cache, table, ln = attention_case(15, 2, 2, 2, 2, d, group, 16, [n, n])
    want = H.hadq_kv4_attention(q, *cache, table, ln)
    for value, at in ((math.nan, 0), (math.inf, 0), (math.nan, n - 1), (math.inf, n - 1), (math.nan, n // 2)):
        dirty = [t.clone() for t in cache]
        dirty[which][table[1, at // 16].long(), 1, at % 16] = value
        got = H.hadq_kv4_attention(q, *dirty, table, ln)
        first = 1 if at == n - 1 else 0                # the newest position is seen by the last query alone
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[1, first:, 2:] = False
        assert torch.equal(got[keep], want[keep])
        if which == 3 or math.isnan(value):            # K: an infinite score of -inf is a position without weight
            assert not bool(got[1, first:, 2:].isfinite().any())


def test_attention_far_scores():
    """Scores down to -2^100: the least of them still sum to one."""
    q, cache, table, ln = attention_case(16, 1, 1, 1, 2, 128, 128, 16, [3])
    cache[0].fill_(0x11), cache[1].fill_(60000.0)
    q = torch.full_like(q, -(2.0 ** 86))
    out = H.hadq_kv4_attention(q, *cache, table, ln, block=1, scale=0.25)
    v = R.cached_rows(cache[2], cache[3], table[0].long(), 3)
    assert bool((out[0, 0].double() - v.mean(1)).abs().le(v.abs().mean(1) * 2.0 ** -7).all())


@pytest.mark.parametrize("bits", [0x7C00, 0xFC00, 0x7E00, 0xFBFF])
def test_attention_ignores_what_lies_beyond_a_length(bits):
    """inf, -inf, NaN and -max scales in positions that no query sees, or only a later query sees."""
    q, cache, table, ln = attention_case(9, 2, 1, 2, 4, 128, 64, 32, [37, 64])
    dirty = [t.clone() for t in cache]
    for i in (1, 3):
        dirty[i][table[0, 1].long(), :, 5:] = torch.tensor(bits, dtype=torch.int32).to(torch.int16).view(torch.float16).item()
    want = H.hadq_kv4_attention(q, *cache, table, ln)
    assert torch.equal(want, H.hadq_kv4_attention(q, *dirty, table, ln))
    # drafted tokens: the newest position is seen by the last query alone
    q4 = randn(gen(1), 1, 4, 8, 128, dtype=torch.bfloat16)
    tab, l4 = table[:1].contiguous(), torch.tensor([38], dtype=torch.int32, device="cuda")
    assert torch.equal(H.hadq_kv4_attention(q4, *cache, tab, l4)[:, :3], H.hadq_kv4_attention(q4, *dirty, tab, l4)[:, :3])


def test_attention_bad_pages_and_lengths_are_recorded():
    q, cache, table, ln = attention_case(10, 3, 1, 2, 2, 128, 128, 16, [40, 40, 40])
    want = H.hadq_kv4_attention(q, *cache, table, ln)
    bad = table.clone()
    bad[0, 1], bad[1, 2] = -1, cache[0].shape[0]
    got = H.hadq_kv4_attention(q, *cache, bad, ln)
    torch.cuda.synchronize()
    assert H.hadq_device_faults(clear=True) == 16
    assert torch.equal(got[2], want[2])
    # sequence 1 lost its last page: as if it had 32 positions
    short = H.hadq_kv4_attention(q, *cache, table, torch.tensor([40, 32, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(got[1], short[1])
    # sequence 0 without its middle page: attention over the other positions
    hole = torch.stack((table[0, 0], table[0, 2])).view(1, 2).contiguous()
    ref, tol = R.attention(q[:1], cache, hole, torch.tensor([24]), 128 ** -0.5, True)
    assert bool(((got[:1].double() - ref).abs() <= tol).all())
    out = H.hadq_kv4_attention(q, *cache, table, torch.tensor([-3, 49, 40], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert H.hadq_device_faults(clear=True) == 32
    assert not bool(out[0].any()) and torch.equal(out[2], want[2])


@pytest.mark.parametrize("batch,q_len,kv_heads,ratio", [(75, 2, 8, 8), (150, 1, 8, 1), (64, 3, 6, 4), (65, 1, 16, 2)])
def test_attention_batches_beyond_the_gpu(batch, q_len, kv_heads, ratio):
    """More units than are computed at once, lengths of all sizes, equal ones and empty ones among them."""
    g = torch.Generator().manual_seed(batch)
    lengths = torch.randint(0, 1101, (batch,), generator=g).tolist()
    lengths[3], lengths[5], lengths[-1], lengths[-2], lengths[7] = 0, 1100, 1100, 0, lengths[8]
    q, cache, table, ln = attention_case(18, batch, q_len, kv_heads, ratio, 128, 128, 64, lengths)
    out = H.hadq_kv4_attention(q, *cache, table, ln)
    check_attention(out, q, cache, table, ln, 128 ** -0.5, True)
    # the same sequences in another order
    order = torch.randperm(batch, generator=g).cuda()
    again = H.hadq_kv4_attention(q[order].contiguous(), *cache, table[order].contiguous(), ln[order].contiguous())
    assert torch.equal(again, out[order])


@pytest.mark.parametrize("as_handle", [False, True])
def test_attention_on_another_stream_keeps_its_workspace(as_handle):
    """Memory that this stream asks for after the call is not what the other stream still computes in."""
    q, cache, table, ln = attention_case(17, 1, 1, 2, 4, 128, 128, 16, [4000])
    need = H.hadq_kv4_attention_workspace(1, 1, 8, 2, 128, table.shape[1] * 16)
    assert need > 0
    want, out = H.hadq_kv4_attention(q, *cache, table, ln), torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)                 # about a millisecond
        H.hadq_kv4_attention(q, *cache, table, ln, out=out, stream=side.cuda_stream if as_handle else side)
        noise = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del noise
    assert torch.equal(H.hadq_kv4_attention(q, *cache, table, ln, stream=0 if as_handle else torch.cuda.default_stream()), want)


def test_attention_query_slices_and_three_dimensions():
    g = gen(11)
    _, cache, table, ln = attention_case(11, 3, 1, 2, 4, 128, 128, 16, [20, 0, 45])
    qkv = randn(g, 3, 12, 128, dtype=torch.bfloat16)
    q = qkv[:, :8]                                   # the queries of a fused projection
    out = H.hadq_kv4_attention(q, *cache, table, ln)
    assert out.shape == (3, 8, 128)
    assert torch.equal(out, H.hadq_kv4_attention(q.contiguous().unsqueeze(1), *cache, table, ln)[:, 0])


def test_attention_splits_agree():
    """Tables of different widths split a sequence differently; the results stay within the bound, and repeat exactly."""
    q, cache, table, ln = attention_case(12, 2, 1, 2, 4, 128, 128, 16, [900, 1777])
    for cols in (112, 300, 2000):
        wide = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
        wide[:, : table.shape[1]] = table
        out = H.hadq_kv4_attention(q, *cache, wide, ln)
        check_attention(out, q, cache, table, ln, 128 ** -0.5, True)
        for _ in range(3):
            assert torch.equal(out, H.hadq_kv4_attention(q, *cache, wide, ln))


def test_cache_offsets_past_32_bits():
    """Pages whose codes start beyond 2^32 bytes."""
    heads, page, d = 8, 64, 128
    pages = (1 << 17) + 4
    cache = [torch.empty((pages, heads, page, d // 2 if i % 2 == 0 else 1), dtype=torch.uint8 if i % 2 == 0 else torch.float16,
                         device="cuda") for i in range(4)]
    assert cache[0].numel() > 1 << 32
    g = gen(13)
    n = 150
    k, v = randn(g, n, heads, d, dtype=torch.bfloat16), randn(g, n, heads, d, dtype=torch.bfloat16)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = table[0].long()[pos // page] * page + pos % page
    H.hadq_kv4_append(k, v, slots, *cache)
    small = [torch.zeros((3, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in cache]
    H.hadq_kv4_append(k, v, pos, *small)
    q = randn(g, 1, 1, 16, d, dtype=torch.bfloat16)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    near = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    want = H.hadq_kv4_attention(q, *small, near, ln)
    assert torch.equal(want, H.hadq_kv4_attention(q, *cache, table, ln))
    check_attention(want, q, small, near, ln, d ** -0.5, True)


# ------------------------------------------------------- together, as a layer

def make_layer(g, hidden, heads, kv_heads, d, inter):
    def linear(n, k):
        w = randn(g, n, k) / math.sqrt(k)
        s = w.abs().amax(1) / 127
        return (w / s[:, None]).round().to(torch.int8), s
    return dict(n1=(1 + 0.1 * randn(g, hidden)).bfloat16(), n2=(1 + 0.1 * randn(g, hidden)).bfloat16(),
                qkv=linear((heads + 2 * kv_heads) * d, hidden), o=linear(hidden, heads * d),
                up=linear(2 * inter, hidden), down=linear(hidden, inter), heads=heads, kv_heads=kv_heads, d=d)


def layer_step(p, delta, stream, cache, slots, table, lengths, q_len):
    """One decoder layer on quantized operands: delta is the previous layer's output, stream the residual."""
    heads, kv, d = p["heads"], p["kv_heads"], p["d"]
    a, sa, stream = H.hadq_rmsnorm_quant(delta, p["n1"], residual=stream)
    qkv = H.hadq_matmul_int8(a, sa, *p["qkv"]).unflatten(1, (heads + 2 * kv, d))
    H.hadq_kv4_append(qkv[:, heads:heads + kv], qkv[:, heads + kv:], slots, *cache)
    q = qkv[:, :heads].unflatten(0, (-1, q_len))
    y = H.hadq_kv4_attention(q, *cache, table, lengths)
    a, sa = H.hadq_rotate_quant(y.reshape(-1, heads * d), 1, "int8", 0)
    delta = H.hadq_matmul_int8(a, sa, *p["o"])
    a, sa, stream = H.hadq_rmsnorm_quant(delta, p["n2"], residual=stream)
    gate, up = H.hadq_matmul_int8(a, sa, *p["up"]).chunk(2, 1)
    a, sa = H.hadq_rotate_quant((torch.nn.functional.silu(gate) * up).contiguous(), 0, "int8", 0)
    return H.hadq_matmul_int8(a, sa, *p["down"]), stream


def layer_reference(p, delta, stream, cache, slots, table, lengths, q_len):
    """The same step from the plain implementations, rounded where the library stores."""
    heads, kv, d = p["heads"], p["kv_heads"], p["d"]
    bf = torch.bfloat16
    a, sa, stream = R.norm(delta, p["n1"], 1e-6, stream)
    qkv = R.matmul(a, sa, *p["qkv"]).to(bf).unflatten(1, (heads + 2 * kv, d))
    cache = expect_append(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], slots, True)
    y = R.attention(qkv[:, :heads].unflatten(0, (-1, q_len)), cache, table, lengths, d ** -0.5, True)[0].to(bf)

    def int8(x, rotate):
        x = x.double()
        if rotate:
            x = x @ torch.from_numpy(R.hadamard(x.shape[1]) / math.sqrt(x.shape[1])).cuda()
        s = x.abs().amax(1) / 127
        return (x / s[:, None]).round(), s
    delta = R.matmul(*int8(y.reshape(-1, heads * d), False), *p["o"]).to(bf)
    a, sa, stream = R.norm(delta, p["n2"], 1e-6, stream)
    gate, up = R.matmul(a, sa, *p["up"]).to(bf).chunk(2, 1)
    act = torch.nn.functional.silu(gate) * up
    return R.matmul(*int8(act, True), *p["down"]).to(bf), stream


def test_layer_prefill_then_decode():
    """Prompts through the layer, then three tokens one by one, then four drafted ones: the residual stream, the
    cache and the output against the plain implementations."""
    g = gen(31)
    p = make_layer(g, 512, 8, 2, 64, 1024)
    cache = new_cache(g, 24, 2, 16, 64, 64)
    table = torch.randperm(24, generator=g, device="cuda", dtype=torch.int32)[:8].view(2, 4).contiguous()
    done = 0
    for q_len in (21, 1, 1, 1, 4):
        delta, stream = randn(g, 2 * q_len, 512, dtype=torch.bfloat16), randn(g, 2 * q_len, 512, dtype=torch.bfloat16)
        pos = torch.arange(done, done + q_len, device="cuda")
        slots = (table.long()[:, pos // 16] * 16 + pos % 16).flatten()
        done += q_len
        ln = torch.full((2,), done, dtype=torch.int32, device="cuda")
        want, wstream = layer_reference(p, delta, stream, [t.clone() for t in cache], slots, table, ln, q_len)
        got, gstream = layer_step(p, delta, stream, cache, slots, table, ln, q_len)
        # A value next to a rounding border may take the other int8 or int4 code in one of the two.  Each of the five
        # quantizers in the chain moves a value by at most a code when that happens, 1/127 (int8) or 1/7 (int4, averaged
        # by the softmax) of its row's largest; norms over the whole output see a few percent at most.
        for a, b in ((got, want), (gstream, wstream)):
            assert float((a.double() - b.double()).norm() / b.double().norm()) < 0.03


def test_layer_captured_and_replayed():
    """A decode step captured into a graph and replayed with new contents gives what the eager calls give; a second
    graph of the same step has its own workspace."""
    g = gen(32)
    p = make_layer(g, 512, 8, 2, 128, 1024)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    state = [(randn(g, 2, 512, dtype=torch.bfloat16), randn(g, 2, 512, dtype=torch.bfloat16)) for _ in range(3)]
    base = new_cache(g, 40, 2, 16, 128, 128)
    graphs = []
    for _ in range(2):
        buf = dict(delta=torch.zeros_like(state[0][0]), stream=torch.zeros_like(state[0][0]), cache=[t.clone() for t in base],
                   slots=torch.zeros(2, dtype=torch.int64, device="cuda"), ln=torch.ones(2, dtype=torch.int32, device="cuda"))

        def step(b=buf):
            return layer_step(p, b["delta"], b["stream"], b["cache"], b["slots"], table, b["ln"], 1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            buf["out"] = step()
        for t, s in zip(buf["cache"], base):
            t.copy_(s)
        graphs.append((graph, buf))
    caches = [[t.clone() for t in base] for _ in graphs]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for i, (delta, stream) in enumerate(state):
        n = [290 + i, 17 + i]
        ln = torch.tensor(n, dtype=torch.int32, device="cuda")
        slots = torch.stack([table[b].long()[(x - 1) // 16] * 16 + (x - 1) % 16 for b, x in enumerate(n)])
        for j, (graph, buf) in enumerate(graphs):
            buf["delta"].copy_(delta * (j + 1)), buf["stream"].copy_(stream), buf["ln"].copy_(ln), buf["slots"].copy_(slots)
        torch.cuda.synchronize()
        for s, (graph, _) in zip(streams, graphs):       # both graphs in flight at once
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for j, (_, buf) in enumerate(graphs):
            want = layer_step(p, delta * (j + 1), stream, caches[j], slots, table, ln, 1)
            for a, b in zip(buf["out"], want):
                assert torch.equal(a, b)
            for a, b in zip(buf["cache"], caches[j]):
                assert torch.equal(a, b)


def test_calls_on_another_stream():
    """Given a stream by argument, or the current one: work waits for that stream's earlier work."""
    g = gen(33)
    x, w = randn(g, 4096, 4096, dtype=torch.bfloat16), randn(g, 4096, dtype=torch.bfloat16)
    want = H.hadq_rmsnorm_quant(x, w)
    late = torch.zeros_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            late.mul_(0.5)
        late.copy_(x)
    got = H.hadq_rmsnorm_quant(late, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
