"""Host-side checks of the int8 linear and int4 cache entry points: every
refusal, made before any CUDA call, so nothing here needs a GPU."""

import pytest
import torch

from hadamard_rotation_bit_b200 import build as hbuild
from hadamard_rotation_bit_b200 import hadq as H

INV, UNS, MIS = H.HADQ_ERR_INVALID_ARG, H.HADQ_ERR_UNSUPPORTED, H.HADQ_ERR_MISALIGNED


def at(i):
    """Fake, aligned device addresses, far apart (never dereferenced)."""
    return i << 44


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return H.load_library()


def norm(lib, x=at(1), xd=1, rows=4, n=1024, residual=at(2), weight=at(3), eps=1e-6, out=at(4), codes=at(5), scales=at(6)):
    return lib.hadq_rmsnorm_quant(x, xd, rows, n, residual, weight, eps, out, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xd=2), INV), (dict(rows=-1), INV), (dict(n=0), INV), (dict(n=1028), UNS), (dict(n=32776), UNS),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(rows=1 << 61), INV),
    (dict(residual=None), INV), (dict(out=None), INV), (dict(x=None), INV), (dict(weight=None), INV),
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(x=at(1) + 8), MIS), (dict(weight=at(3) + 2), MIS),
    (dict(residual=at(2) + 4), MIS), (dict(out=at(4) + 8), MIS), (dict(codes=at(5) + 8), MIS),
    (dict(scales=at(6) + 4), MIS), (dict(codes=at(1)), INV), (dict(codes=at(2) + 16), INV), (dict(scales=at(3)), INV),
    (dict(scales=at(5) + 4080), INV), (dict(out=at(1) + 16), INV), (dict(out=at(2) - 16), INV), (dict(out=at(3)), INV),
    (dict(out=at(5) - 16), INV), (dict(out=at(6) - 16), INV)])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status
    assert lib.hadq_last_error().decode()


def test_empty_calls(lib):
    assert norm(lib, rows=0, x=None, weight=None, codes=None, scales=None, out=None) == H.HADQ_OK
    assert matmul(lib, rows=0, a=None, out=None) == H.HADQ_OK
    assert matmul(lib, cols=0, w=None, out=None) == H.HADQ_OK
    assert append(lib, tokens=0, k=None, slots=None, cache=(None,) * 4) == H.HADQ_OK
    assert attend(lib, batch=0, q=None, out=None, cache=(None,) * 4) == H.HADQ_OK


def matmul(lib, a=at(1), sa=at(2), rows=4, w=at(3), sw=at(4), cols=8, k=64, bias=at(5), out=at(6), od=1):
    return lib.hadq_matmul_int8(a, sa, rows, w, sw, cols, k, bias, out, od, None)


@pytest.mark.parametrize("kw,status", [
    (dict(od=2), INV), (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(k=0), INV), (dict(k=-16), INV), (dict(k=72), UNS),
    (dict(k=131072), UNS), (dict(rows=(1 << 30) + 1), UNS), (dict(cols=(1 << 30) + 1), UNS), (dict(a=None), INV),
    (dict(sa=None), INV), (dict(w=None), INV), (dict(sw=None), INV), (dict(out=None), INV), (dict(a=at(1) + 8), MIS),
    (dict(sa=at(2) + 4), MIS), (dict(w=at(3) + 1), MIS), (dict(sw=at(4) + 4), MIS), (dict(bias=at(5) + 4), MIS),
    (dict(out=at(6) + 2), MIS), (dict(out=at(1) + 16), INV), (dict(out=at(2)), INV), (dict(out=at(3) - 16), INV),
    (dict(out=at(4)), INV), (dict(out=at(5)), INV)])
def test_matmul_refusals(lib, kw, status):
    assert matmul(lib, **kw) == status
    assert lib.hadq_last_error().decode()


CACHE = (at(10), at(11), at(12), at(13))


def append(lib, k=at(1), ks=512, v=at(2), vs=512, dt=1, tokens=3, heads=4, d=128, block=0, group=128, slots=at(3), pages=8,
           page=16, cache=CACHE):
    return lib.hadq_kv4_append(k, ks, v, vs, dt, tokens, heads, d, block, group, slots, pages, page, *cache, None)


CACHE_BAD = [
    (dict(heads=0), INV), (dict(pages=0), INV), (dict(page=0), INV), (dict(page=24), UNS), (dict(page=8), UNS),
    (dict(d=96, group=32), UNS), (dict(d=256), UNS), (dict(group=48), INV), (dict(d=64, group=128), INV), (dict(block=64), UNS),
    (dict(block=2), UNS), (dict(block=-2), UNS), (dict(pages=1 << 27, page=16), UNS), (dict(pages=1 << 40), UNS), (dict(pages=1 << 26, heads=32768), UNS),
    (dict(cache=(None, *CACHE[1:])), INV), (dict(cache=(*CACHE[:3], None)), INV),
    (dict(cache=(CACHE[0] + 8, *CACHE[1:])), MIS), (dict(cache=(*CACHE[:3], CACHE[3] + 2)), MIS),
    (dict(cache=(CACHE[0], CACHE[1], CACHE[0] + 64, CACHE[3])), INV)]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(dt=2), INV), (dict(tokens=-1), INV), (dict(ks=511), INV), (dict(ks=516), MIS), (dict(vs=504), INV),
    (dict(dt=0, vs=514), MIS), (dict(heads=1 << 17, ks=1 << 24, vs=1 << 24), UNS), (dict(tokens=1 << 31), UNS),
    (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV), (dict(k=at(1) + 8), MIS), (dict(v=at(2) + 2), MIS),
    (dict(slots=at(3) + 8), MIS), (dict(k=CACHE[0] + 16), INV), (dict(v=CACHE[1]), INV), (dict(slots=CACHE[3]), INV)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status
    assert lib.hadq_last_error().decode()


def attend(lib, q=at(1), qs=1024, dt=1, batch=2, q_len=1, heads=8, kv=4, d=128, block=0, group=128, cache=CACHE, pages=8,
           page=16, table=at(2), most=4, lengths=at(3), scale=0.1, out=at(4), ws=at(5), nbytes=1 << 30, **kw):
    kv = kw.get("kv_heads", kv)
    return lib.hadq_kv4_attention(q, qs, dt, batch, q_len, heads, kv, d, block, group, *cache, pages, page, table, most, lengths,
                                  scale, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [(dict(kw, kv_heads=kw["heads"], heads=8) if "heads" in kw else kw, st)
                                       for kw, st in CACHE_BAD] + [
    (dict(dt=2), INV), (dict(dt=0), UNS), (dict(batch=-1), INV), (dict(q_len=0), INV), (dict(q_len=65), UNS), (dict(heads=0), INV),
    (dict(heads=6), INV), (dict(most=0), INV), (dict(most=1 << 31), INV), (dict(most=1 << 28), UNS), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(qs=1016), INV), (dict(qs=1028), MIS), (dict(q=None), INV), (dict(table=None), INV),
    (dict(lengths=None), INV), (dict(out=None), INV), (dict(q=at(1) + 8), MIS), (dict(table=at(2) + 4), MIS),
    (dict(lengths=at(3) + 4), MIS), (dict(out=at(4) + 8), MIS), (dict(ws=at(5) + 4), MIS), (dict(out=at(1)), INV),
    (dict(out=at(2)), INV), (dict(out=at(3)), INV), (dict(out=CACHE[2]), INV), (dict(most=4096, ws=None), INV),
    (dict(most=4096, nbytes=64), INV), (dict(most=4096, ws=CACHE[1]), INV), (dict(most=4096, ws=at(4)), INV),
    (dict(most=4096, ws=at(1)), INV)])
def test_attention_refusals(lib, kw, status):
    assert attend(lib, **kw) == status
    assert lib.hadq_last_error().decode()


def test_workspace_sizes(lib):
    f = H.hadq_kv4_attention_workspace
    assert f(0, 1, 8, 4, 128, 64) == 0
    assert f(1024, 1, 8, 4, 128, 1 << 20) == 0                     # enough sequences: no split
    assert f(1, 1, 8, 4, 128, 1 << 20) % (4 * 8 * 130 * 4) == 0 and f(1, 1, 8, 4, 128, 1 << 20) > 0
    assert f(1, 1, 8, 4, 128, 64) == 0                             # too short
    for bad in ((-1, 1, 8, 4, 128, 64), (1, 0, 8, 4, 128, 64), (1, 1, 6, 4, 128, 64), (1, 1, 8, 4, 80, 64),
                (1, 1, 8, 4, 128, 0), (1, 65, 8, 4, 128, 64)):
        assert lib.hadq_kv4_attention_workspace(*bad) == -1
        with pytest.raises(H.HadqError):
            f(*bad)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64)
    for call in (lambda: H.hadq_rmsnorm_quant(x, torch.ones(64)),
                 lambda: H.hadq_matmul_int8(torch.zeros(4, 64, dtype=torch.int8), torch.ones(4),
                                            torch.zeros(8, 64, dtype=torch.int8), torch.ones(8)),
                 lambda: H.hadq_kv4_append(torch.zeros(2, 4, 64), torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int64),
                                           *_host_cache()),
                 lambda: H.hadq_kv4_attention(torch.zeros(2, 4, 64), *_host_cache(), torch.zeros((2, 1), dtype=torch.int32),
                                              torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(H.HadqError):
            call()


def _host_cache():
    return [torch.zeros((2, 4, 16, 32), dtype=torch.uint8), torch.zeros((2, 4, 16, 1), dtype=torch.float16)] * 2


@pytest.mark.parametrize("shape,stride,want", [((3, 4, 64), None, 256), ((3, 4, 64), (768, 64, 1), 768), ((1, 4, 64), (5, 64, 1), 256),
                                               ((2, 3, 4, 64), (2304, 768, 64, 1), 768), ((2, 1, 4, 64), (999, 7, 64, 1), 999)])
def test_token_spacing(shape, stride, want):
    t = torch.zeros(8000)
    t = t[: torch.Size(shape).numel()].view(shape) if stride is None else t.as_strided(shape, stride)
    assert H._token_rows("x", t, shape[-2:]) == want


@pytest.mark.parametrize("shape,stride", [((3, 4, 64), (256, 64, 2)), ((3, 4, 64), (256, 65, 1)), ((2, 3, 4, 64), (3000, 768, 64, 1))])
def test_token_spacing_refusals(shape, stride):
    with pytest.raises(H.HadqError):
        H._token_rows("x", torch.zeros(8000).as_strided(shape, stride), shape[-2:])


def test_every_cluster_barrier_is_arrived_at_before_it_is_waited_for():
    """Read from the source: a wait without its arrival returns early, which no result has to show."""
    import re
    from pathlib import Path

    text = (Path(hbuild.__file__).parent / "csrc" / "hadq_imm.cuh").read_text()
    kernels = re.split(r"^imm_\w+_kernel\(", text, flags=re.M)[1:]
    seen = 0
    for body in kernels:
        calls = re.findall(r"cluster_(arrive|wait)\(\);", body)
        assert calls == ["arrive", "wait"] * (len(calls) // 2)
        seen += len(calls)
    assert seen >= 8
