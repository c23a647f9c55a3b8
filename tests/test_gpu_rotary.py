"""rotary and rotary_and_cache against the rotation in 64 bits."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def rows(gen, *shape):
    x = torch.randn(shape, generator=gen)
    x[..., 3::29] *= 30.0
    return x.to(torch.bfloat16).cuda()


def reference(x, pos, freqs, inter, factor, inverse):
    """(rotated rows in float64, what the two products of an element sum to in magnitude)."""
    x = x.detach().cpu().double().numpy()
    f = freqs.cpu().numpy().view(np.uint64)
    with np.errstate(over="ignore"):
        turns = np.asarray(pos, np.int64).view(np.uint64)[:, None] * f[None]
    t = turns.view(np.int64).astype(np.float64) * 2.0 ** -63 * np.pi
    if inverse:
        t = -t
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    r = 2 * len(f)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., i], x[..., j]
    out, mag = x.copy(), np.zeros_like(x)
    out[..., i], out[..., j] = (a * c - b * s) * factor, (b * c + a * s) * factor
    mag[..., i] = mag[..., j] = (np.abs(a) + np.abs(b)) * abs(factor)
    return out, mag


def check(got, ref):
    # the result is rounded to bf16 (half a step: 2^-8); before that, the angle is off by 2^-25 half turns (1e-7
    # radians), sine and cosine by two steps (2^-22), factor, products and sum by half a step each (2^-24): below
    # 2^-20 of |a| + |b|
    out, mag = ref
    g = got.detach().cpu().double().numpy()
    assert np.isfinite(g).all()
    assert (np.abs(g - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -20 * mag).all()
    assert (g[mag == 0] == out[mag == 0]).all()  # the rest of a head is copied


POSITIONS = [0, 1, -1, 7, 4095, 131071, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 12345678]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,r", [(1, 1, 1, 32, 16), (1, 24, 4, 256, 64), (3, 32, 8, 128, 128), (10, 6, 1, 256, 256),
                                          (10, 5, 0, 80, 48), (2, 7, 3, 96, 96), (2, 1, 1, 1024, 1024), (130, 48, 4, 256, 112),
                                          (10, 8, 8, 64, 32)])
def test_rows(n, hq, hkv, d, r, inter):
    gen = torch.Generator().manual_seed(n * 31 + d)
    pos = [POSITIONS[i % len(POSITIONS)] for i in range(n)]
    freqs, _ = pa.rotary_frequencies(r, base=1e6)
    q, k = rows(gen, n, hq, d), rows(gen, n, hkv, d) if hkv else None
    q0, k0 = q.clone(), k.clone() if hkv else None
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for inverse in (False, True):
        q_out, k_out = torch.full_like(q, float("nan")), torch.full_like(k, float("nan")) if hkv else None
        pa.rotary(q, k, p, freqs, q_out, k_out, interleaved=inter, inverse=inverse, factor=1.25)
        check(q_out, reference(q, pos, freqs, inter, 1.25, inverse))
        if hkv:
            check(k_out, reference(k, pos, freqs, inter, 1.25, inverse))
    # in place, the same bits; inputs of the calls before untouched
    assert torch.equal(q, q0)
    pa.rotary(q, k, p, freqs, q, k, interleaved=inter, inverse=True, factor=1.25)
    assert torch.equal(q, q_out) and (not hkv or torch.equal(k, k_out) and not torch.equal(k, k0) or n == 1)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    """The inverse rotation of an output's gradient is the gradient of the rows: against differences of the rotation
    in 64 bits along random directions."""
    gen = torch.Generator().manual_seed(5)
    freqs, _ = pa.rotary_frequencies(64)
    pos = [3, 70, 1000]
    g, x, e = rows(gen, 3, 4, 128), rows(gen, 3, 4, 128), rows(gen, 3, 4, 128)
    got = torch.empty_like(g)
    pa.rotary(g, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), freqs, got, None, interleaved=inter,
              inverse=True, factor=1.5)
    up, _ = reference(x.double() + e.double(), pos, freqs, inter, 1.5, False)  # (linear: a whole step is exact)
    down, _ = reference(x.double() - e.double(), pos, freqs, inter, 1.5, False)
    want = (g.cpu().double().numpy() * (up - down) / 2).sum()
    terms = np.abs(got.cpu().double().numpy() * e.cpu().double().numpy()).sum()
    assert abs((got.double() * e.double()).sum().item() - want) <= 2.0 ** -8 * terms * 1.01


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n,hq,hkv,d,r,bs", [(1, 24, 4, 256, 64, 784), (37, 32, 8, 128, 128, 16), (200, 6, 1, 256, 112, 48),
                                             (64, 4, 2, 128, 16, 832)])
def test_cache_equals_the_two_calls(n, hq, hkv, d, r, bs, kind, inter):
    gen = torch.Generator().manual_seed(n + d + r)
    pages = n // bs + 2
    freqs, factor = pa.rotary_frequencies(r, scaling="yarn", factor=4.0, original_len=4096)
    buf = rows(gen, n, hq + 2 * hkv, d)  # rows of one projection, read in place
    q, k, v = buf[:, :hq], buf[:, hq:hq + hkv], buf[:, hq + hkv:]
    slots = torch.randperm(pages * bs, generator=gen)[:n]
    if n > 4:
        slots[2], slots[n - 1] = -1, pages * bs + 3  # a padding token, a slot past the cache
    slots = slots.cuda()
    lens = torch.randint(1, 100000, (n,), generator=gen).int().cuda()
    kg, vg = torch.rand(hkv, generator=gen).cuda() + 0.05, torch.rand(hkv, generator=gen).cuda() + 0.05
    shape = pa.fp4_cache_shape(pages, bs, hkv, d) if kind == "fp4" else (pages, bs, hkv, d)
    caches = [torch.randint(0, 120, shape, generator=gen).to(torch.uint8).cuda() for _ in range(2)]
    if kind == "bf16":
        caches = [c.to(torch.bfloat16) for c in caches]
    got, want = [c.clone() for c in caches], [c.clone() for c in caches]
    status, status2 = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, q_ref, k_ref = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty_like(q), torch.empty_like(k)
    opts = dict(interleaved=inter, factor=factor, position_offset=-1)
    scales = () if kind == "bf16" else (kg, vg)
    suffix = "" if kind == "bf16" else "_" + kind
    getattr(pa, "rotary_and_cache" + suffix)(q, k, v, lens, freqs, q_out, *got, slots, *scales, status=status, **opts)
    pa.rotary(q, k, lens, freqs, q_ref, k_ref, **opts)
    getattr(pa, "reshape_and_cache" + suffix)(k_ref, v.contiguous(), *want, slots, *scales, status=status2)
    assert torch.equal(q_out, q_ref)
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
    assert int(status) == int(status2) == (pa.PA_DEV_BAD_SLOT if n > 4 else 0)
    check(q_out, reference(q, lens.cpu().numpy() - 1, freqs, inter, factor, False))
    # q turned in place in the projection's rows, k and v beside it as before
    kv = buf[:, hq:].clone()
    getattr(pa, "rotary_and_cache" + suffix)(q, k, v, lens, freqs, q, *got, slots, *scales, **opts)
    assert torch.equal(q, q_ref) and torch.equal(buf[:, hq:], kv)


def test_one_row_of_k_for_every_token():
    """An expanded row (stride 0) is read as any other."""
    gen = torch.Generator().manual_seed(9)
    freqs, _ = pa.rotary_frequencies(32)
    q = rows(gen, 1, 2, 64).expand(20, 2, 64)
    out, pos = torch.empty((20, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.arange(20, device="cuda").int()
    pa.rotary(q, None, pos, freqs, out, None)
    check(out, reference(q, range(20), freqs, False, 1.0, False))


def test_values_that_are_not_finite_stay_in_their_pair():
    freqs, _ = pa.rotary_frequencies(64)
    q = torch.ones((1, 3, 128), dtype=torch.bfloat16, device="cuda")
    q[0, 1, 5], q[0, 1, 100] = float("nan"), float("inf")
    out = torch.empty_like(q)
    pa.rotary(q, None, torch.tensor([17], dtype=torch.int32, device="cuda"), freqs, out, None)
    bad = ~torch.isfinite(out)
    assert bad[0, 1].nonzero().flatten().tolist() == [5, 37, 100] and not bad[0, 0].any() and not bad[0, 2].any()
    assert out[0, 1, 100] == float("inf")


def test_no_rows():
    freqs, _ = pa.rotary_frequencies(32)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    pa.rotary(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), freqs, q, None)


def test_stream_and_graph():
    """On a stream of its own and as a replayed graph, behind a kernel that makes its input."""
    gen = torch.Generator().manual_seed(2)
    freqs, _ = pa.rotary_frequencies(128)
    src, q, out = rows(gen, 50, 32, 128), torch.empty((50, 32, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((50, 32, 128), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(1000, 1050, device="cuda").int()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q.copy_(src)
        pa.rotary(q, None, pos, freqs, out, None)
    s.synchronize()
    want = reference(src, range(1000, 1050), freqs, False, 1.0, False)
    check(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.copy_(src)
        pa.rotary(q, None, pos, freqs, out, None)
    for k in range(3):
        pos.add_(1000)
        src.neg_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        first = 1000 * (k + 2)
        check(out, reference(src, range(first, first + 50), freqs, False, 1.0, False))
