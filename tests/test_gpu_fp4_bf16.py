"""bf16 outputs over an fp4 cache: these are kernels of their own (the weights
enter the second product as one f16), at the shapes, masks and values where the
fp32 ones are tested.

Tolerance: that of fp32 outputs (fp4_ref.tolerance, fp4_ref.vanished), half a
step of the bf16 output (in fp4_ref.tolerance), and half a step of f16, 2^-11,
for each weight: 2^-11 of the sum of |weight v| at most."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import fp4_ref as ref
from tests.test_gpu_fp4 import Problem

pytestmark = pytest.mark.gpu

BF16 = dict(out_dtype=pa.PA_OUT_BF16)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def check(p, runs, window=0):
    args = (p.q.float().numpy(), p.k, p.v, p.g, p.table, p.lens, p.scale, p.q_len, window)
    with np.errstate(invalid="ignore"):
        want, mag, reach = ref.attention(*args)
        off = ref.vanished(*args)
    mag, reach, off = (np.where(np.isfinite(x), x, 0.0) for x in (mag, reach, off))
    tol = ref.tolerance(mag, reach, p.d, max(p.lens), True, want) + off + 2.0 ** -11 * mag
    live = np.isfinite(want)
    for kw in runs:
        out, status = p.run(window=window, **BF16, **kw)
        assert status == 0
        assert np.array_equal(np.isnan(out), ~live)
        worst = (np.abs(out - want)[live] / tol[live]).max()
        assert worst <= 1, (kw, worst)


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("gap", [6, 14, 20])
@pytest.mark.parametrize("hq,hkv,d", [(6, 1, 256), (16, 1, 256), (4, 2, 128), (24, 2, 128)])
def test_small_weights_and_small_scales(hq, hkv, d, gap, q_len):
    """A first key that takes nearly all of the weight and has no value, beside
    keys with 2^-gap of its weight whose block scales are 2^-9 to 2^-4: their
    sum is the output."""
    p = Problem(gap + d + q_len, [600, 90], hq, hkv, d, 16, q_len=q_len)
    rng = np.random.default_rng(gap)
    p.q = torch.from_numpy(1 + 0.1 * rng.standard_normal(p.q.shape).astype(np.float32)).to(torch.bfloat16)
    for b, n in enumerate(p.lens):
        first = [int(p.table[b, 0]) * 16]
        ref.write_rows("k", np.full((1, hkv, d), gap * np.log(2) / np.sqrt(d), np.float32), p.g[0], p.k, first)
        ref.write_rows("v", np.zeros((1, hkv, d), np.float32), p.g[1], p.v, first)
        for t in range(1, n):
            places = ref.byte_places("v", t % 16, d)[1]
            p.v[p.table[b, t // 16], :, 0, places] = rng.integers(1, 0x19, (len(places), hkv))
    check(p, (dict(num_splits=1), dict()))


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200]


@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (6, 2), (4, 1), (10, 2), (18, 3), (16, 2), (36, 3), (32, 2)])
@pytest.mark.parametrize("d", [128, 256])
def test_decode_groups_and_tails(hq, hkv, d):
    check(Problem(hq * 100 + d + 1, LENS, hq, hkv, d, 48),
          (dict(), dict(num_splits=1), dict(num_splits=3, flags=pa.PA_FLAG_EARLY_KV_READ)))


def hide_before(p, window):
    """NaN scales in the rows before the window, as in a page given away."""
    for b, n in enumerate(p.lens):
        for t in range(max(0, n - p.q_len + 1 - window)):
            for kind, c in (("k", p.k), ("v", p.v)):
                c[p.table[b, t // 16]][:, 0, np.concatenate(ref.byte_places(kind, t % 16, p.d))] = 0xFF


@pytest.mark.parametrize("window", [1, 17, 100])
@pytest.mark.parametrize("hq,hkv,d,q_len", [(18, 3, 128, 1), (24, 2, 256, 1), (12, 2, 128, 9), (6, 1, 256, 30)])
def test_windows(hq, hkv, d, q_len, window):
    p = Problem(window + d + q_len, [q_len, 16 + q_len, 100, 333], hq, hkv, d, 16, q_len=q_len)
    hide_before(p, window)
    check(p, (dict(), dict(num_splits=1), dict(flags=pa.PA_FLAG_EARLY_KV_READ)), window)


@pytest.mark.parametrize("hq,hkv,d,splits,flags", [(16, 2, 256, 0, 0), (24, 2, 256, 1, 1), (16, 2, 128, 3, 1),
                                                   (32, 2, 128, 0, 0)])
def test_append_is_the_write_then_the_decode(hq, hkv, d, splits, flags):
    rng = np.random.default_rng(d + hq)
    p = Problem(d + hq, [0, 1, 16, 17, 400, 33], hq, hkv, d, 16)
    k_new, v_new = (torch.from_numpy(rng.standard_normal((6, hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda()
                    for _ in range(2))
    slots = torch.tensor([-1 if n == 0 else int(p.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16
                          for b, n in enumerate(p.lens)]).cuda()
    desc = p.desc(num_splits=splits, flags=flags, **BF16)
    ws = torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
    res = []
    for fused in (False, True):
        q, kc, vc, ks, vs, bt, sl = p.tensors()
        out = torch.full(p.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        if fused:
            pa.paged_attention_decode_append_fp4(q, k_new, v_new, kc, vc, ks, vs, bt, sl, desc, out, ws)
        else:
            pa.reshape_and_cache_fp4(k_new, v_new, kc, vc, slots, ks, vs)
            torch.cuda.synchronize()  # (the early read is told that the rows before the new one are there)
            pa.paged_attention_decode_fp4(q, kc, vc, ks, vs, bt, sl, desc, out, ws)
        res.append((out, kc, vc))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    p.k, p.v = res[1][1].cpu().numpy(), res[1][2].cpu().numpy()
    check(p, (dict(num_splits=splits),))


@pytest.mark.parametrize("hq,hkv,d,q_len,lens", [
    (24, 4, 256, 16, [16, 17, 80, 333]),     # one 96-row block
    (48, 4, 256, 5, [5, 70, 700]),           # 12 heads per KV head
    (8, 8, 128, 2, [2, 3, 64, 65, 129]),     # two live rows
    (14, 2, 128, 5, [5, 70, 200]),           # 7 heads per KV head
    (24, 2, 256, 11, [11, 64, 127]),         # 132 rows: a second block of 4
    (6, 1, 128, 60, [60, 100, 190]),         # three blocks
])
def test_verify_shapes(hq, hkv, d, q_len, lens):
    check(Problem(q_len + 7, lens, hq, hkv, d, 48, q_len=q_len),
          (dict(), dict(num_splits=1), dict(num_splits=2, flags=pa.PA_FLAG_EARLY_KV_READ)))


@pytest.mark.parametrize("hq,hkv,d,q_len,lens,window", [
    (6, 1, 256, 4, [1500, 700, 4], 0), (24, 2, 256, 11, [900, 11], 0), (8, 8, 128, 3, [1100, 333], 500),
    (6, 1, 256, 1, [4600, 3100], 0), (8, 1, 128, 1, [6000], 0), (16, 1, 128, 1, [4000], 3900), (12, 1, 256, 1, [1000], 0)])
def test_growing_scores_and_large_scales(hq, hkv, d, q_len, lens, window):
    """Keys that grow along the sequence, so that the reference max rises again
    and again, and V blocks whose scales are 1 to 448."""
    rng = np.random.default_rng(q_len + window)
    p = Problem(q_len + window + 3, lens, hq, hkv, d, 16, q_len=q_len)
    for b, n in enumerate(lens):
        for t in range(n):
            p.k[p.table[b, t // 16]][:, 0, ref.byte_places("k", t % 16, d)[1]] = 0x30 + t * 64 // n
            places = ref.byte_places("v", t % 16, d)[1]
            p.v[p.table[b, t // 16], :, 0, places] = rng.integers(0x38, 0x7F, (len(places), hkv))
    check(p, (dict(num_splits=1), dict(num_splits=2, flags=pa.PA_FLAG_EARLY_KV_READ)), window)


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("d,q_len,hq,hkv,window", [(128, 1, 12, 2, 0), (256, 1, 24, 2, 30), (128, 9, 12, 2, 0),
                                                   (256, 60, 6, 1, 0), (128, 30, 8, 2, 7), (256, 40, 4, 4, 25)])
def test_nan_scales_reach_the_rows_that_see_them(what, d, q_len, hq, hkv, window):
    p = Problem(q_len + window + 5, [q_len, 100, 203], hq, hkv, d, 16, q_len=q_len)
    cache = p.k if what == "k" else p.v
    for b, n in enumerate(p.lens):
        for i, blk in ((q_len // 2, 1), (q_len - 1, 0), (q_len // 3, 5)):
            t = n - q_len + i
            cache[p.table[b, t // 16], i % hkv, 0, ref.byte_places(what, t % 16, d)[1][blk]] = 0x7F
    if window:  # a row that the first rows see and the last ones do not
        t = 203 - q_len - window + 4
        cache[p.table[2, t // 16], 0, 0, ref.byte_places(what, t % 16, d)[1][3]] = 0xFF
    check(p, (dict(), dict(num_splits=1), dict(num_splits=3, flags=pa.PA_FLAG_EARLY_KV_READ)), window)


@pytest.mark.parametrize("q_len", [1, 4])
def test_bad_pages_and_lengths_give_zero_rows(q_len):
    p = Problem(12, [100, 50, 80], 8, 2, 128, 16, q_len=q_len)
    for splits in (1, 3):
        want = p.run(num_splits=splits, **BF16)[0]
        good = np.r_[0:q_len, 2 * q_len:3 * q_len]
        for k, bad, bits in ((5, None, pa.PA_DEV_BAD_PAGE), (6, [100, p.max_len + 1, 80], pa.PA_DEV_BAD_SEQLEN)):
            t = list(p.tensors())
            if bad is None:
                t[5][1, 2] = p.pages  # outside the pool
            else:
                t[6] = torch.tensor(bad, dtype=torch.int32, device="cuda")
            out, status = p.run(t, num_splits=splits, **BF16)
            assert status == bits
            assert (out[q_len:2 * q_len] == 0).all() and np.array_equal(out[good], want[good])


@pytest.mark.parametrize("hq,hkv,d,q_len,length", [
    (6, 1, 256, 1, 49189), (16, 1, 256, 1, 40000), (8, 1, 128, 1, 60000), (16, 1, 128, 1, 131072), (6, 1, 256, 4, 20011),
    (8, 1, 128, 16, 131072)])
def test_long_unsplit_contexts(hq, hkv, d, q_len, length):
    """Against float64 over the rows read back.  An output may be off by half a
    step of bf16, 2^-8 of itself, and by the weights' half step of f16 and one
    step of binary32 for each 16-key product, of the sum of |weight v|."""
    rng = np.random.default_rng(length)
    bs, pages = 784, -(-length // 784)
    g = [ref.cuda(x) for x in ref.head_scales(hkv)]
    cache = [torch.zeros(pa.fp4_cache_shape(pages, bs, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows = [torch.from_numpy(rng.standard_normal((length, hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda()
            for _ in range(2)]
    slots = torch.arange(length, device="cuda")
    pa.reshape_and_cache_fp4(*rows, *cache, slots, *g)
    k, v = (torch.empty((length, hkv, d), device="cuda") for _ in range(2))
    pa.gather_cache_fp4(*cache, slots, *g, k, v)
    q = torch.from_numpy(rng.standard_normal((q_len, hq, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    desc = pa.make_desc(num_seqs=1, q_len=q_len, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                        max_pages_per_seq=pages, max_seq_len=length, num_pages=pages, scale=d ** -0.5, num_splits=1,
                        **BF16)
    out = torch.empty((q_len, hq, d), dtype=torch.bfloat16, device="cuda")
    call = pa.paged_attention_decode_fp4 if q_len == 1 else pa.paged_attention_verify_fp4
    call(q, *cache, *g, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
         torch.tensor([length], dtype=torch.int32, device="cuda"), desc, out,
         torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda"))
    x = torch.einsum("qhd,td->qht", q.double(), k[:, 0].double()) * d ** -0.5
    hidden = torch.arange(length, device="cuda") > length - q_len + torch.arange(q_len, device="cuda")[:, None]
    w = x.masked_fill(hidden[:, None], -torch.inf).softmax(-1)
    want, mag = w @ v[:, 0].double(), w @ v[:, 0].double().abs()
    reach = (q.double().abs() @ k[:, 0].double().abs().T).amax(-1) * d ** -0.5
    tol = (want.abs() * 2.0 ** -8 + 2.0 ** -11 * mag
           + mag * (2.02 * (d + 4) * 2.0 ** -23 * reach[..., None] + 2 * 2.0 ** -21 + (length / 16 + 64) * 2.0 ** -23))
    assert ((out.double() - want).abs() <= tol).all()
