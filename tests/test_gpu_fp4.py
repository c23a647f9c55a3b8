"""GPU parity of the fp4 KV cache: reshape_and_cache_fp4 and gather_cache_fp4
bit for bit against the format's definition; decode, append and verify against
float64 attention over the same bytes, within a tolerance counted from the
roundings (fp4_ref.tolerance)."""
import math

import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def bf16_rows(rng, n, hkv, d):
    return torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32)).to(torch.bfloat16)


# -- writing and reading rows ---------------------------------------------------------------------

def special_rows(rng, n, hkv, d):
    """Rows with zeros, ties of both rounding steps, tiny and huge values,
    infinities and a NaN in some blocks."""
    x = rng.standard_normal((n, hkv, d)).astype(np.float32)
    x[0, :, :16] = 0.0
    x[0, :, 16:32] = -0.0
    x[1, :, :16] = [6, 0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5, 0.5, 1, -1.5, 2, 3, -4, -6, 0]
    x[2, :, :16] *= 1e-30
    x[3, :, 16:32] *= 1e30
    x[4, :, 3] = np.inf
    x[5, :, 20] = -np.inf
    x[6, 0, 40] = np.nan
    x[7, :, 64:80] *= 2.0 ** -8  # subnormal scales
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("hkv,d,bs", [(4, 256, 16), (8, 128, 48), (1, 128, 784), (3, 256, 32)])
def test_reshape_and_cache_fp4_bit_exact(hkv, d, bs):
    rng = np.random.default_rng(hkv * d + bs)
    pages, n = 5, 37
    k_new, v_new = special_rows(rng, n, hkv, d), special_rows(rng, n, hkv, d)
    g = ref.head_scales(hkv)
    if hkv == 4:  # ties need an exact scale
        g = tuple(np.full(hkv, 1 / 64, np.float32) for _ in range(2))
    slots = rng.permutation(pages * bs)[:n].astype(np.int64)
    slots[[9, 20]] = -1
    slots[30] = pages * bs + 3
    k_ref = rng.integers(0, 256, (pages, hkv, bs // 16, 9 * d), dtype=np.uint8)  # bytes that must stay
    v_ref = k_ref[::-1].copy()
    kc, vc = ref.cuda(k_ref), ref.cuda(v_ref)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert tuple(kc.shape) == pa.fp4_cache_shape(pages, bs, hkv, d)
    pa.reshape_and_cache_fp4(k_new.cuda(), v_new.cuda(), kc, vc, ref.cuda(slots), ref.cuda(g[0]), ref.cuda(g[1]), status)
    ref.write_rows("k", k_new.float().numpy(), g[0], k_ref, slots)
    ref.write_rows("v", v_new.float().numpy(), g[1], v_ref, slots)
    assert np.array_equal(kc.cpu().numpy(), k_ref)
    assert np.array_equal(vc.cpu().numpy(), v_ref)
    assert status.item() == pa.PA_DEV_BAD_SLOT


@pytest.mark.parametrize("hkv,d,bs,dtype", [(4, 256, 16, torch.float32), (8, 128, 48, torch.bfloat16),
                                            (1, 256, 784, torch.bfloat16)])
def test_gather_cache_fp4_bit_exact(hkv, d, bs, dtype):
    rng = np.random.default_rng(7 * d + bs)
    pages, n = 4, 50
    cache = [rng.integers(0, 256, (pages, hkv, bs // 16, 9 * d), dtype=np.uint8) for _ in range(2)]  # NaN scales too
    g = ref.head_scales(hkv)
    slots = rng.integers(0, pages * bs, n)  # a row may be read twice
    slots[[3, 17]] = -1
    slots[11] = pages * bs
    out = [torch.full((n, hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.gather_cache_fp4(ref.cuda(cache[0]), ref.cuda(cache[1]), ref.cuda(slots), ref.cuda(g[0]), ref.cuda(g[1]),
                        out[0], out[1], status)
    for kind, c, scale, o in zip("kv", cache, g, out):
        want = ref.read_rows(kind, c, slots)
        want = torch.from_numpy(want.astype(np.float32)) * torch.from_numpy(scale)[:, None]  # one rounding
        want = want.to(dtype).float().numpy()
        assert np.array_equal(o.float().cpu().numpy(), want, equal_nan=True)
    assert status.item() == pa.PA_DEV_BAD_SLOT


def test_rows_written_and_read_back_are_near_what_went_in():
    """What the format keeps: a code is within 1/6 of the block's largest value
    (half the step 4 .. 6, a sixth of the scale's rounding beside it)."""
    rng = np.random.default_rng(3)
    x = bf16_rows(rng, 64, 4, 256)
    g = [torch.full((4,), 1 / 64, device="cuda") for _ in range(2)]
    cache = [torch.zeros(pa.fp4_cache_shape(4, 16, 4, 256), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.randperm(64).cuda()
    pa.reshape_and_cache_fp4(x.cuda(), x.cuda(), *cache, slots, *g)
    out = [torch.empty((64, 4, 256), device="cuda") for _ in range(2)]
    pa.gather_cache_fp4(*cache, slots, *g, *out)
    assert torch.equal(out[0], out[1])
    off = (out[0].cpu() - x.float()).abs().unflatten(-1, (-1, 16)).amax(-1)
    top = x.float().abs().unflatten(-1, (-1, 16)).amax(-1)
    # a code is off by at most one (half the widest step, and saturation), S by 1/16 of itself
    assert (off <= top * (1 / 6 + 1 / 16) * (1 + 1 / 16)).all()


# -- attention ------------------------------------------------------------------------------------

class Problem:
    def __init__(self, seed, lens, hq, hkv, d, bs, q_len=1, max_len=None, pool=None):
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.bs, self.q_len = list(lens), hq, hkv, d, bs, q_len
        self.width = max(1, -(-(max_len or max(lens)) // bs))
        used = [-(-n // bs) for n in lens]
        self.pages = pool or sum(used) + 2
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.g = ref.head_scales(hkv)
        self.k, self.v = ref.random_cache(rng, self.pages, bs, hkv, d, self.g)
        # what no sequence uses: every byte 0xFF (NaN scales)
        live = np.zeros(self.pages * bs, bool)
        for b, n in enumerate(lens):
            live[ref.slots_of(self.table[b], n, bs)] = True
        for kind, c in (("k", self.k), ("v", self.v)):
            for t in range(16):
                places = np.concatenate(ref.byte_places(kind, t, d))
                dead = ~live.reshape(self.pages, bs // 16, 16)[:, :, t]
                rows = c[..., places]
                rows[np.broadcast_to(dead[:, None, :], rows.shape[:3])] = 0xFF
                c[..., places] = rows
        self.q = torch.from_numpy(rng.standard_normal((len(lens) * q_len, hq, d)).astype(np.float32)).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(d)
        self.max_len = max_len or max(lens)

    def desc(self, **kw):
        return pa.make_desc(num_seqs=len(self.lens), q_len=self.q_len, num_q_heads=self.hq, num_kv_heads=self.hkv,
                            head_dim=self.d, block_size=self.bs, max_pages_per_seq=self.width,
                            max_seq_len=self.max_len, num_pages=self.pages, scale=self.scale, **kw)

    def tensors(self):
        return (self.q.cuda(), ref.cuda(self.k), ref.cuda(self.v), ref.cuda(self.g[0]), ref.cuda(self.g[1]),
                ref.cuda(self.table), torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def run(self, tensors=None, **kw):
        desc = self.desc(**kw)
        ws = torch.full((max(1, pa.workspace_bytes(desc)),), 0xFF, dtype=torch.uint8, device="cuda")
        bf = desc.out_dtype == pa.PA_OUT_BF16
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16 if bf else torch.float32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call = pa.paged_attention_decode_fp4 if self.q_len == 1 else pa.paged_attention_verify_fp4
        call(*(tensors or self.tensors()), desc, out, ws, status)
        return out.float().cpu().double().numpy(), int(status.item())

    def check(self, out, window=0, bf=False):
        want, mag, reach = ref.attention(self.q.float().numpy(), self.k, self.v, self.g, self.table, self.lens,
                                         self.scale, self.q_len, window)
        tol = ref.tolerance(mag, reach, self.d, max(self.lens), bf, want)
        assert np.isfinite(out).all()
        worst = (np.abs(out - want) / tol).max()
        assert worst <= 1, worst
        if not bf:  # the error of a sum of roundings is far below their bound: 2^-13 overall
            assert np.linalg.norm(out - want) <= 2.0 ** -13 * max(np.linalg.norm(want), 1e-30)
        empty = np.array(self.lens).repeat(self.q_len) == 0
        assert (out[empty] == 0).all()


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200]


@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (6, 2), (4, 1), (10, 2), (18, 3), (16, 2), (36, 3), (32, 2)])
@pytest.mark.parametrize("d", [128, 256])
def test_decode_groups_and_tails(hq, hkv, d):
    p = Problem(hq * 100 + d, LENS, hq, hkv, d, 48)
    for kw in (dict(), dict(num_splits=1), dict(num_splits=3)):
        out, status = p.run(**kw)
        assert status == 0
        p.check(out)


@pytest.mark.parametrize("bs", [16, 784, 832])
@pytest.mark.parametrize("bf", [False, True])
def test_decode_page_sizes_and_output_types(bs, bf):
    p = Problem(bs, [783, 784, 785, 831, 833, 1700], 24, 4, 256, bs, max_len=3000)
    for flags in (0, pa.PA_FLAG_EARLY_KV_READ):
        out, status = p.run(out_dtype=pa.PA_OUT_BF16 if bf else pa.PA_OUT_F32, flags=flags)
        assert status == 0
        p.check(out, bf=bf)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 5000])
@pytest.mark.parametrize("d", [128, 256])
def test_decode_window_with_nan_before_it(window, d):
    p = Problem(window, [5, 16, 100, 333, 0], 18, 3, d, 16)
    for b, n in enumerate(p.lens):  # rows before the window: NaN scales, as in a page given away
        for t in range(max(0, n - window)):
            page, pos = p.table[b, t // 16], t % 16
            for kind, c in (("k", p.k), ("v", p.v)):
                c[page][:, 0, np.concatenate(ref.byte_places(kind, pos, d))] = 0xFF
    for kw in (dict(), dict(num_splits=1), dict(flags=pa.PA_FLAG_EARLY_KV_READ)):
        out, status = p.run(window=window, **kw)
        assert status == 0
        p.check(out, window=window)


@pytest.mark.parametrize("d,splits,flags", [(256, 0, 0), (256, 1, 1), (128, 0, 1), (128, 3, 0)])
def test_append_is_the_write_then_the_decode(d, splits, flags):
    rng = np.random.default_rng(d + splits)
    p = Problem(d, [0, 1, 16, 17, 400, 33], 16, 2, d, 16)
    k_new, v_new = (bf16_rows(rng, 6, 2, d).cuda() for _ in range(2))
    slots = torch.tensor([-1 if n == 0 else int(p.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16
                          for b, n in enumerate(p.lens)]).cuda()
    desc = p.desc(num_splits=splits, flags=flags)
    ws = torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
    res = []
    for fused in (False, True):
        q, kc, vc, ks, vs, bt, sl = p.tensors()
        out = torch.full(p.q.shape, float("nan"), device="cuda")
        if fused:
            pa.paged_attention_decode_append_fp4(q, k_new, v_new, kc, vc, ks, vs, bt, sl, desc, out, ws)
        else:
            pa.reshape_and_cache_fp4(k_new, v_new, kc, vc, slots, ks, vs)
            pa.paged_attention_decode_fp4(q, kc, vc, ks, vs, bt, sl, desc, out, ws)
        res.append((out, kc, vc))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    p.k, p.v = res[1][1].cpu().numpy(), res[1][2].cpu().numpy()
    p.check(res[1][0].double().cpu().numpy())


@pytest.mark.parametrize("hq,hkv,d,q_len,lens", [
    (24, 4, 256, 16, [16, 17, 80, 333]),     # one 96-row block
    (8, 8, 128, 2, [2, 3, 64, 65, 129]),     # two live rows
    (14, 2, 128, 5, [5, 70, 200]),           # 7 heads per KV head
    (24, 2, 256, 11, [11, 64, 127]),         # 132 rows: a second block of 4
    (6, 1, 128, 60, [60, 100, 190]),         # three blocks
])
def test_verify_shapes(hq, hkv, d, q_len, lens):
    p = Problem(q_len, lens, hq, hkv, d, 48, q_len=q_len)
    for kw in (dict(), dict(num_splits=1), dict(num_splits=2, flags=pa.PA_FLAG_EARLY_KV_READ)):
        out, status = p.run(**kw)
        assert status == 0
        p.check(out)


@pytest.mark.parametrize("bs", [16, 64, 784])
@pytest.mark.parametrize("bf", [False, True])
def test_verify_page_sizes_and_output_types(bs, bf):
    p = Problem(bs + 1, [790, 1000, 47], 24, 4, 256, bs, q_len=4, max_len=2000)
    out, status = p.run(out_dtype=pa.PA_OUT_BF16 if bf else pa.PA_OUT_F32)
    assert status == 0
    p.check(out, bf=bf)


@pytest.mark.parametrize("window", [1, 7, 64, 100])
def test_verify_window(window):
    p = Problem(window + 50, [9, 65, 300], 12, 2, 128, 16, q_len=9)
    out, status = p.run(window=window)
    assert status == 0
    p.check(out, window=window)


def test_large_scores_and_rescaling():
    """Keys that grow along the sequence: every chunk raises the reference max."""
    for q_len in (1, 3):
        p = Problem(5, [300, 77], 8, 2, 128, 16, q_len=q_len)
        for b, n in enumerate(p.lens):
            for t in range(n):
                places = ref.byte_places("k", t % 16, 128)[1]
                p.k[p.table[b, t // 16]][:, 0, places] = 0x28 + min(70, t // 4)  # block scales that only grow
        out, status = p.run()
        assert status == 0
        p.check(out)


@pytest.mark.parametrize("q_len", [1, 4])
def test_bad_pages_and_lengths_give_zero_rows(q_len):
    p = Problem(11, [100, 50, 80], 8, 2, 128, 16, q_len=q_len)
    for splits in (1, 3):
        t = list(p.tensors())
        t[5] = t[5].clone()
        t[5][1, 2] = p.pages  # outside the pool
        out, status = p.run(t, num_splits=splits)
        assert status == pa.PA_DEV_BAD_PAGE
        assert (out[q_len:2 * q_len] == 0).all()
        good = np.r_[0:q_len, 2 * q_len:3 * q_len]
        want = p.run(num_splits=splits)[0]
        assert np.array_equal(out[good], want[good])
        t = list(p.tensors())
        t[6] = torch.tensor([100, p.max_len + 1, 80], dtype=torch.int32, device="cuda")
        out, status = p.run(t, num_splits=splits)
        assert status == pa.PA_DEV_BAD_SEQLEN
        assert (out[q_len:2 * q_len] == 0).all() and np.array_equal(out[good], want[good])


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_visible_nan_shows_and_stays_in_its_head(what, splits, q_len):
    p = Problem(21, [90, 40], 8, 2, 128, 16, q_len=q_len)
    cache = p.k if what == "k" else p.v
    cache[p.table[0, 1], 0, 0, ref.byte_places(what, 3, 128)[1][2]] = 0x7F  # token 19, block 2, KV head 0
    out, status = p.run(num_splits=splits)
    assert status == 0
    hit = out[:q_len, :4]
    assert np.isnan(hit if what == "k" else hit[..., 32:48]).all()
    assert np.isfinite(out[:q_len, 4:]).all() and np.isfinite(out[q_len:]).all()


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("d,q_len,hq,hkv,window", [(128, 9, 12, 2, 0), (256, 60, 6, 1, 0), (128, 30, 8, 2, 7),
                                                   (256, 40, 4, 4, 25)])
def test_verify_rows_that_do_not_see_a_nan_stay_finite(what, d, q_len, hq, hkv, window):
    """NaN scales in new rows that earlier rows do not see, and with a window in
    rows that later rows do not see: the same rows and dims are NaN as by the formula."""
    p = Problem(q_len + window, [q_len, 100, 203], hq, hkv, d, 16, q_len=q_len)
    cache = p.k if what == "k" else p.v
    for b, n in enumerate(p.lens):
        for i, blk in ((q_len // 2, 1), (q_len - 1, 0), (q_len // 3, 5)):
            t = n - q_len + i
            cache[p.table[b, t // 16], i % hkv, 0, ref.byte_places(what, t % 16, d)[1][blk]] = 0x7F
    if window:  # a row that the first rows see and the last ones do not
        t = 203 - q_len - window + 4
        cache[p.table[2, t // 16], 0, 0, ref.byte_places(what, t % 16, d)[1][3]] = 0xFF
    want, mag, reach = ref.attention(p.q.float().numpy(), p.k, p.v, p.g, p.table, p.lens, p.scale, q_len, window)
    clean = [np.where(np.isnan(x), 0.0, x) for x in (mag, reach)]
    tol = ref.tolerance(*clean, d, max(p.lens), False, want)
    assert np.isnan(want).any() and np.isfinite(want).any()
    for kw in (dict(), dict(num_splits=1), dict(num_splits=3, flags=pa.PA_FLAG_EARLY_KV_READ)):
        out, status = p.run(window=window, **kw)
        assert status == 0
        assert np.array_equal(np.isnan(out), np.isnan(want))
        assert (np.abs(out - want) <= tol)[np.isfinite(want)].all()


@pytest.mark.parametrize("hq,hkv,d,q_len,lens,window", [
    (6, 1, 256, 4, [1500, 700, 4], 0),    # 24 rows: one warp, not all of it live
    (24, 2, 256, 11, [900, 11], 0),       # 132 rows: a full block and one of 4 rows
    (8, 8, 128, 3, [1100, 333], 500),
    (12, 2, 128, 16, [1303], 0),          # 96 rows
    (6, 1, 256, 1, [4600, 3100], 0), (8, 1, 128, 1, [6000], 0), (16, 1, 128, 1, [4000], 3900)])
def test_second_sum_with_growing_scores(hq, hkv, d, q_len, lens, window):
    """fp32 outputs whose accumulators move to a second sum, with keys that grow
    along the sequence, so that the reference max rises again and again."""
    p = Problem(q_len + window, lens, hq, hkv, d, 16, q_len=q_len)
    for b, n in enumerate(lens):
        for t in range(n):
            p.k[p.table[b, t // 16]][:, 0, ref.byte_places("k", t % 16, d)[1]] = 0x30 + t * 64 // n
    args = (p.q.float().numpy(), p.k, p.v, p.g, p.table, p.lens, p.scale, q_len, window)
    want, mag, reach = ref.attention(*args)
    tol = ref.tolerance(mag, reach, d, max(lens), False, want) + ref.vanished(*args)
    for kw in (dict(num_splits=1), dict(num_splits=2, flags=pa.PA_FLAG_EARLY_KV_READ)):
        out, status = p.run(window=window, **kw)
        assert status == 0
        assert (np.abs(out - want) <= tol).all()
        assert np.linalg.norm(out - want) <= 2.0 ** -18 * np.linalg.norm(want)


@pytest.mark.parametrize("hq,hkv,d,q_len,length", [
    (6, 1, 256, 1, 49189), (4, 1, 256, 1, 33000), (16, 1, 256, 1, 40000), (8, 1, 128, 1, 60000),
    (16, 1, 128, 1, 40000), (6, 1, 256, 4, 20011), (8, 1, 128, 16, 40000)])
def test_fp32_outputs_of_long_unsplit_contexts(hq, hkv, d, q_len, length):
    """Against float64 over the rows read back.  The tensor core cuts additions
    off towards zero: half a step, 2^-24 of at most 17 x 64 / 16 x 2 growing
    sums before they move to another sum, is a loss of 2.9e-6 at most on the
    average (the mean of 1 / mantissa is 0.72, of a growing sum half its end);
    what rounds both ways averages out below that.  4e-6 overall."""
    rng = np.random.default_rng(length)
    bs, pages = 784, -(-length // 784)
    g = [ref.cuda(x) for x in ref.head_scales(hkv)]
    cache = [torch.zeros(pa.fp4_cache_shape(pages, bs, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows = [bf16_rows(rng, length, hkv, d).cuda() for _ in range(2)]
    slots = torch.arange(length, device="cuda")
    pa.reshape_and_cache_fp4(*rows, *cache, slots, *g)
    k, v = (torch.empty((length, hkv, d), device="cuda") for _ in range(2))
    pa.gather_cache_fp4(*cache, slots, *g, k, v)
    q = bf16_rows(rng, q_len, hq, d).cuda()
    desc = pa.make_desc(num_seqs=1, q_len=q_len, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                        max_pages_per_seq=pages, max_seq_len=length, num_pages=pages, scale=d ** -0.5, num_splits=1)
    ws = torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
    out = torch.empty((q_len, hq, d), device="cuda")
    call = pa.paged_attention_decode_fp4 if q_len == 1 else pa.paged_attention_verify_fp4
    call(q, *cache, *g, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
         torch.tensor([length], dtype=torch.int32, device="cuda"), desc, out, ws)
    x = torch.einsum("qhd,td->qht", q.double(), k[:, 0].double()) * d ** -0.5
    hidden = torch.arange(length, device="cuda") > length - q_len + torch.arange(q_len, device="cuda")[:, None]
    want = x.masked_fill(hidden[:, None], -math.inf).softmax(-1) @ v[:, 0].double()
    assert ((out.double() - want).norm() / want.norm()).item() <= 4e-6


def test_offsets_past_32_bits():
    """Pages whose byte offset passes 2^32 in each cache."""
    bs, hkv, d = 784, 4, 256
    pages = (1 << 32) // (hkv * bs // 16 * 9 * d) + 40
    rng = np.random.default_rng(1)
    small_k, small_v = ref.random_cache(rng, 2, bs, hkv, d, ref.head_scales(hkv))
    kc, vc = (torch.empty(pa.fp4_cache_shape(pages, bs, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = [pages - 1, pages - 3]
    kc[ids], vc[ids] = ref.cuda(small_k), ref.cuda(small_v)
    g = [ref.cuda(x) for x in ref.head_scales(hkv)]
    for q_len in (1, 2):
        p = Problem(2, [800], 24, hkv, d, 784, q_len=q_len, pool=2)
        p.k, p.v, p.table = small_k, small_v, np.array([[0, 1]], np.int32)
        desc = pa.make_desc(num_seqs=1, q_len=q_len, num_q_heads=24, num_kv_heads=hkv, head_dim=d, block_size=bs,
                            max_pages_per_seq=2, max_seq_len=800, num_pages=pages, scale=p.scale)
        ws = torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
        out = torch.empty(p.q.shape, device="cuda")
        call = pa.paged_attention_decode_fp4 if q_len == 1 else pa.paged_attention_verify_fp4
        call(p.q.cuda(), kc, vc, *g, torch.tensor([ids], dtype=torch.int32, device="cuda"),
             torch.tensor([800], dtype=torch.int32, device="cuda"), desc, out, ws)
        p.check(out.double().cpu().numpy())
    rows = [bf16_rows(rng, 2, hkv, d).cuda() for _ in range(2)]
    slots = torch.tensor([pages * bs - 1, (pages - 3) * bs + 5], device="cuda")
    pa.reshape_and_cache_fp4(*rows, kc, vc, slots, *g)
    back = [torch.empty((2, hkv, d), device="cuda") for _ in range(2)]
    pa.gather_cache_fp4(kc, vc, slots, *g, *back)
    ref.write_rows("k", rows[0].float().cpu().numpy(), g[0].cpu().numpy(), small_k, [bs - 1, bs + 5])
    assert torch.equal(kc[ids].cpu(), torch.from_numpy(small_k))
    assert np.array_equal(back[0].cpu().double().numpy(),
                          ref.read_rows("k", small_k, [bs - 1, bs + 5], g[0].cpu().numpy()).astype(np.float32))


def test_calls_on_another_stream_and_two_at_once():
    p, r = Problem(31, [500, 77], 24, 4, 256, 16), Problem(32, [300, 200], 24, 4, 256, 16, q_len=3)
    jobs = []
    for x in (p, r):
        desc = x.desc()
        jobs.append((x, desc, x.tensors(), torch.empty(x.q.shape, device="cuda"),
                     torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for x, desc, t, out, ws, s in jobs:
            call = pa.paged_attention_decode_fp4 if x.q_len == 1 else pa.paged_attention_verify_fp4
            call(*t, desc, out, ws, stream=s)
    torch.cuda.synchronize()
    for x, _, _, out, _, _ in jobs:
        x.check(out.double().cpu().numpy())


def test_two_graphs_share_a_workspace():
    """Two captured calls of different shapes over one workspace, replayed in turn."""
    jobs = []
    for p in (Problem(41, [900, 77, 400], 8, 2, 128, 16), Problem(42, [700, 300], 24, 4, 256, 16, q_len=5)):
        jobs.append([p, p.desc(num_splits=4), p.tensors(), torch.empty(p.q.shape, device="cuda")])
    ws = torch.empty(max(pa.workspace_bytes(j[1]) for j in jobs), dtype=torch.uint8, device="cuda")
    for j in jobs:
        p, desc, t, out = j
        call = pa.paged_attention_decode_fp4 if p.q_len == 1 else pa.paged_attention_verify_fp4
        call(*t, desc, out, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*t, desc, out, ws)
        j.append(g)
    for _ in range(3):
        for j in jobs:
            j[3].fill_(float("nan"))
        for j in jobs + jobs[::-1]:
            j[4].replay()
        torch.cuda.synchronize()
        for p, _, _, out, _ in jobs:
            p.check(out.double().cpu().numpy())


def test_rows_on_another_stream():
    """Write and gather on a given stream, with inputs made there."""
    rng = np.random.default_rng(8)
    x = [bf16_rows(rng, 100, 4, 128).cuda() for _ in range(2)]
    g = [ref.cuda(v) for v in ref.head_scales(4)]
    cache = [torch.zeros(pa.fp4_cache_shape(9, 16, 4, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.randperm(144, device="cuda")[:100].contiguous()
    out = [torch.empty((100, 4, 128), device="cuda") for _ in range(2)]
    want = [torch.empty_like(o) for o in out]
    other = [c.clone() for c in cache]
    pa.reshape_and_cache_fp4(*x, *other, slots, *g)
    pa.gather_cache_fp4(*other, slots, *g, *want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2000000)  # the rows are late
        late = [v.clone() for v in x]
    pa.reshape_and_cache_fp4(*late, *cache, slots, *g, stream=stream)
    pa.gather_cache_fp4(*cache, slots, *g, *out, stream=stream)
    stream.synchronize()
    for a, b in zip(out + cache, want + other):
        assert torch.equal(a, b)


@pytest.mark.parametrize("q_len", [1, 2])
def test_one_token_and_nothing(q_len):
    """The smallest calls: contexts of nothing but the new rows, beside an empty one."""
    p = Problem(61, [q_len, 0, q_len], 4, 1, 128, 16, q_len=q_len)
    for splits in (1, 2):
        for bf in (False, True):
            out, status = p.run(num_splits=splits, out_dtype=pa.PA_OUT_BF16 if bf else pa.PA_OUT_F32)
            assert status == (0 if q_len == 1 else pa.PA_DEV_BAD_SEQLEN)  # a sequence shorter than its rows
            p.check(out, bf=bf)
