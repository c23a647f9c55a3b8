"""extend_block_tables and release_block_tables against a request-by-request
model in Python, and a serving step built from them (tables, cache write,
verify, decode) eagerly and as a replayed graph."""
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


def pages_of(n, bs):
    return -(-n // bs)


def extend_model(lens, new, table, free, num_free, bs, rows):
    """(table, seq_lens, slots, num_free, status) by walking the requests."""
    table, out, slots, status = table.copy(), [], np.full(rows, -1, np.int64), 0
    pool, P = min(max(num_free, 0), len(free)), len(free)
    if pool != num_free:
        status |= pa.PA_DEV_BAD_PAGE
    at = wanted = 0
    left = pool
    for b, (n, m) in enumerate(zip(lens, new)):
        ok = n >= 0 and m >= 0 and n + m <= table.shape[1] * bs
        m = max(m, 0)
        need = pages_of(n + m, bs) - pages_of(n, bs) if ok else 0
        wanted += need
        yes = ok and at + m <= rows and (need == 0 or wanted <= pool)
        if not ok:
            status |= pa.PA_DEV_BAD_SEQLEN
        elif at + m > rows and m > 0:
            status |= pa.PA_DEV_BAD_SLOT
        elif not yes and m > 0:
            status |= pa.PA_DEV_NO_PAGES
        if yes:
            have = pages_of(n, bs)
            for k in range(need):
                page = free[pool - 1 - (wanted - need + k)]
                if not 0 <= page < P:
                    status |= pa.PA_DEV_BAD_PAGE
                table[b, have + k] = page
            if need:
                left = pool - wanted
            for i in range(m):
                page = table[b, (n + i) // bs]
                if 0 <= page < P:
                    slots[at + i] = int(page) * bs + (n + i) % bs
        out.append(n + m if yes else max(n, 0))
        at += m
    return table, np.array(out, np.int32), slots, left, status


def run_extend(lens, new, table, free, num_free, bs, rows):
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    t, f = i32(table).reshape(table.shape), i32(free)
    out = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((rows,), -9, dtype=torch.int64, device="cuda")
    left, status = i32([-9]), i32([0])
    pa.extend_block_tables(i32(lens), i32(new), t, f, i32([num_free]), bs, out, slots, left, status)
    assert torch.equal(f, i32(free))
    return t.cpu().numpy(), out.cpu().numpy(), slots.cpu().numpy(), int(left), int(status)


def state(rng, B, width, bs, longest, spare):
    lens = rng.integers(0, width * bs + 1, B).astype(np.int32)
    new = np.minimum(rng.integers(0, longest + 1, B), width * bs - lens).astype(np.int32)
    held = pages_of(lens, bs)
    P = int(held.sum()) + int(pages_of(lens + new, bs).sum() - held.sum()) + spare
    order = rng.permutation(max(P, 1)).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(max(P, 1), -1, np.int32)
    free[:len(order) - at] = order[at:]
    return lens, new, table, free, len(order) - at


def same(got, want):
    for name, a, b in zip(("table", "seq_lens", "slots", "num_free", "status"), got, want):
        assert np.array_equal(a, b), name


@pytest.mark.parametrize("B,width,bs,longest", [(1, 3, 16, 1), (1, 40, 16, 600), (3, 1, 1, 1), (32, 42, 784, 1),
                                                (100, 9, 48, 100), (511, 5, 7, 20), (513, 4, 16, 64),
                                                (5000, 3, 16, 30), (2, 700, 3, 2100)])
def test_extend_matches_the_model(B, width, bs, longest):
    rng = np.random.default_rng(B + width)
    lens, new, table, free, n = state(rng, B, width, bs, longest, 3)
    rows = int(new.sum()) + 5
    same(run_extend(lens, new, table, free, n, bs, rows), extend_model(lens, new, table, free, n, bs, rows))


@pytest.mark.parametrize("B,width,bs,longest", [(128, 7, 16, 40), (129, 7, 16, 40), (256, 4, 32, 3), (257, 4, 32, 3),
                                                (512, 5, 16, 60), (60, 500, 16, 7900), (300, 90, 48, 4000),
                                                (600, 60, 48, 2500)])
def test_extend_at_the_sizes_where_the_launch_changes(B, width, bs, longest):
    """Threads per CTA change at 128, 256 and 512 requests, slots per thread with
    their number: half a million slots and more."""
    rng = np.random.default_rng(B)
    lens, new, table, free, n = state(rng, B, width, bs, longest, 1)
    rows = int(new.sum())
    same(run_extend(lens, new, table, free, n, bs, rows), extend_model(lens, new, table, free, n, bs, rows))


@pytest.mark.parametrize("B", [7, 600])
def test_extend_refuses_in_order(B):
    """A pool that runs out, packed rows that run out, lengths that make no sense."""
    rng = np.random.default_rng(B)
    lens, new, table, free, n = state(rng, B, 6, 16, 50, 0)
    rows = int(new.sum())
    for pool, cap in ((n // 2, rows), (0, rows), (n, rows // 2), (n, 0), (n // 2, rows // 3), (-4, rows)):
        same(run_extend(lens, new, table, free, pool, 16, cap), extend_model(lens, new, table, free, pool, 16, cap))
    lens, new = lens.copy(), new.copy()
    lens[1], new[2], new[3], lens[5] = -3, -1, 6 * 16 + 1, 6 * 16 + 1
    rows = int(np.maximum(new, 0).sum())
    same(run_extend(lens, new, table, free, n, 16, rows), extend_model(lens, new, table, free, n, 16, rows))
    big = lens.copy()
    big[0], new[0] = 2 ** 31 - 1, 2 ** 31 - 1  # sums pass 32 bits
    same(run_extend(big, new, table, free, n, 16, 40), extend_model(big.astype(object), new.astype(object), table, free, n, 16, 40))


def test_extend_with_bad_entries_in_the_pool():
    table = np.full((2, 4), -1, np.int32)
    free = np.array([3, 99, 1, -2, 0, 2], np.int32)
    args = ([0, 0], [20, 40], table, free, 5, 16, 60)
    same(run_extend(*args), extend_model(*args))
    assert run_extend(*args)[4] == pa.PA_DEV_BAD_PAGE


def test_extend_without_requests_or_rows():
    table = np.zeros((0, 4), np.int32)
    got = run_extend([], [], table, [4, 5], 2, 16, 6)
    assert (got[2] == -1).all() and got[3] == 2 and got[4] == 0
    same(run_extend([3], [0], np.array([[1]]), [0, 1], 1, 16, 0), (np.array([[1]]), [3], [], 1, 0))


@pytest.mark.parametrize("B,width,bs", [(1, 5, 16), (40, 30, 784), (700, 6, 16), (3000, 4, 5)])
def test_release_matches_the_model(B, width, bs):
    rng = np.random.default_rng(B)
    lens, _, table, free, n = state(rng, B, width, bs, 0, 11)
    lens[0] = 0
    done = (rng.random(B) < 0.4).astype(np.int32) * rng.integers(1, 5, B).astype(np.int32)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    t, f, out, left, status = i32(table), i32(free), i32([0] * B), i32([0]), i32([0])
    pa.release_block_tables(i32(lens), i32(done), t, f, i32([n]), bs, out, left, status)
    want = free.copy()
    at = n
    for b in range(B):
        if done[b]:
            h = pages_of(int(lens[b]), bs)
            want[at:at + h] = table[b, :h]
            at += h
    assert np.array_equal(f.cpu().numpy(), want) and int(left) == at and int(status) == 0
    assert np.array_equal(out.cpu().numpy(), np.where(done, 0, lens)) and np.array_equal(t.cpu().numpy(), table)


def test_release_refuses_what_the_pool_cannot_hold():
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[0, 1], [2, 7], [3, -1], [-1, -1]])
    free, out, left, status = i32([4, 5, -1, -1, -1]), i32([0] * 4), i32([0]), i32([0])
    pa.release_block_tables(i32([20, 32, 16, -1]), i32([1, 1, 0, 0]), table, free, i32([2]), 16, out, left, status)
    # two pages fit, the next two would pass the five of the pool; a negative length
    assert free.tolist() == [4, 5, 0, 1, -1] and left.item() == 4 and out.tolist() == [0, 32, 16, 0]
    assert status.item() == pa.PA_DEV_BAD_PAGE | pa.PA_DEV_BAD_SEQLEN


def test_tables_on_another_stream():
    """Inputs made, and outputs read, on the stream the calls are given."""
    rng = np.random.default_rng(4)
    lens, new, table, free, n = state(rng, 40, 9, 16, 60, 2)
    rows = int(new.sum())
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    host = [i32(x) for x in (lens, new, table, free, [n], np.zeros(40))]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2000000)  # the inputs are late
        t_lens, t_new, t, f, left, zero = (x.clone() for x in host)
    out, done = torch.empty_like(t_lens), torch.empty_like(t_lens)
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    after, back, status = i32([0]), i32([0]), i32([0])
    ones = torch.ones_like(t_lens)
    stream.wait_stream(torch.cuda.current_stream())
    pa.extend_block_tables(t_lens, t_new, t, f, left, 16, out, slots, after, status, stream=stream)
    pa.release_block_tables(out, ones, t, f, after, 16, done, back, status, stream=stream)
    stream.synchronize()
    want = extend_model(lens, new, table, free, n, 16, rows)
    same((t.cpu().numpy(), out.cpu().numpy(), slots.cpu().numpy(), int(after), int(status)), want)
    # every page is back
    assert int(back) == n + int(pages_of(lens, 16).sum()) and (done == 0).all()
    assert sorted(f[:int(back)].tolist()) == sorted(set(f[:int(back)].tolist()))


# -- a serving loop --------------------------------------------------------------------------------

class Serving:
    """Prompts and decode steps over an fp4 cache whose tables live on the GPU."""

    def __init__(self, B, hq, hkv, d, bs, width, pages, prompt):
        self.B, self.hq, self.hkv, self.d, self.bs, self.width, self.pages, self.prompt = B, hq, hkv, d, bs, width, pages, prompt
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((B, width), -1, **i32)
        self.free = torch.randperm(pages, device="cuda").int()
        self.pool = [torch.tensor([pages], **i32), torch.zeros(1, **i32)]
        self.lens = [torch.zeros(B, **i32), torch.zeros(B, **i32)]
        self.status = torch.zeros(1, **i32)
        shape = pa.fp4_cache_shape(pages, bs, hkv, d)
        self.k, self.v = (torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.g = [ref.cuda(x) for x in ref.head_scales(hkv)]
        self.slots = torch.empty(B * prompt, dtype=torch.int64, device="cuda")
        self.new = torch.empty(B, **i32)

    def desc(self, q_len):
        return pa.make_desc(num_seqs=self.B, q_len=q_len, num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d,
                            block_size=self.bs, max_pages_per_seq=self.width, max_seq_len=self.width * self.bs,
                            num_pages=self.pages, scale=self.d ** -0.5)

    def step(self, q, k_new, v_new, out, ws, n):
        """n new tokens of every request: tables, cache write, attention; the state's halves change places."""
        slots = self.slots[:self.B * n]
        self.new.fill_(n)
        pa.extend_block_tables(self.lens[0], self.new, self.table, self.free, self.pool[0], self.bs, self.lens[1], slots,
                               self.pool[1], self.status)
        pa.reshape_and_cache_fp4(k_new, v_new, self.k, self.v, slots, *self.g, self.status)
        call = pa.paged_attention_decode_fp4 if n == 1 else pa.paged_attention_verify_fp4
        call(q, self.k, self.v, *self.g, self.table, self.lens[1], self.desc(n), out, ws, self.status)
        self.lens.reverse()
        self.pool.reverse()


@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(graph):
    """A prompt, then decode steps; each output against float64 attention over
    the rows as the model of the format stores them.  As a graph, two decode
    steps (the state's halves change places twice) are captured and replayed."""
    rng = np.random.default_rng(9)
    B, hq, hkv, d, bs, prompt, steps = 3, 8, 2, 128, 16, 21, 6
    s = Serving(B, hq, hkv, d, bs, 4, 14, prompt)
    rows = lambda n, h: torch.from_numpy(rng.standard_normal((B * n, h, d)).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    model = [np.zeros((B, 0, hkv, d)), np.zeros((B, 0, hkv, d))]

    def check(q, k, v, out, n):
        for i, (kind, x) in enumerate((("k", k), ("v", v))):
            cache = np.zeros((B * n, hkv, 1, 9 * d), np.uint8)  # a page per row
            g = s.g[i].cpu().numpy()
            slots = np.arange(B * n) * 16
            ref.write_rows(kind, x.float().numpy(), g, cache, slots)
            model[i] = np.concatenate([model[i], ref.read_rows(kind, cache, slots, g).reshape(B, n, hkv, d)], 1)
        total = model[0].shape[1]
        got = out.double().cpu().numpy().reshape(B, n, hq, d)
        for b in range(B):
            for i in range(n):
                upto = total - n + i + 1
                for h in range(hq):
                    kk, vv = model[0][b, :upto, h * hkv // hq], model[1][b, :upto, h * hkv // hq]
                    x = kk @ q.double().numpy().reshape(B, n, hq, d)[b, i, h] * d ** -0.5
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    reach = (np.abs(kk) @ np.abs(q.double().numpy().reshape(B, n, hq, d)[b, i, h])).max() * d ** -0.5
                    tol = ref.tolerance(w @ np.abs(vv), np.array(reach), d, upto, False, None)
                    assert (np.abs(got[b, i, h] - w @ vv) <= tol).all()
        assert s.lens[0].tolist() == [total] * B and s.status.item() == 0
        assert s.pool[0].item() == s.pages - B * pages_of(total, bs)

    q, k, v = rows(prompt, hq), rows(prompt, hkv), rows(prompt, hkv)
    out = torch.empty(q.shape, device="cuda")
    s.step(q.cuda(), k.cuda(), v.cuda(), out, ws, prompt)
    check(q, k, v, out, prompt)

    bufs = [[torch.empty((B, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)] for _ in range(2)]
    outs = [torch.empty((B, hq, d), device="cuda") for _ in range(2)]
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for i in range(2):
                s.step(*bufs[i], outs[i], ws, 1)
    for step in range(0, steps, 2):
        ins = [[rows(1, hq), rows(1, hkv), rows(1, hkv)] for _ in range(2)]
        for i in range(2):
            for dst, src in zip(bufs[i], ins[i]):
                dst.copy_(src)
        if graph:
            g.replay()
        else:
            for i in range(2):
                s.step(*bufs[i], outs[i], ws, 1)
        final, s_lens, s_pool = outs, s.lens, s.pool
        # the state after the first of the two steps is gone: check the second one's lengths with both
        lens_after = s.lens[0].clone()
        s.lens, s.pool = [lens_after - 1] + s_lens[1:], [torch.tensor([s.pages - B * pages_of(int(lens_after[0]) - 1, bs)])] + s_pool[1:]
        check(*ins[0], final[0], 1)
        s.lens, s.pool = s_lens, s_pool
        check(*ins[1], final[1], 1)
