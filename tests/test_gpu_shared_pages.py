"""fork_block_tables, release_shared_block_tables, compact_block_tables and
copy_cache_pages against the request-by-request model."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import shared_pages_model as model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def out(n):
    return torch.full((n,), -9, dtype=torch.int32, device="cuda")


def same(got, want):
    for name, w in want.items():
        assert np.array_equal(got[name].cpu().numpy().reshape(np.shape(w)), w), name


def run_fork(p, parent, bs):
    B, P = len(p["lens"]), len(p["free"])
    g = dict(table=i32(p["table"]).reshape(p["table"].shape), lens=out(B), shares=out(P), src=out(B), dst=out(B), tokens=out(B),
             num_free=out(1))
    free, status = i32(p["free"]), i32([0])
    pa.fork_block_tables(i32(p["lens"]), i32(parent), g["table"], free, i32([p["num_free"]]), i32(p["shares"]), bs, g["lens"],
                         g["shares"], g["src"], g["dst"], g["tokens"], g["num_free"], status)
    assert torch.equal(free, i32(p["free"]))
    return g, int(status)


def run_release(p, finished, bs):
    B, P = len(p["lens"]), len(p["free"])
    g = dict(free=i32(p["free"]), lens=out(B), shares=out(P), num_free=out(1))
    table, status = i32(p["table"]).reshape(p["table"].shape), i32([0])
    pa.release_shared_block_tables(i32(p["lens"]), i32(finished), table, g["free"], i32([p["num_free"]]), i32(p["shares"]), bs,
                                   g["lens"], g["shares"], g["num_free"], status)
    assert np.array_equal(table.cpu().numpy(), p["table"])
    return g, int(status)


def run_compact(p, bs, most):
    P = len(p["free"])
    g = dict(table=i32(p["table"]).reshape(p["table"].shape), free=out(P), num_free=out(1), shares=out(P), map=out(P), src=out(most),
             dst=out(most), extent=out(1))
    status = i32([0])
    args = (i32(p["lens"]), g["table"], i32(p["free"]), i32([p["num_free"]]), i32(p["shares"]), bs, g["free"], g["num_free"],
            g["shares"], g["map"], g["src"], g["dst"], g["extent"], status)
    pa.compact_block_tables(*args)
    first = {k: v.clone() for k, v in g.items()}
    pa.compact_block_tables(*args)  # again: what has moved stays where it is
    for k in g:
        assert torch.equal(g[k], first[k]), k
    return g, int(status)


SIZES = [(1, 3, 16, 5), (2, 1, 1, 1), (9, 12, 16, 40), (40, 30, 784, 7), (255, 9, 16, 300), (257, 5, 48, 3), (700, 6, 16, 1),
         (3000, 4, 5, 2000), (2100, 70, 16, 900)]  # (the last: more entries than one cluster walks)


@pytest.mark.parametrize("B,width,bs,spare", SIZES)
def test_fork_matches_the_model(B, width, bs, spare):
    rng = np.random.default_rng(B + width)
    p = model.pool(rng, B, width, bs, spare)
    parent = np.full(B, -1, np.int32)
    idle = np.nonzero(p["lens"] == 0)[0]
    busy = np.nonzero(p["lens"] > 0)[0]
    if len(busy):
        parent[idle] = np.where(rng.random(len(idle)) < 0.8, busy[rng.integers(0, len(busy), len(idle))], -1)
    want, code = model.fork(p["lens"], parent, p["table"], p["free"], p["num_free"], p["shares"], bs)
    got, status = run_fork(p, parent, bs)
    same(got, want)
    assert status == code


def test_fork_refuses():
    """Children of children, of themselves, of requests that are not there, into slots in use, of bad lengths; a
    pool that runs out, one of a bad size, and bad entries in the pool and in a parent's row."""
    rng = np.random.default_rng(3)
    p = model.pool(rng, 12, 6, 16, 30, share=0.0)
    p["lens"][:] = [70, 0, 0, 33, 0, 0, 90, 0, 0, 0, 97, -4]
    p["table"][0, :5], p["table"][6, :6], p["table"][3, :3] = p["free"][:5], p["free"][5:11], p["free"][11:14]
    p["free"] = np.roll(p["free"], -14)
    p["num_free"] = 4
    parent = np.array([-1, 0, 1, 0, 4, 99, -1, 10, 11, 6, -1, -1], np.int32)
    for pages in (4, 1, 0, -3, 10 ** 6):
        p["num_free"] = pages
        want, code = model.fork(p["lens"], parent, p["table"], p["free"], pages, p["shares"], 16)
        got, status = run_fork(p, parent, 16)
        same(got, want)
        assert status == code and status & pa.PA_DEV_BAD_SEQLEN
    p["num_free"], p["free"][1], p["table"][0, 2] = 2, -1, 10 ** 6
    parent[:] = [-1, 0, 0, -1, -1, -1, -1, 6, -1, -1, -1, -1]
    want, code = model.fork(p["lens"], parent, p["table"], p["free"], 2, p["shares"], 16)
    got, status = run_fork(p, parent, 16)
    same(got, want)
    assert status == code and status & pa.PA_DEV_BAD_PAGE and status & pa.PA_DEV_NO_PAGES


@pytest.mark.parametrize("B,width,bs,spare", SIZES)
def test_release_matches_the_model(B, width, bs, spare):
    rng = np.random.default_rng(B * 3 + width)
    p = model.pool(rng, B, width, bs, spare)
    for finished in (rng.integers(0, 2, B), np.ones(B, np.int64) * 7, np.zeros(B, np.int64)):
        want, code = model.release(p["lens"], finished, p["table"], p["free"], p["num_free"], p["shares"], bs)
        got, status = run_release(p, finished, bs)
        same(got, want)
        assert status == code == 0
    p["lens"][0], p["num_free"] = -1, -2
    if B > 2:
        p["lens"][2] = width * bs + 1
        used = np.nonzero(p["lens"] > 0)[0][-1]
        p["table"][used, 0] = -1
    want, code = model.release(p["lens"], finished + 1, p["table"], p["free"], p["num_free"], p["shares"], bs)
    got, status = run_release(p, finished + 1, bs)
    same(got, want)
    assert status == code != 0


def test_release_of_what_was_not_held():
    """Pages let go of twice come back once; pages that the pool has no room for are dropped."""
    p = dict(lens=np.array([32, 32, 16], np.int32), table=np.array([[1, 2], [1, 3], [1, 0]], np.int32),
             free=np.array([4, 0, -1, -1, -1], np.int32), num_free=2, shares=np.array([0, 1, 0, 0, 0], np.int32))
    for finished in ([1, 1, 1], [1, 1, 0], [0, 0, 1]):
        want, code = model.release(p["lens"], np.array(finished), p["table"], p["free"], 2, p["shares"], 16)
        got, status = run_release(p, finished, 16)
        same(got, want)
        assert status == code
    assert run_release(p, [1, 1, 1], 16)[1] == pa.PA_DEV_BAD_PAGE
    p["num_free"] = 4
    want, code = model.release(p["lens"], np.array([1, 1, 0]), p["table"], p["free"], 4, p["shares"], 16)
    got, status = run_release(p, [1, 1, 0], 16)
    same(got, want)
    assert status == code == pa.PA_DEV_BAD_PAGE


@pytest.mark.parametrize("B,width,bs,spare", SIZES + [(30, 400, 16, 70000), (30, 400, 16, 420000)])  # (the last: more pages than one cluster holds)
@pytest.mark.parametrize("most", [1, 7, 300])
def test_compact_matches_the_model(B, width, bs, spare, most):
    rng = np.random.default_rng(B * 7 + width)
    p = model.pool(rng, B, width, bs, spare)
    want, code = model.compact(p["lens"], p["table"], p["free"], p["num_free"], p["shares"], bs, most)
    got, status = run_compact(p, bs, most)
    same(got, want)
    assert status == code == 0


def test_compact_of_odd_pools():
    rng = np.random.default_rng(1)
    p = model.pool(rng, 10, 8, 16, 50)
    P = len(p["free"])
    everything = np.arange(P, dtype=np.int32)
    for free, n in ((p["free"], 0), (everything, P), (everything[::-1].copy(), P // 2), (np.zeros(P, np.int32), P),
                    (np.full(P, -1, np.int32), 3), (p["free"], -1), (p["free"], P + 5)):
        q = p | dict(free=free, num_free=n)
        want, code = model.compact(q["lens"], q["table"], free, n, q["shares"], 16, 20)
        got, status = run_compact(q, 16, 20)
        same(got, want)
        assert status == code
    p["lens"][0], p["lens"][1], p["table"][2, 0], p["lens"][2] = -1, 8 * 16 + 1, P, 5
    want, code = model.compact(p["lens"], p["table"], p["free"], p["num_free"], p["shares"], 16, 0)
    got, status = run_compact(p, 16, 0)  # no move at all
    same(got, want)
    assert status == code == pa.PA_DEV_BAD_SEQLEN | pa.PA_DEV_BAD_PAGE


def cache(rng, kind, pages, bs, hkv, d):
    shape = pa.fp4_cache_shape(pages, bs, hkv, d) if kind == "fp4" else (pages, bs, hkv, d * (2 if kind == "bf16" else 1))
    t = torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).cuda()
    return t.view(torch.bfloat16) if kind == "bf16" else t


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("pages,bs,hkv,d,n,caches", [(3, 16, 1, 128, 1, 1), (40, 16, 8, 128, 300, 3), (9, 784, 4, 256, 5, 2),
                                                     (30, 48, 3, 128, 17, 128), (12, 832, 8, 128, 4, 1)])
def test_copies(kind, pages, bs, hkv, d, n, caches):
    rng = np.random.default_rng(pages + n)
    all_caches = [cache(rng, kind, pages, bs, hkv, d) for _ in range(caches)]
    before = [c.clone() for c in all_caches]
    order = rng.permutation(pages)
    moves = min(n, pages // 2)
    src, dst = np.full(n, -1), np.full(n, -1)
    at = rng.permutation(n)[:moves]  # the others copy nothing
    src[at], dst[at] = order[rng.integers(0, pages - moves, moves)], order[pages - moves:]
    tokens = rng.integers(0, bs + 1, n)
    if moves > 1:
        src[at[0]], tokens[at[1]] = -1, 0
    call = pa.copy_cache_pages_fp4 if kind == "fp4" else pa.copy_cache_pages
    for t in (tokens, None):
        for c, b in zip(all_caches, before):
            c.copy_(b)
        status = i32([0])
        call(all_caches, i32(src), i32(dst), None if t is None else i32(t), status)
        assert int(status) == 0
        for c, b in zip(all_caches, before):
            want = b.clone()
            for i in range(n):
                if src[i] < 0 or dst[i] < 0:
                    continue
                rows = bs if t is None else -(-int(t[i]) // 16) * 16
                if kind == "fp4":
                    want[dst[i], :, :rows // 16] = b[src[i], :, :rows // 16]
                else:
                    want[dst[i], :rows] = b[src[i], :rows]
            assert torch.equal(c.view(torch.uint8), want.view(torch.uint8))


def test_copies_skip_bad_pairs():
    rng = np.random.default_rng(0)
    c = cache(rng, "bf16", 6, 32, 2, 128)
    b, status = c.clone(), i32([0])
    pa.copy_cache_pages([c], i32([0, 6, 2, 3, 1]), i32([4, 5, 10 ** 9, 3, 5]), i32([32, 32, 32, 32, 33]), status)
    assert int(status) == pa.PA_DEV_BAD_PAGE | pa.PA_DEV_BAD_SEQLEN
    b[4] = b[0]
    assert torch.equal(c.view(torch.uint8), b.view(torch.uint8))
    pa.copy_cache_pages([c], i32([]), i32([]))


def test_offsets_past_two_to_the_32():
    """Pages whose bytes lie beyond 2^32 of the cache's start."""
    pages, bs = 700, 832  # 6.8 MB a page
    c = torch.zeros((pages, bs, 32, 128), dtype=torch.bfloat16, device="cuda")
    c[650] = torch.randn((bs, 32, 128), device="cuda").bfloat16()
    pa.copy_cache_pages([c], i32([650, 650]), i32([699, 3]), i32([832, 17]))
    assert torch.equal(c[699], c[650]) and torch.equal(c[3, :32], c[650, :32]) and not c[3, 32:].any()


def test_a_step_as_a_graph():
    """Release, fork, copies and compaction in one graph, replayed: the same as eagerly, and again."""
    rng = np.random.default_rng(8)
    bs, B = 16, 20
    p = model.pool(rng, B, 10, bs, 60)
    finished = (rng.random(B) < 0.4).astype(np.int32)
    r, _ = model.release(p["lens"], finished, p["table"], p["free"], p["num_free"], p["shares"], bs)
    parent = np.full(B, -1, np.int32)
    busy, idle = np.nonzero(r["lens"] > 0)[0], np.nonzero(r["lens"] == 0)[0]
    parent[idle] = busy[rng.integers(0, len(busy), len(idle))]
    f, _ = model.fork(r["lens"], parent, p["table"], r["free"], r["num_free"], r["shares"], bs)
    c, _ = model.compact(f["lens"], f["table"], r["free"], f["num_free"], f["shares"], bs, 50)
    P = len(p["free"])
    lens, fin, par, table, shares = i32(p["lens"]), i32(finished), i32(parent), i32(p["table"]).reshape(B, -1), i32(p["shares"])
    free, num = i32(p["free"]), i32([p["num_free"]])
    k = cache(rng, "e4m3", P, bs, 2, 128)
    start = (table.clone(), free.clone(), k.clone())
    m = {n: out(s) for n, s in dict(l1=B, s1=P, n1=1, l2=B, s2=P, n2=1, src=B, dst=B, tok=B, fo=P, no=1, so=P, map=P, cs=50,
                                    cd=50, ext=1).items()}

    def step():
        pa.release_shared_block_tables(lens, fin, table, free, num, shares, bs, m["l1"], m["s1"], m["n1"])
        pa.fork_block_tables(m["l1"], par, table, free, m["n1"], m["s1"], bs, m["l2"], m["s2"], m["src"], m["dst"], m["tok"],
                             m["n2"])
        pa.copy_cache_pages([k], m["src"], m["dst"], m["tok"])
        pa.compact_block_tables(m["l2"], table, free, m["n2"], m["s2"], bs, m["fo"], m["no"], m["so"], m["map"], m["cs"], m["cd"],
                                m["ext"])
        pa.copy_cache_pages([k], m["cs"], m["cd"])

    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in (table, k, *m.values())]
    same(dict(table=table, free=m["fo"], num_free=m["no"], shares=m["so"], map=m["map"], src=m["cs"], dst=m["cd"], extent=m["ext"]), c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t, s in zip((table, free, k), start):
            t.copy_(s)
        for t in m.values():
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((table, k, *m.values()), eager):
            assert torch.equal(a, b)
