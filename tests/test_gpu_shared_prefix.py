"""paged_attention_decode_shared over bf16, e4m3 and fp4 caches against
attention in float64, within tolerances counted from the roundings
(shared_ref.Batch.reference)."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests.shared_ref import KINDS, Batch, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def status0():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# Small batches are read without sharing unless the prefixes' splits are forced: both ways are tried.
BOTH = pytest.mark.parametrize("splits", [0, 2], ids=["plain", "shared"])
HYBRID, DENSE, WIDE = (24, 4, 256), (32, 8, 128), (48, 4, 256)
# prefixes of no chunk, one, a page and a bit, several tiles; own parts of no token, one, a chunk, more; idle sequences
GROUPS = {
    "one of one": [(16, [1])],
    "no prefix": [(0, [1, 40, None, 3])],
    "nothing beyond": [(64, [0, 0, 0])],
    "short of a chunk": [(15, [1, 2, 100])],
    "inside a page": [(100, [1, 17, 300, 64])],
    "leader idle": [(96, [None, 5, None, 20])],
    "all idle": [(32, [None, None]), (48, [1, 2])],
    "uneven": [(160, [3, 1, 40]), (0, [9]), (48, []), (400, [1] * 9 + [130]), (16, [0, 1])],
    "past a block of rows": [(256, [i % 37 for i in range(45)])],
    "rows of three blocks": [(80, [1 + i % 5 for i in range(66)]), (208, [2, None, 7])],
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("shape,bs,out", [(HYBRID, 16, "f32"), (DENSE, 48, "bf16"), (WIDE, 32, "f32"), ((6, 1, 256), 784, "bf16"),
                                          ((16, 16, 128), 64, "f32"), ((32, 2, 128), 16, "bf16")])
def test_groups(name, shape, bs, out, kind):
    b = Batch(len(name), GROUPS[name], *shape, bs, kind, out)
    ref = b.reference()
    for splits in (0, 2):
        status = status0()
        got = b.run(status=status, prefix_splits=splits)
        check(got, *ref)
        assert int(status) == 0
        assert pa.last_plan()["path_id"] == pa.PA_PATH_DECODE_SHARED
        assert torch.equal(got, b.run(prefix_splits=splits))  # bit for bit


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 8, 12, 16])
@pytest.mark.parametrize("d", [128, 256])
def test_heads_per_kv_head(g, d, kind):
    b = Batch(g + d, [(144, [1, 0, 33]), (64, [70] * 8)], 2 * g, 2, d, 32, kind)
    ref = b.reference()
    for splits in (0, 2):
        check(b.run(prefix_splits=splits), *ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [31, 32, 33, 256, 257])
@BOTH
def test_many_sequences_of_all_lengths(n, kind, splits):
    """Own parts of many lengths, equal ones and none, which are taken in an order of their own (up to 256)."""
    own = [(i * 37) % 150 if i % 5 else (None if i % 3 else 0) for i in range(n - 8)]
    b = Batch(n, [(48, own), (160, [1, 149, None, 149, 0, 149, 2, 149])], 4, 2, 128, 16, kind, "bf16")
    t, status = b.tensors(), status0()
    check(b.run(t, status=status, prefix_splits=splits), *b.reference())
    assert int(status) == 0
    t["lens"][3], t["lens"][n - 1] = -1, 2 ** 31 - 1
    check(b.run(t, status=status, prefix_splits=splits), *zero_rows(b, {3, n - 1}))
    assert int(status) == pa.PA_DEV_BAD_SEQLEN


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("prefix_splits,splits", [(1, 1), (2, 1), (1, 5), (7, 3), (40, 40), (300, 2)])
def test_forced_splits(prefix_splits, splits, kind):
    b = Batch(7, [(700, [1, 90, None, 333]), (320, [5, 0])], *HYBRID, 64, kind)
    check(b.run(desc=b.desc(num_splits=splits), shared=b.shared(prefix_splits=prefix_splits)), *b.reference())


@pytest.mark.parametrize("kind", KINDS)
def test_hints_bound_nothing(kind):
    """Prefixes and own parts far longer, and far shorter, than the plan was told."""
    b = Batch(3, [(1200, [1, 700]), (64, [1500, 2, 2])], *DENSE, 16, kind)
    ref = b.reference()
    for kw in (dict(max_prefix_len=16, max_suffix_len=1), dict(max_prefix_len=0, max_suffix_len=0),
               dict(max_prefix_len=10 ** 9, max_suffix_len=10 ** 9, max_group_seqs=10 ** 6)):
        for splits in (0, 1, 5):
            check(b.run(prefix_splits=splits, **kw), *ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_long_prefixes(kind, out):
    """Splits of many tiles, several row blocks, long own parts beside short ones."""
    b = Batch(11, [(9000, [i * 7 for i in range(25)]), (3000, [2000, 1])], *HYBRID, 784, kind, out)
    check(b.run(), *b.reference())
    check(b.run(desc=b.desc(num_splits=1), shared=b.shared(prefix_splits=1)), *b.reference())


@pytest.mark.parametrize("kind", KINDS)
def test_one_group_of_everything_equals_decode(kind):
    """The same batch through the plain decode (every sequence's own table)."""
    b = Batch(5, [(2048, [300 + 11 * i for i in range(40)])], *HYBRID, 16, kind)
    t, desc = b.tensors(), b.desc()
    out = torch.empty((b.n, b.hq, b.d), device="cuda")
    ws = torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
    getattr(pa, "paged_attention_decode" + ("" if kind == "bf16" else "_" + kind))(t["q"], *t["caches"], *t["scales"], t["table"],
                                                                                  t["lens"], desc, out, ws)
    ref, tol = b.reference()
    check(out, ref, tol)
    check(b.run(t), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
def test_growing_scores(kind):
    """Logits that rise along the prefix and again in the own part: the running maximum is raised in every tile."""
    b = Batch(2, [(512, [1, 100, 64]), (256, [40] * 30)], *DENSE, 16, kind)
    if kind == "bf16":
        b.k = torch.ones_like(b.k)
        for s in range(b.n):
            at = torch.from_numpy(b.slots(s))
            b.k.view(-1, b.hkv, b.d)[at] *= (torch.arange(len(at)) / 40 + 1).to(torch.bfloat16)[:, None, None]
    b.q = (b.q.abs() * 8).to(torch.bfloat16)
    ref = b.reference()
    for splits in (0, 2):
        check(b.run(prefix_splits=splits), *ref)


@pytest.mark.parametrize("rows", [5, 30])
def test_rising_scores(rows):
    """K grows along every sequence, so that the running maximum is raised tile after tile (64- and 128-key tiles)."""
    b = Batch(2, [(512, [1 + 9 * i for i in range(rows)])], *DENSE, 16)
    for s in range(b.n):
        at = torch.from_numpy(b.slots(s))
        b.k.view(-1, b.hkv, b.d)[at] = (torch.arange(len(at)) / 200 + 0.1).to(torch.bfloat16)[:, None, None]
    b.q = (b.q.abs() * 4).to(torch.bfloat16)
    for out in ("f32", "bf16"):
        b.out = out
        ref = b.reference()
        for splits in (0, 1):
            check(b.run(prefix_splits=splits), *ref)


@BOTH
@pytest.mark.parametrize("shape,out", [(HYBRID, "f32"), (HYBRID, "bf16"), (DENSE, "f32"), (DENSE, "bf16"), (WIDE, "f32"), (WIDE, "bf16")])
def test_small_weights_beside_small_values(shape, out, splits):
    """e4m3: keys at 2^-20 of the first one's weight carry the output, as the first one's values are 2^-18 of theirs.
    The reference is 2^7 or more below the largest score, and f16 ends half a step below 2^-24: 2^-32 of a weight."""
    b = Batch(6, [(160, [3, 40, 100]), (320, [5] * 9)], *shape, 16, "fp8", out)
    g = b.hq // b.hkv
    b.k.reshape(-1, b.hkv, b.d)[..., 0] = 0
    b.v[...] = np.random.default_rng(1).integers(0x70, 0x7F, b.v.shape)  # 128 to 448
    b.q[...] = 0
    for h in range(b.hkv):
        b.q[:, h * g:(h + 1) * g, 0] = 20 * np.log(2) / (16 * float(b.g[0][h]) * b.scale)
    for s, at in ((0, 0), (1, 170), (3, 0), (4, 322)):  # of both prefixes and of two own parts
        b.k.reshape(-1, b.hkv, b.d)[b.slots(s)[at], :, 0] = 0x58  # 16
        b.v.reshape(-1, b.hkv, b.d)[b.slots(s)[at]] = 0x01        # 2^-9
    ref, tol = b.reference(f16_end=2.0 ** -32)
    check(b.run(prefix_splits=splits), ref, tol)


# -- lengths, groups and pages that make no sense --------------------------------------------------

def zero_rows(b, bad):
    """The batch with the sequences in `bad` taken for idle."""
    ref, tol = b.reference()
    ref[list(bad)], tol[list(bad)] = 0, 0
    return ref, tol


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("change,bad", [
    (dict(prefix={2: 96}), {2}), (dict(prefix={2: -16}), {2}), (dict(prefix={2: 10 ** 9}), {2}), (dict(lens={3: -5}), {3}),
    (dict(lens={3: 10 ** 9}), {3}), (dict(lens={1: 100}), {1}),      # shorter than its prefix
    (dict(prefix={0: -1}), {0, 1, 2, 3}),                            # the leader's: nobody agrees with it
    (dict(starts={0: 1}), {0}), (dict(starts={2: 5}), {5}),          # not in any group
    (dict(starts={1: 5, 2: 3}), {0, 1, 2, 3, 4, 5}), (dict(starts={0: -1}), {0, 1, 2, 3, 4, 5})])
@BOTH
def test_bad_lengths_and_groups(change, bad, kind, splits):
    b = Batch(4, [(112, [3, 20, 1, 60]), (32, [5, 9])], *HYBRID, 16, kind)
    want = zero_rows(b, bad)
    t = b.tensors()
    for name, values in change.items():
        for i, v in values.items():
            t[name][i] = v
    status = status0()
    check(b.run(t, status=status, prefix_splits=splits), *want)
    assert int(status) == pa.PA_DEV_BAD_SEQLEN


@BOTH
@pytest.mark.parametrize("kind", KINDS)
def test_more_sequences_than_the_host_said(kind, splits):
    b = Batch(4, [(64, [3] * 50), (32, [5, 9])], *HYBRID, 16, kind)  # 50 x 6 rows: three blocks
    ref = b.reference()
    for most in (20, 21, 49):
        want = [x.copy() for x in ref]
        want[0][most:50], want[1][most:50] = 0, 0
        status = status0()
        check(b.run(max_group_seqs=most, prefix_splits=splits, status=status), *want)
        assert int(status) == pa.PA_DEV_BAD_SEQLEN


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [-1, 10 ** 6])
def test_bad_pages(page, kind):
    b = Batch(6, [(128, [3, 20, 1]), (32, [90, 9])], *DENSE, 16, kind)
    for where, bad in (((0, 2), {0, 1, 2}), ((1, 8), {1}), ((3, 4), {3})):  # the prefix, two own parts
        for splits in (0, 2):
            t, status = b.tensors(), status0()
            t["table"][where] = page
            check(b.run(t, status=status, prefix_splits=splits), *zero_rows(b, bad if splits else {where[0]}))
            assert int(status) == pa.PA_DEV_BAD_PAGE


@pytest.mark.parametrize("kind", KINDS)
@BOTH
def test_what_no_sequence_sees_may_be_anything(kind, splits):
    """NaN in every slot that is not in use, in the rows of q of idle sequences, and in the workspace."""
    b = Batch(8, [(100, [1, 17, None, 64]), (48, [0, 5]), (16, [None])], *HYBRID, 48, kind)
    ref, tol = b.reference()
    dead = np.ones(b.pages * b.bs, bool)
    for s in range(b.n):
        dead[b.slots(s)] = False
    if kind == "bf16":
        for c in (b.k, b.v):
            c.view(-1, b.hkv, b.d)[torch.from_numpy(dead)] = float("nan")
    elif kind == "fp8":
        for c in (b.k, b.v):
            c.reshape(-1, b.hkv, b.d)[dead] = 0x7F
    else:
        from tests import fp4_ref
        for which, c in zip("kv", (b.k, b.v)):
            for tok in range(16):
                places = np.concatenate(fp4_ref.byte_places(which, tok, b.d))
                rows = c[..., places]
                rows[np.broadcast_to(dead.reshape(b.pages, 1, -1, 16)[..., tok], rows.shape[:3])] = 0xFF
                c[..., places] = rows
    b.q[b.lens == 0] = float("nan")
    check(b.run(prefix_splits=splits), ref, tol)


@BOTH
@pytest.mark.parametrize("kind", KINDS)
def test_nan_reaches_what_depends_on_it(kind, splits):
    b = Batch(9, [(96, [3, 20, 1]), (64, [5, 9])], *HYBRID, 16, kind)
    ref, tol = b.reference()
    b.q[1, 4, 7] = float("nan")  # one head of one sequence
    bad = np.zeros((b.n, b.hq), bool)
    bad[1, 4] = True

    def spoil(slot, head):
        if kind == "bf16":
            b.k.view(-1, b.hkv, b.d)[slot, head, 3] = float("nan")
        elif kind == "fp8":
            b.k.reshape(-1, b.hkv, b.d)[slot, head, 3] = 0x7F
        else:
            from tests import fp4_ref
            _, scales = fp4_ref.byte_places("k", slot % 16, b.d)
            b.k[slot // b.bs, head, slot % b.bs // 16, scales[0]] = 0x7F

    spoil(int(b.slots(0)[50]), 2)   # a key of the first group's prefix, KV head 2: heads 12 .. 17 of its sequences
    bad[:3, 12:18] = True
    spoil(int(b.slots(4)[66]), 0)   # a key of the last sequence's own part
    bad[4, :6] = True
    got = b.run(prefix_splits=splits).cpu()
    assert torch.isnan(got[torch.from_numpy(bad)]).all()
    good = torch.from_numpy(~bad)
    check(got[good], ref[~bad], tol[~bad])


def spoil_value(b, slot, head):
    """A NaN value of dim 21 (over an fp4 cache of its block of 16 dims, 16 .. 31) of a slot; returns the dims."""
    if b.kind == "bf16":
        b.v.view(-1, b.hkv, b.d)[slot, head, 21] = float("nan")
    elif b.kind == "fp8":
        b.v.reshape(-1, b.hkv, b.d)[slot, head, 21] = 0x7F
    else:
        from tests import fp4_ref
        _, scales = fp4_ref.byte_places("v", slot % 16, b.d)
        b.v[slot // b.bs, head, slot % b.bs // 16, scales[1]] = 0x7F
        return slice(16, 32)
    return slice(21, 22)


@BOTH
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,out", [(HYBRID, "f32"), (HYBRID, "bf16"), (DENSE, "f32"), (DENSE, "bf16")])
@pytest.mark.parametrize("n", [3, 12, 30])  # rows of the first group: copies of them share a tile, or a block, or blocks
def test_nan_values_reach_who_sees_them(n, shape, out, kind, splits):
    b = Batch(n, [(96, [3 + i for i in range(n)]), (64, [5, 9])], *shape, 16, kind, out)
    ref, tol = b.reference()
    g = b.hq // b.hkv
    bad = np.zeros((b.n, b.hq, b.d), bool)
    bad[:n, 2 * g:3 * g, spoil_value(b, int(b.slots(0)[70]), 2)] = True      # of the first group's prefix
    bad[n + 1, :g, spoil_value(b, int(b.slots(n + 1)[66]), 0)] = True        # of the last sequence's own part
    got = b.run(prefix_splits=splits).cpu()
    assert torch.isnan(got[torch.from_numpy(bad)]).all()
    check(got[torch.from_numpy(~bad)], ref[~bad], tol[~bad])


@BOTH
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 12])
def test_slots_past_the_sequences_may_be_nan_at_128(n, out, kind, splits):
    b = Batch(n, [(100, [1 + 5 * i for i in range(n)]), (48, [0, 5])], *DENSE, 48, kind, out)
    ref, tol = b.reference()
    dead = np.ones(b.pages * b.bs, bool)
    for s in range(b.n):
        dead[b.slots(s)] = False
    if kind == "fp4":
        whole = dead.reshape(b.pages, 1, -1, 16).all(-1)  # chunks without a token in use
        for c in (b.k, b.v):
            c[np.broadcast_to(whole, c.shape[:3])] = 0xFF
    else:
        for c in (b.k, b.v):
            if kind == "bf16":
                c.view(-1, b.hkv, b.d)[torch.from_numpy(dead)] = float("nan")
            else:
                c.reshape(-1, b.hkv, b.d)[dead] = 0x7F
    check(b.run(prefix_splits=splits), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,out", [((8, 2, 128), "f32"), ((6, 1, 256), "bf16")])
def test_more_pages_than_a_cta_stages(kind, shape, out):
    """Prefixes and own parts of more than 512 pages in one split."""
    b = Batch(5, [(9000, [9001, 3, 1]), (8200, [20] * 7)], *shape, 16, kind, out)
    check(b.run(desc=b.desc(num_splits=1), shared=b.shared(prefix_splits=1)), *b.reference())


# -- calls side by side ----------------------------------------------------------------------------

@BOTH
@pytest.mark.parametrize("kind", KINDS)
def test_stream_and_graphs_with_one_workspace(kind, splits):
    """Two captured calls of different shapes share a workspace and are replayed in turn, with lengths that change on
    the GPU between replays; and a call on a stream of its own."""
    a = Batch(1, [(512, [1, 40, 7]), (64, [3])], *HYBRID, 16, kind)
    c = Batch(2, [(80, [9] * 30)], *DENSE, 16, kind, "bf16")
    ta, tc = a.tensors(), c.tensors()
    ws = torch.empty(max(pa.shared_workspace_bytes(x.desc(), x.shared(prefix_splits=splits)) for x in (a, c)), dtype=torch.uint8,
                     device="cuda")
    outs = [torch.zeros((x.n, x.hq, x.d), device="cuda", dtype=torch.bfloat16 if x.out == "bf16" else torch.float32) for x in (a, c)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.run(ta, workspace=ws, out=outs[0], stream=s, prefix_splits=splits)
    s.synchronize()
    check(outs[0], *a.reference())
    graphs = []
    for x, t, o in ((a, ta, outs[0]), (c, tc, outs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(t, workspace=ws, out=o, prefix_splits=splits)
        graphs.append(g)
    for step in range(3):
        for g, x, t, o in zip(graphs, (a, c), (ta, tc), outs):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            check(o, *x.reference())
            x.lens = np.where(x.lens > x.prefix + 1, x.lens - 1, x.lens)
            t["lens"].copy_(torch.from_numpy(x.lens))


@BOTH
def test_many_calls_behind_one_another(splits):
    """Calls with one workspace and no wait between them, their inputs written just before on the same stream."""
    b = Batch(3, [(256, [1, 33, 80]), (1024, [5] * 12)], *HYBRID, 16)
    t, desc, shared = b.tensors(), b.desc(), b.shared(prefix_splits=splits)
    ws = torch.empty(pa.shared_workspace_bytes(desc, shared), dtype=torch.uint8, device="cuda")
    want = b.run(t, prefix_splits=splits)
    src = {k: t[k].clone() for k in ("q", "table", "lens", "starts", "prefix")}
    outs = []
    for i in range(20):
        for k in src:
            t[k].zero_()
            t[k].copy_(src[k])
        outs.append(b.run(t, desc, shared, workspace=ws))
    for o in outs:
        assert torch.equal(o, want)


@BOTH
@pytest.mark.parametrize("kind", KINDS)
def test_two_calls_at_once(kind, splits):
    """Calls on two streams beside each other, each with a workspace of its own."""
    batches = [Batch(3, [(256, [1, 33, 80]), (1024, [5] * 12)], *HYBRID, 16, kind), Batch(4, [(640, [7, 200, None])], *DENSE, 16, kind)]
    jobs = []
    for b in batches:
        t, desc, shared = b.tensors(), b.desc(), b.shared(prefix_splits=splits)
        want = b.run(t, desc, shared)
        jobs.append((b, t, desc, shared, want, torch.empty(pa.shared_workspace_bytes(desc, shared), dtype=torch.uint8, device="cuda"),
                     [torch.full_like(want, float("nan")) for _ in range(15)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(15):
        for b, t, desc, shared, _, ws, outs, stream in jobs:
            b.run(t, desc, shared, workspace=ws, out=outs[i], stream=stream)
    torch.cuda.synchronize()
    for _, _, _, _, want, _, outs, _ in jobs:
        assert all(torch.equal(o, want) for o in outs)


def test_cache_past_two_to_the_32_bytes():
    pages, bs, hkv, d = 2700, 832, 8, 128  # 4.6 GB each
    b = Batch(1, [(bs * 2, [30, 900]), (bs, [5])], 32, hkv, d, bs)
    big = [torch.zeros((pages, bs, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    t = b.tensors()
    shift = pages - b.pages
    for x, c in zip(big, t["caches"]):
        x[shift:] = c
    t["caches"] = tuple(big)
    t["table"] = torch.where(t["table"] >= 0, t["table"] + shift, t["table"])
    ref = b.reference()
    for splits in (0, 2):
        check(b.run(t, desc=b.desc(num_pages=pages), prefix_splits=splits), *ref)


def test_no_sequences():
    b = Batch(1, [(16, [1])], *HYBRID, 16)
    t = b.tensors()
    t |= dict(q=t["q"][:0], table=t["table"][:0], lens=t["lens"][:0], prefix=t["prefix"][:0], starts=t["starts"][:1] * 0)
    desc, shared = b.desc(num_seqs=0), pa.make_prefix(num_groups=0, max_group_seqs=0)
    pa.paged_attention_decode_shared(t["q"], *t["caches"], t["table"], t["lens"], t["starts"], t["prefix"], desc, shared,
                                     torch.empty((0, 24, 256), device="cuda"), torch.empty(1, dtype=torch.uint8, device="cuda"))


# -- the operators together ------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@BOTH
@pytest.mark.parametrize("graph", [False, True])
def test_a_sampling_run(kind, graph, splits):
    """A prompt is written with its rotations, forked into samples that each go on by a few tokens and are then let
    go: block tables, rotary_and_cache, fork, page copies, shared decode and release, all on the GPU, against
    attention in float64 over the rows as they were written."""
    hq, hkv, d, bs, prompt, n, steps, P = 24, 4, 256, 16, 85, 6, 20, 64
    dev = dict(device="cuda")
    i32 = dict(dtype=torch.int32, **dev)
    gen = torch.Generator().manual_seed(4)
    freqs, factor = pa.rotary_frequencies(64, base=1e6)
    suffix = "" if kind == "bf16" else "_" + kind
    shape = pa.fp4_cache_shape(P, bs, hkv, d) if kind == "fp4" else (P, bs, hkv, d)
    caches = [torch.zeros(shape, dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, **dev) for _ in range(2)]
    scales = () if kind == "bf16" else tuple(torch.full((hkv,), 1 / 50, **dev) for _ in range(2))
    copy = pa.copy_cache_pages_fp4 if kind == "fp4" else pa.copy_cache_pages
    width = 12
    table = torch.full((n, width), -1, **i32)
    free, num = torch.randperm(P, generator=gen).int().cuda(), torch.tensor([P], **i32)
    zeros = lambda k: torch.zeros(k, **i32)  # noqa: E731
    status = zeros(1)

    # the prompt, into request 0
    lens, num2, slots = zeros(n), zeros(1), torch.zeros(prompt, dtype=torch.int64, **dev)
    new = zeros(n)
    new[0] = prompt
    pa.extend_block_tables(zeros(n), new, table, free, num, bs, lens, slots, num2, status)
    qkv = torch.randn((prompt, hq + 2 * hkv, d), generator=gen).bfloat16().cuda()
    q_out = torch.empty((prompt, hq, d), dtype=torch.bfloat16, **dev)
    getattr(pa, "rotary_and_cache" + suffix)(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], torch.arange(prompt, **i32),
                                             freqs, q_out, *caches, slots, *scales, factor=factor, status=status)
    # the samples
    parent = torch.zeros(n, **i32)
    parent[0] = -1
    src, dst, tok, lens1, shares, num3 = zeros(n), zeros(n), zeros(n), zeros(n), zeros(P), zeros(1)
    pa.fork_block_tables(lens, parent, table, free, num2, zeros(P), bs, lens1, shares, src, dst, tok, num3, status)
    copy(caches, src, dst, tok, status)
    assert lens1.tolist() == [prompt] * n and int(num3) == P - 6 - (n - 1)
    starts, prefix = torch.tensor([0, n], **i32), torch.full((n,), prompt // bs * bs, **i32)

    # steps: one token per sample
    desc = pa.make_desc(num_seqs=n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs, max_pages_per_seq=width,
                        max_seq_len=width * bs, num_pages=P, scale=1 / 16)
    shared = pa.make_prefix(num_groups=1, max_group_seqs=n, max_prefix_len=prompt, max_suffix_len=40, prefix_splits=splits)
    ws = torch.empty(pa.shared_workspace_bytes(desc, shared), dtype=torch.uint8, **dev)
    rows = torch.empty((n, hq + 2 * hkv, d), dtype=torch.bfloat16, **dev)
    q, out = torch.empty((n, hq, d), dtype=torch.bfloat16, **dev), torch.empty((n, hq, d), **dev)
    held, pool, lens2, pool2, slot = lens1.clone(), num3.clone(), zeros(n), zeros(1), torch.zeros(n, dtype=torch.int64, **dev)
    one = torch.ones(n, **i32)

    def step():
        pa.extend_block_tables(held, one, table, free, pool, bs, lens2, slot, pool2, status)
        getattr(pa, "rotary_and_cache" + suffix)(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], lens2, freqs, q, *caches,
                                                 slot, *scales, factor=factor, position_offset=-1, status=status)
        getattr(pa, "paged_attention_decode_shared" + suffix)(q, *caches, *scales, table, lens2, starts, prefix, desc, shared, out,
                                                              ws, status=status)
        held.copy_(lens2)
        pool.copy_(pool2)

    rows.copy_(torch.randn(rows.shape, generator=gen))
    step()
    replay = step
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        replay = g.replay
    b = Batch(0, [(prompt // bs * bs, [1] * n)], hq, hkv, d, bs, kind)  # (its reference, over what the GPU holds)
    b.scale, b.width, b.pages = 1 / 16, width, P
    for i in range(steps):
        if i:
            rows.copy_(torch.randn(rows.shape, generator=gen))
            replay()
        torch.cuda.synchronize()
        assert int(status) == 0 and held.tolist() == [prompt + i + 1] * n
        b.lens, b.table, b.q = held.cpu().numpy(), table.cpu().numpy(), q.cpu()
        b.k, b.v = (c.cpu() if kind == "bf16" else c.cpu().numpy() for c in caches)
        b.g = None if kind == "bf16" else tuple(s.cpu().numpy() for s in scales)
        check(out, *b.reference())
    # every page comes back
    lens3, shares2, num4 = zeros(n), zeros(P), zeros(1)
    pa.release_shared_block_tables(held, one, table, free, pool, shares, bs, lens3, shares2, num4, status)
    assert int(num4) == P and sorted(free.tolist()) == list(range(P)) and not shares2.any() and not lens3.any()
    assert int(status) == 0
