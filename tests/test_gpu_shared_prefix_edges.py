"""paged_attention_decode_shared where the values, groups and lengths are at
their edges: NaN beside large logits, starts past the sequences, leaders that
make no sense.  Tolerances: shared_ref.Batch.reference."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import fp4_ref
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


HYBRID, DENSE = (24, 4, 256), (32, 8, 128)


# -- NaN beside large logits -----------------------------------------------------------------------

def only_key(b, slot, logit):
    """K is zero but for dim 0 of one slot, q but for dim 0: that key's logit is `logit`, the others' are 0."""
    b.k[...] = 0
    if b.kind == "bf16":
        b.k.view(-1, b.hkv, b.d)[slot, :, 0] = 8.0
        at = np.full(b.hkv, 8.0)
    elif b.kind == "fp8":
        b.k.reshape(-1, b.hkv, b.d)[slot, :, 0] = 0x50  # 8
        at = 8.0 * b.g[0]
    else:
        codes, scales = fp4_ref.byte_places("k", slot % 16, b.d)
        rec = b.k[slot // b.bs, :, slot % b.bs // 16]
        rec[:, codes[0]], rec[:, scales[0]] = 7, 0x38  # 6 * 1
        at = 6.0 * b.g[0]
    b.q[...] = 0
    grp = b.hq // b.hkv
    for h in range(b.hkv):
        b.q[:, h * grp:(h + 1) * grp, 0] = logit / (b.scale * float(at[h]))


def spoil(b, which, slot, head):
    """A NaN in dim 21 of a slot's K or V row (fp4: in its block of 16 dims); returns the dims."""
    c = (b.k, b.v)[which]
    if b.kind == "bf16":
        c.view(-1, b.hkv, b.d)[slot, head, 21] = float("nan")
    elif b.kind == "fp8":
        c.reshape(-1, b.hkv, b.d)[slot, head, 21] = 0x7F
    else:
        _, scales = fp4_ref.byte_places("kv"[which], slot % 16, b.d)
        c[slot // b.bs, head, slot % b.bs // 16, scales[1]] = 0x7F
        return slice(16, 32)
    return slice(21, 22)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,out", [(HYBRID, "f32"), (DENSE, "bf16")])
@pytest.mark.parametrize("n,own_splits,prefix_splits", [(3, 2, 4), (3, 2, 12), (14, 1, 1), (14, 2, 12), (14, 12, 0)])
def test_nan_far_below_the_largest_logit(kind, shape, out, own_splits, prefix_splits, n):
    """A NaN whose split's largest logit is so far below the row's that its weight is 0 in binary32 (2^-289) is NaN
    all the same: by each of the merges, which differ by the numbers of splits and rows (14 x 24: more than two per
    SM), and for any place of the large logit."""
    pre = 768
    for large, low in ((700, 20), (pre + 80, 300), (300, pre + 80)):  # tokens; those past 768 of sequence 2 alone
        b = Batch(n, [(pre, [100 + i for i in range(n)])], *shape, 16, kind, out)
        only_key(b, int(b.slots(2)[large]), 200.0)
        ref, tol = b.reference()
        g = b.hq // b.hkv
        who = slice(2, 3) if low >= pre else slice(0, n)
        bad = np.zeros((b.n, b.hq, b.d), bool)
        bad[who, g:2 * g] = True                                                 # a NaN key: the whole rows
        spoil(b, 0, int(b.slots(2)[low]), 1)
        bad[who, 2 * g:3 * g, spoil(b, 1, int(b.slots(2)[low + 16]), 2)] = True  # a NaN value: its dims
        got = b.run(desc=b.desc(num_splits=own_splits), shared=b.shared(prefix_splits=prefix_splits)).cpu()
        assert torch.isnan(got[torch.from_numpy(bad)]).all()
        check(got[torch.from_numpy(~bad)], ref[~bad], tol[~bad])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,out", [(HYBRID, "f32"), (DENSE, "bf16")])
@pytest.mark.parametrize("n,own_splits,prefix_splits", [(3, 2, 4), (3, 2, 12), (3, 3, 0), (14, 1, 1), (14, 2, 12), (14, 12, 0)])
def test_bad_pages_beside_nan(kind, shape, out, own_splits, prefix_splits, n):
    """A sequence with a bad page is a zero row, also where another of its splits has a NaN."""
    pre = 768
    b = Batch(n, [(pre, [100 + i for i in range(n)])], *shape, 16, kind, out)
    ref, tol = b.reference()
    g = b.hq // b.hkv
    bad = np.zeros((b.n, b.hq, b.d), bool)
    bad[:, g:2 * g, spoil(b, 1, int(b.slots(0)[40]), 1)] = True  # a value of the prefix
    t = b.tensors()
    t["table"][1, pre // 16 + 3] = 10 ** 6                       # a page of sequence 1's own part
    ref[1], tol[1], bad[1] = 0, 0, False
    run = lambda t: b.run(t, desc=b.desc(num_splits=own_splits), shared=b.shared(prefix_splits=prefix_splits), status=status).cpu()  # noqa: E731
    status = status0()
    got = run(t)
    assert torch.isnan(got[torch.from_numpy(bad)]).all()
    check(got[torch.from_numpy(~bad)], ref[~bad], tol[~bad])
    assert int(status) == pa.PA_DEV_BAD_PAGE
    if prefix_splits:  # the prefix itself
        t = b.tensors()
        t["table"][0, pre // 16 - 2] = -1
        check(run(t), np.zeros_like(ref), np.zeros_like(tol))


# -- groups that make no sense ---------------------------------------------------------------------

BOTH = pytest.mark.parametrize("splits", [0, 2], ids=["plain", "shared"])


@BOTH
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("end", [7, 37, 2 ** 31 - 1])
def test_a_start_past_the_sequences(end, kind, splits):
    """The last group ends with the sequences, whatever its end says; a group past them is empty."""
    b = Batch(4, [(112, [3, 20, 1, 60]), (32, [5, 9])], *HYBRID, 16, kind)
    t, status = b.tensors(), status0()
    t["starts"] = torch.tensor([0, 4, end, end, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    got = b.run(t, shared=b.shared(num_groups=4, max_group_seqs=40, prefix_splits=splits), status=status)
    check(got, *b.reference())
    assert int(status) == 0
    # ... and a sequence there that no one else of its group is in front of
    t["starts"] = torch.tensor([0, 5, end], dtype=torch.int32, device="cuda")
    ref, tol = b.reference()
    ref[4], tol[4] = 0, 0  # (of the first group now, and not with its prefix)
    check(b.run(t, shared=b.shared(num_groups=2, max_group_seqs=40, prefix_splits=splits), status=status), ref, tol)
    assert int(status) == pa.PA_DEV_BAD_SEQLEN





@BOTH
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("change,bad", [
    (dict(lens={0: 100}), {0}), (dict(lens={0: 1}), {0}), (dict(lens={0: 100, 1: 111}), {0, 1}), (dict(prefix={0: 10 ** 9}), {0}),
    (dict(lens={0: 0, 1: 50}), {0, 1}), (dict(lens={0: -1, 1: 50}), {0, 1}), (dict(lens={0: 5, 1: 5, 2: 5, 3: 5}), {0, 1, 2, 3}),
    (dict(lens={4: 31}), {4})])
def test_a_leader_shorter_than_its_prefix(change, bad, kind, splits):
    """It is a zero row itself; the others of its group, whose lengths make sense, are computed."""
    b = Batch(4, [(112, [3, 20, 1, 60]), (32, [5, 9])], *HYBRID, 16, kind)
    ref, tol = b.reference()
    ref[list(bad)], tol[list(bad)] = 0, 0
    t = b.tensors()
    for name, values in change.items():
        for i, v in values.items():
            t[name][i] = v
    status = status0()
    check(b.run(t, status=status, prefix_splits=splits), ref, tol)
    assert int(status) == pa.PA_DEV_BAD_SEQLEN


# -- lengths ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_a_bound_of_two_to_the_31_tokens(kind, num_splits):
    """A description for sequences of any length (max_seq_len nearly 2^31, no hints), a prefix of 1.2 million tokens:
    prefix and planned splits end past token 2^31 together.  Two keys, one of the prefix and one of the own part, have
    a logit of 30, the others 0: the output is the mean of their values, but for 1.2e6 e^-30 = 1.1e-7 of the others."""
    bs, width, d, hq, prefix = 2 ** 20, 2047, 128, 4, 1200005
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    gen = torch.Generator(device="cuda").manual_seed(5)
    k = torch.zeros((2, bs, 1, d), dtype=torch.uint8 if kind == "fp8" else dtype, device="cuda")
    v = torch.randn((2, bs, 1, d), generator=gen, device="cuda", dtype=torch.bfloat16).to(dtype)
    a, b = 777777, prefix + 21
    flat = k.view(dtype).view(2 * bs, d)
    flat[a, 0] = flat[b, 0] = 8.0
    q = torch.zeros((1, hq, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 30 * d ** 0.5 / 8
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.ones((1, width), dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    desc = pa.make_desc(num_seqs=1, num_q_heads=hq, num_kv_heads=1, head_dim=d, block_size=bs, max_pages_per_seq=width,
                        max_seq_len=width * bs, num_pages=2, scale=d ** -0.5, num_splits=num_splits)
    shared = pa.make_prefix(num_groups=1, max_group_seqs=1, prefix_splits=8)
    ws = torch.empty(pa.shared_workspace_bytes(desc, shared), dtype=torch.uint8, device="cuda")
    out, status = torch.empty((1, hq, d), device="cuda"), status0()
    args = (table, i32(prefix + 37), i32(0, 1), i32(prefix), desc, shared, out, ws, status)
    if kind == "bf16":
        pa.paged_attention_decode_shared(q, k, v, *args)
    else:
        one = torch.ones(1, device="cuda")
        pa.paged_attention_decode_shared_fp8(q, k, v.view(torch.uint8), one, one, *args)
    rows = v.view(2 * bs, d)
    want = ((rows[a].double() + rows[b].double()) / 2).cpu()
    # the two weights are the same number; sums and merges as in shared_ref for what has weight, 64 * 2^-23 of |v| < 6
    assert (out[0].double().cpu() - want).abs().max() < 6 * (2 * 1.2e-7 + 64 * 2.0 ** -23)
    assert int(status) == 0


# -- what the weights lose -------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [HYBRID, DENSE, (48, 4, 256), (32, 2, 128)])
@pytest.mark.parametrize("n,own_splits", [(3, 0), (3, 1), (40, 1)])
def test_plain_reads_keep_the_decodes_weights(shape, n, own_splits):
    """bf16 outputs over an e4m3 cache, read without sharing: as exact as the decode that such a call stands for.  All
    keys but one, whose value is 0, have the same logit and the same value, so what a weight loses as it enters the
    product does not average out."""
    b = Batch(n, [(64, [150 + i % 7 for i in range(n)])], *shape, 16, "fp8", "bf16")
    slot = int(b.slots(0)[20])
    only_key(b, slot, 4.0)
    b.q[:, :, 0] *= torch.linspace(0.7, 1.4, b.n * b.hq).reshape(b.n, b.hq).to(torch.bfloat16)
    b.v[...] = np.random.default_rng(n).integers(0x20, 0x7F, (b.hkv, b.d))
    b.v.reshape(-1, b.hkv, b.d)[slot] = 0
    ref, _ = b.reference()
    # A logit is one product: exact, then scaled in three roundings of 2^-24 of at most 1.45 * 5.6 log2 units, 1.5e-6
    # of a weight; exp2 2^-22 and two f16 numbers 2^-22 of it, and of the sum; 250 keys' sums and merges as in
    # shared_ref, (250 / 16 + 64) * 2^-23.  One f16 would be off by up to 2^-11, 4.9e-4.
    rel = 2 * (1.5e-6 + 2.0 ** -22 + 2.0 ** -22) + (250 / 16 + 64) * 2.0 ** -23
    half_step = np.exp2(np.floor(np.log2(np.abs(ref))) - 8)
    t, desc = b.tensors(), b.desc(num_splits=own_splits)
    check(b.run(t, desc=desc), ref, half_step + rel * np.abs(ref))
    out, ws = torch.empty_like(t["q"]), torch.empty(max(1, pa.workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
    pa.paged_attention_decode_fp8(t["q"], *t["caches"], *t["scales"], t["table"], t["lens"], desc, out, ws)
    check(out, ref, half_step + rel * np.abs(ref))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,d", [(4, 256), (12, 256), (16, 256), (4, 128), (12, 128), (16, 128)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_scores_rise_while_values_fall(kind, hq, d, out):
    """Logits rise in 16 levels along the prefix and again along the own parts, and the values fall as the weights grow:
    every level carries as much of the output, so a sum that is rescaled wrongly, one that was moved aside among them
    (each stream of the longest own part moves its sums several times, with the maximum raised between), shows."""
    prefix, own = 2600, [3900, 40, 2100]
    b = Batch(d + hq, [(prefix, own)], hq, 1, d, 16, kind, out)
    reach = 40.0 if kind == "bf16" else 16.0  # log2 units; e4m3 values and fp4 scales span 17 binades
    rng = np.random.default_rng(hq)
    b.q[...] = 0
    b.k[...] = 0
    unit = 1.0 if b.g is None else float(b.g[0][0])
    b.q[:, :, 0] = (reach / 15 * np.log(2) / (b.scale * unit) * (1 + torch.arange(hq) / 256)).to(torch.bfloat16)
    for s in range(b.n):
        slots = b.slots(s)
        t = np.arange(len(slots))
        level = np.where(t < prefix, 16 * t // prefix, 16 * (t - prefix) // own[s])
        down = np.round(level * reach / 15)
        if kind == "fp4":
            for at in range(16):
                mine = slots[slots % 16 == at]
                n, dn = level[slots % 16 == at], down[slots % 16 == at]
                (kc, ks), (_, vs) = (fp4_ref.byte_places(w, at, d) for w in "kv")
                where = (mine // 16, 0, mine % 16 // 16)
                b.k[where + (kc[0],)] = 2  # 1.0, times the level as the block's scale
                b.k[where + (ks[0],)] = torch.from_numpy(n.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                scale = torch.from_numpy(np.exp2(8 - dn).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                for place in vs:
                    b.v[where + (place,)] = scale
            continue
        v = torch.from_numpy((rng.standard_normal((len(t), d)) * np.exp2(6 - down)[:, None]).astype(np.float32)).clamp(-448, 448)
        if kind == "bf16":
            b.k.view(-1, d)[slots, 0] = torch.from_numpy(level.astype(np.float32)).to(torch.bfloat16)
            b.v.view(-1, d)[slots] = v.to(torch.bfloat16)
        else:
            b.k.reshape(-1, d)[slots, 0] = torch.from_numpy(level.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            b.v.reshape(-1, d)[slots] = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # A logit is one product: exact, then at most four roundings of 2^-24 of it.  exp2 2^-22; the numbers a weight
    # enters the product as, as in shared_ref (one f16 for bf16 outputs over e4m3, too: 2^-11), and what f16 loses
    # below 2^-32 of the largest weight; the sums over keys and the merges and rescales as there.
    weight = 2.0 ** -17 if kind == "bf16" else 2.0 ** -11 if out == "bf16" else 2.0 ** -21
    ref, tol = np.zeros((b.n, hq, d)), np.zeros((b.n, hq, d))
    for s in range(b.n):
        k, v = (b.rows(w, b.slots(s))[:, 0] for w in (0, 1))
        x = b.q[s, :, :1].double().numpy() * k[:, 0] * b.scale
        w = np.exp(x - x.max(-1, keepdims=True))
        total = w.sum(-1, keepdims=True)
        ref[s], mag = w / total @ v, w / total @ np.abs(v)
        rel = 2.02 * 4 * 2.0 ** -24 * x.max() + 2 * (weight + 2.0 ** -22) + (len(k) / 16 + 64) * 2.0 ** -23
        tol[s] = rel * mag + (0 if kind == "bf16" else np.minimum(w, 2.0 ** -32) / total @ np.abs(v))
    if out == "bf16":
        tol += np.abs(ref) * 2.0 ** -8
    for prefix_splits, num_splits in ((1, 1), (3, 2), (0, 1), (0, 0)):
        check(b.run(desc=b.desc(num_splits=num_splits), shared=b.shared(prefix_splits=prefix_splits)), ref, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("groups,prefix_splits,num_splits", [([(38000, [1, 1])], 4, 1), ([(38000, [1, 1])], 1, 1),
                                                             ([(16, [6000, 1, 5000])], 1, 1)])
def test_fp32_outputs_lose_a_millionth(kind, d, groups, prefix_splits, num_splits):
    """Normal rows: the error of fp32 outputs, relative to their norm, over tens of thousands of keys with and without
    splits.  A score is two sums of 8 steps (D = 256) that each cut off half of 2^-23 of a sum that is half of a half
    of the score on average; where weights matter scores reach 4: 16 / 2 * 2^-23 * 1 = 0.95e-6.  The sums over keys
    lose 2.4e-9 per key up to 192 keys, 0.46e-6, then move.  exp2, the weights' numbers and the sums of binary32, 2^-22
    each at most and of any sign, average out.  Together 1.4e-6; twice what is promised, 2e-6, is allowed.  (Scores in
    one sum: 2.4e-6; sums that stay where they are: 2.4e-9 * 38,000 / 2 = 4.6e-5.)"""
    b = Batch(d, groups, 4, 1, d, 16, kind)
    ref, _ = b.reference()
    got = b.run(desc=b.desc(num_splits=num_splits), shared=b.shared(prefix_splits=prefix_splits)).double().cpu().numpy()
    assert np.linalg.norm(got - ref) < 2e-6 * np.linalg.norm(ref)


def awkward_distances(unit, n):
    """bf16 numbers q0 whose weight p = 2^-(q0 * unit) leaves most behind after two bf16 numbers: 2.5e-6 of it or more."""
    q0 = torch.arange(1, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    q0 = q0[torch.isfinite(q0)]
    y = q0.double() * unit
    q0, y = q0[(y > 1) & (y < 3)], y[(y > 1) & (y < 3)]
    p = torch.exp2(-y)
    head = p.to(torch.bfloat16).double()
    left = (p - head - (p - head).to(torch.bfloat16).double()).abs() / p
    order = left.argsort(descending=True)[:n]
    assert left[order[0]] > 2.8e-6
    return q0[order]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("prefix_splits", [0, 1], ids=["plain", "shared"])
def test_fp32_outputs_keep_the_weights_bits(kind, d, prefix_splits):
    """63 keys of one logit and one value beside one key with a larger logit and the value 0, so that what a weight
    loses as it enters the product stays in the output, with weights for which two bf16 numbers lose 2.5e-6 and more.
    Allowed: the product's 4 steps of 16 keys for each of three numbers cut off 2^-23 of the sum so far, 3 * (1 + 2 + 3
    + 4) / 4 * 2^-23 = 0.9e-6; the weights themselves are summed in binary32, in two chains of 32 equal ones at most,
    whose j-th sum is rounded by 2^-24 of its j weights, (2 + 3 + .. + 32) / 32 * 2^-24 = 0.98e-6; the weight, 1 to 8
    times in 64 of the sum, is off by 0.6e-6, a ninth of which stays; six roundings of the merges, 2^-24 each: 2.3e-6
    in all."""
    b = Batch(1, [(64, [0, 0])], 8, 1, d, 16, kind)
    only_key(b, int(b.slots(0)[0]), 1.0)
    at = 8.0 if kind == "bf16" else 8.0 * float(b.g[0][0])
    b.q[...] = 0
    b.q[:, :, 0] = awkward_distances(at * b.scale / np.log(2), 16).view(2, 8)
    if kind == "bf16":
        b.v[...] = (torch.arange(d) / 64 + 1).to(torch.bfloat16)
        b.v.view(-1, d)[int(b.slots(0)[0])] = 0
    else:
        b.v[...] = 0x30 + np.arange(d) % 64
        b.v.reshape(-1, d)[int(b.slots(0)[0])] = 0
    ref, _ = b.reference()
    check(b.run(prefix_splits=prefix_splits), ref, 2.3e-6 * np.abs(ref))
