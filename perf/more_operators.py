"""The operators of a batch of requests forked from common prompts, as cases that
can be run and timed: rotary positions with the cache write behind them, cache
pages with several holders (fork, release, compaction, copies), and decode
attention that reads a prefix shared by a group of sequences once.

Each case runs one pass through one operator, in one of two forms:

* the plain form (``own`` false): elementary torch operations in 32 bits (angles
  in 64), rounded once at the end;
* the library's own calls (``own`` true), as a serving loop makes them.
"""
import math

import torch

own = False

_DEV = "cuda"
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# -- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the decode step of a batch: a token per request rotated and written, a quarter of each head rotates; latency
        dict(name="rope_step", op="rope", back=False, n=32, hq=24, hkv=4, d=256, r=64, inter=False, scaling="none",
             factor=1.0, orig=0, pmax=32768, cache="bf16", bs=784, fused=True),
        # a wave of prompt chunks beside a long context (scaled positions), rows read in place from the q/k/v projection
        dict(name="rope_prompt", op="rope", back=False, n=16411, hq=24, hkv=4, d=256, r=64, inter=False,
             scaling="yarn", factor=4.0, orig=32768, pmax=131072, cache="bf16", bs=784, fused=True),
        # the dense model, whole heads in the interleaved layout, into an e4m3 cache; far positions
        dict(name="rope_e4m3", op="rope", back=False, n=2051, hq=32, hkv=8, d=128, r=128, inter=True, scaling="bands",
             factor=8.0, orig=8192, pmax=1000000, cache="e4m3", bs=16, fused=False),
        # the gradients of a training step's queries and keys
        dict(name="rope_back", op="rope", back=True, n=8192, hq=32, hkv=8, d=128, r=128, inter=False, scaling="none",
             factor=1.0, orig=0, pmax=8192, cache="bf16", bs=16, fused=False),
        # one request forked into four samples: tables, holders, the partly filled last page copied; latency
        dict(name="fork_step", op="fork", b=8, parents=1, kids=4, bs=16, hkv=8, d=128, cache="bf16", layers=1,
             len_hi=500, finished=0, short=False),
        # a scheduler step: finished samples leave, prompts fork into their slots, last pages copied in two layers
        dict(name="fork_wave", op="fork", b=256, parents=24, kids=8, bs=784, hkv=4, d=256, cache="bf16", layers=2,
             len_hi=6000, finished=150, short=False),
        # a pool of small pages compacted before it is shrunk: up to 4096 pages move in a step
        dict(name="compact", op="compact", b=100, bs=16, hkv=8, d=128, cache="e4m3", pages=40000, len_hi=4000,
             moves=4096),
        # four short samples of one prompt: all launch latency
        dict(name="shared_small", op="shared", cache="bf16", b=4, groups=1, p_lo=512, p_hi=512, s_hi=40, hq=24, hkv=4,
             d=256, bs=16, out="f32"),
        # a full serving batch behind one long system prompt
        dict(name="shared_batch", op="shared", cache="bf16", b=64, groups=1, p_lo=32768, p_hi=32768, s_hi=1500, hq=24,
             hkv=4, d=256, bs=784, out="bf16"),
        # rollouts: several samples of each of 16 prompts, dense model on small pages
        dict(name="shared_groups", op="shared", cache="bf16", b=128, groups=16, p_lo=1024, p_hi=8192, s_hi=2000, hq=32,
             hkv=8, d=128, bs=16, out="f32"),
        # one document, many questions, wide groups, over an e4m3 cache
        dict(name="shared_e4m3", op="shared", cache="e4m3", b=33, groups=1, p_lo=16640, p_hi=16640, s_hi=3000, hq=48,
             hkv=4, d=256, bs=832, out="bf16"),
        # uneven groups behind long prompts over an fp4 cache
        dict(name="shared_fp4", op="shared", cache="fp4", b=40, groups=5, p_lo=8000, p_hi=24000, s_hi=2000, hq=24,
             hkv=4, d=256, bs=784, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(24, 4, 256), (48, 4, 256), (32, 8, 128), (6, 1, 256), (8, 8, 128), (20, 4, 256), (32, 2, 128), (10, 2, 256)]


def draw(rng):
    op = rng.choice(["rope", "rope", "fork", "compact", "shared", "shared", "shared"])
    hq, hkv, d = rng.choice(_HEADS)
    bs = rng.choice([16, 48, 64, 784, 832])
    if op == "rope":
        scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        r = rng.choice([d, d, d // 2, d // 4, 16 * rng.randint(1, d // 16)])
        return dict(op="rope", back=rng.random() < 0.3, n=_log_int(rng, 1, 12000), hq=hq, hkv=hkv, d=d, r=r,
                    inter=rng.random() < 0.5, scaling=scaling, factor=rng.choice([2.0, 4.0, 8.0]), orig=8192,
                    pmax=_log_int(rng, 12001, 2000000), cache=rng.choice(["bf16", "bf16", "e4m3"]), bs=bs,
                    fused=rng.random() < 0.5)
    if op == "fork":
        parents, kids = _log_int(rng, 1, 24), _log_int(rng, 1, 8)
        return dict(op="fork", b=parents * (kids + 1) + _log_int(rng, 1, 200), parents=parents, kids=kids, bs=bs,
                    hkv=hkv, d=d, cache=rng.choice(["bf16", "e4m3", "fp4"]), layers=rng.randint(1, 2),
                    len_hi=_log_int(rng, 20, 6000), finished=_log_int(rng, 1, 150), short=rng.random() < 0.3)
    if op == "compact":
        pages = _log_int(rng, 64, 40000) if bs <= 64 else _log_int(rng, 64, 500)
        if bs == 64:
            pages = min(pages, 8000)
        return dict(op="compact", b=_log_int(rng, 1, 300), bs=bs, hkv=min(hkv, 4), d=d,
                    cache=rng.choice(["bf16", "e4m3", "fp4"]), pages=pages, len_hi=_log_int(rng, 16, 4000),
                    moves=_log_int(rng, 1, 4096 if bs <= 64 else 200))
    p_hi = _log_int(rng, bs, 32768)
    b = min(_log_int(rng, 1, 128), max(1, 1_500_000 * 4 * 256 // ((p_hi + 1000) * hkv * d)))
    return dict(op="shared", cache=rng.choice(["bf16", "e4m3", "fp4"]), b=b, groups=rng.randint(1, max(1, b // 4)),
                p_lo=rng.choice([bs, p_hi // 2, p_hi]), p_hi=p_hi, s_hi=_log_int(rng, 1, 3000), hq=hq, hkv=hkv, d=d, bs=bs,
                out=rng.choice(["f32", "bf16"]))


# -- caches --------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed)


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device=_DEV)


def _perm(gen, n):
    return torch.randperm(n, generator=gen, device=_DEV)


def _rows(gen, shape):
    """bf16 K or V rows: normal, with every 32nd channel eight times as large, as K caches have them."""
    x = torch.randn(shape, generator=gen, device=_DEV, dtype=torch.bfloat16)
    x[..., 7::32] *= 8.0
    return x


def _scales(kind, hkv):
    h = torch.arange(hkv, device=_DEV, dtype=torch.float32)
    if kind == "fp4":
        return (1 + h / 4) / 96, (1 + h / 8) / 80
    return (1 + h / 4) / 16, (1 + h / 8) / 12


def _fill(gen, kind, pages, bs, hkv, d):
    """A cache of rows as they stand after a quantising write: bf16 values, e4m3 codes, or fp4 records of 9 d bytes
    for 16 tokens of a KV head (8 d code bytes, then d scale bytes; every byte's place is taken up in `_offsets`)."""
    if kind == "bf16":
        return _rows(gen, (pages, bs, hkv, d))
    if kind == "e4m3":
        return (_rows(gen, (pages, bs, hkv, d)) * 8).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    shape = (pages, hkv, bs // 16)
    rec = torch.empty(shape + (9 * d,), dtype=torch.uint8, device=_DEV)
    # a block's largest element has code 6, the others are spread as a normal's values are beside its largest of 16
    x = torch.randn(shape + (16 * d,), generator=gen, device=_DEV, dtype=torch.bfloat16).mul_(3.4)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=_DEV, dtype=torch.bfloat16)
    code = torch.bucketize(x.abs(), edges, out_int32=True).byte() | (torch.signbit(x).byte() << 3)
    rec[..., :8 * d] = code[..., ::2] | (code[..., 1::2] << 4)
    s = torch.randn(shape + (d,), generator=gen, device=_DEV).mul_(0.35).exp_().mul_(28.0)
    rec[..., 8 * d:] = s.clamp_(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return rec


def _offsets(d):
    """Byte positions inside a 16-token record: code byte m (dims 2m, 2m + 1)
    and scale byte blk (dims 16 blk ..) of each token, for K and for V."""
    t = torch.arange(16, device=_DEV)[:, None]
    m = torch.arange(d // 2, device=_DEV)[None]
    blk = torch.arange(d // 16, device=_DEV)[None]
    half, r = t // 8, t % 8
    i, j = (m // 8) % 8, m // 64
    k_code = (2 * j + half) * 512 + (4 * r + (m % 8) // 2) * 16 + 2 * i + m % 2
    k_scale = 8 * d + t * (d // 16) + blk
    c, u = (t % 8) // 2, 2 * half + t % 2
    v_code = u * 2 * d + (4 * (m % 8) + c) * (d // 16) + m // 8
    v_scale = 8 * d + (blk // 4) * 64 + c * 16 + (blk % 4) * 4 + u
    return (k_code, k_scale), (v_code, v_scale)


# -- inputs --------------------------------------------------------------------------------------

def prepare(case, seed):
    return {"rope": _prepare_rope, "fork": _prepare_fork, "compact": _prepare_compact,
            "shared": _prepare_shared}[case["op"]](case, seed)


def _frequencies(case):
    """Radians per position of each pair of a head, float64 [r / 2], and the factor on the rotated values."""
    r, factor, orig, base = case["r"], case["factor"], case["orig"], _base(case)
    j = torch.arange(r // 2, device=_DEV, dtype=torch.float64)
    if case["scaling"] == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2))
    w = base ** (-2.0 * j / r)
    if case["scaling"] == "linear":
        return w / factor, 1.0
    if case["scaling"] == "yarn":
        at = lambda turns: r * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = ((j - low) / max(high - low, 0.001)).clamp(0, 1)
        return w / factor * ramp + w * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "bands":
        turns = orig * w / (2 * math.pi)
        mix = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return w / factor * (1 - mix) + w * mix, 1.0
    return w, 1.0


def _base(case):
    return 10000.0 if case["pmax"] <= 32768 else 1000000.0


def _prepare_rope(case, seed):
    gen, n, hq, hkv, d, bs = _gen(seed), case["n"], case["hq"], case["hkv"], case["d"], case["bs"]
    if case["fused"]:  # rows of the projection's output, q, k and v of a token side by side
        rows = _rows(gen, (n, hq + 2 * hkv, d))
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    else:
        q, k, v = _rows(gen, (n, hq, d)), _rows(gen, (n, hkv, d)), _rows(gen, (n, hkv, d))
    if n <= 64:  # a decode step: every request at a place of its own
        pos = _ints(gen, 0, case["pmax"] - 1, n)
    else:
        pos = torch.arange(n, device=_DEV) + _ints(gen, 0, case["pmax"] - n, 1)
    state = dict(case=case, q=q, k=k, v=v, pos=pos.int(), q_out=torch.empty((n, hq, d), dtype=torch.bfloat16, device=_DEV))
    if case["back"]:
        state["k_out"] = torch.empty((n, hkv, d), dtype=torch.bfloat16, device=_DEV)
    else:
        pages = -(-n * 9 // (8 * bs)) + 2
        slots = (_perm(gen, pages)[:, None] * bs + torch.arange(bs, device=_DEV)).flatten()[3:n + 3].contiguous()
        if n > 64:
            slots[_ints(gen, 0, n - 1, 5)] = -1  # padding rows
        kind = torch.uint8 if case["cache"] == "e4m3" else torch.bfloat16
        state |= dict(slots=slots, k_cache=torch.zeros((pages, bs, hkv, d), dtype=kind, device=_DEV),
                      v_cache=torch.zeros((pages, bs, hkv, d), dtype=kind, device=_DEV),
                      one=torch.ones(hkv, device=_DEV))
    if own:
        import paged_attention_decode_split_gb300 as pa
        state["freqs"], state["factor"] = pa.rotary_frequencies(
            case["r"], base=_base(case), scaling=case["scaling"], factor=case["factor"], original_len=case["orig"])
    else:
        state["freqs"], state["factor"] = _frequencies(case)
    return state


def _tables(gen, lens, shared, first_of, bs, width, pages):
    """Block tables of requests of lens tokens, the first shared[b] pages of which are those of request first_of[b],
    over a shuffled pool; returns the table and the pool in the order in which it was dealt."""
    lp = torch.arange(width, device=_DEV)[None]
    used = -(-lens // bs)
    mine = (used - shared).clamp(min=0)  # pages of a request's own; the first of a group also owns the shared ones
    leader = first_of == torch.arange(len(lens), device=_DEV)
    mine = torch.where(leader, used, mine)
    start = (mine.cumsum(0) - mine)[:, None]
    pool = _perm(gen, pages)
    at = torch.where(leader[:, None], start + lp, start + lp - shared[:, None])
    table = torch.where(lp < used[:, None], pool[at.clamp(0, pages - 1)], -1)
    table = torch.where(lp < torch.minimum(shared, used)[:, None], table[first_of], table)
    return table.int(), pool.int(), int(mine.sum())


def _holders(table, lens, bs, pages):
    lp = torch.arange(table.shape[1], device=_DEV)[None]
    n = torch.bincount(table[lp < -(-lens // bs)[:, None]].long(), minlength=pages)
    return (n - 1).clamp(min=0).int()


def _spread(gen, lo, hi, n):
    """n whole numbers spread evenly over lo .. hi, in random order."""
    return lo + _perm(gen, n) * (hi - lo) // max(1, n - 1)


def _prepare_fork(case, seed):
    gen, b, bs, hkv, d = _gen(seed), case["b"], case["bs"], case["hkv"], case["d"]
    place = _perm(gen, b)
    kid = torch.full((b,), -1, device=_DEV)
    kid[place[case["parents"]:case["parents"] * (case["kids"] + 1)]] = place[:case["parents"]].repeat_interleave(case["kids"])
    lens = _spread(gen, 1, case["len_hi"], b)
    used = int((-(-lens // bs)).sum())  # (the same for every seed)
    # the others go on, in pairs that were forked before and share their first pages; some have finished
    first_of = torch.arange(b, device=_DEV)
    rest = place[case["parents"] * (case["kids"] + 1):]
    first_of[rest[1::2]] = rest[:-1:2][:len(rest[1::2])]
    finished = torch.zeros(b, dtype=torch.int32, device=_DEV)
    finished[rest[:case["finished"]]] = 1
    # the slots of the children-to-be are idle, or fall idle in the call before
    before = kid >= 0
    if case["finished"]:
        finished[before] = 1
    else:
        lens = torch.where(before, 0, lens)
    shared = torch.where(first_of != torch.arange(b, device=_DEV), torch.minimum(lens, lens[first_of]) // bs, 0)
    width = -(-case["len_hi"] // bs) + 1
    spare = case["parents"] * case["kids"] + 7
    if case["short"]:
        spare = max(1, spare // 3)
    pages = used + spare + 5
    table, pool, held = _tables(gen, lens, shared, first_of, bs, width, pages)
    free = torch.full((pages,), -1, dtype=torch.int32, device=_DEV)
    free[:spare] = pool[held:held + spare]
    i32 = dict(dtype=torch.int32, device=_DEV)
    empty = lambda n: torch.empty(n, **i32)  # noqa: E731
    return dict(case=case, lens=lens.int(), parent=kid.int(), finished=finished, table=table, free=free,
                num_free=torch.tensor([spare], **i32), shares=_holders(table, lens, bs, pages),
                lens_mid=empty(b), shares_mid=empty(pages), num_mid=empty(1), lens_out=empty(b), shares_out=empty(pages),
                num_out=empty(1), src=empty(b), dst=empty(b), tokens=empty(b),
                caches=[_fill(gen, case["cache"], pages, bs, hkv, d) for _ in range(2 * case["layers"])])


def _prepare_compact(case, seed):
    gen, b, bs, hkv, d, pages = _gen(seed), case["b"], case["bs"], case["hkv"], case["d"], case["pages"]
    most = max(1, min(case["len_hi"], (pages // (2 * b)) * bs))
    lens = _spread(gen, 0, most, b)
    number = torch.arange(b, device=_DEV)
    first_of = number // 4 * 4  # requests in fours share a third of their pages
    shared = torch.where(first_of != number, torch.minimum(lens, lens[first_of]) // (3 * bs), 0)
    width = -(-most // bs) + 1
    if b * -(-most // bs) > pages:  # more requests than pages: those past the pool are idle
        lens = torch.where(number < pages // (-(-most // bs)), lens, 0)
        shared = torch.minimum(shared, lens // bs)
    table, pool, held = _tables(gen, lens, shared, first_of, bs, width, pages)
    free = torch.full((pages,), -1, dtype=torch.int32, device=_DEV)
    free[:pages - held] = pool[held:]
    i32 = dict(dtype=torch.int32, device=_DEV)
    empty = lambda n: torch.empty(n, **i32)  # noqa: E731
    return dict(case=case, lens=lens.int(), table=table, free=free, num_free=torch.tensor([pages - held], **i32),
                shares=_holders(table, lens, bs, pages), free_out=empty(pages), num_out=empty(1), shares_out=empty(pages),
                page_map=empty(pages), src=empty(case["moves"]), dst=empty(case["moves"]), extent=empty(1),
                caches=[_fill(gen, case["cache"], pages, bs, hkv, d) for _ in range(2)])


def _group_starts(case):
    return [case["b"] - int(case["b"] * (1 - g / case["groups"]) ** 1.3) for g in range(case["groups"])] + [case["b"]]


def _prepare_shared(case, seed):
    gen, b, hkv, d, bs = _gen(seed), case["b"], case["hkv"], case["d"], case["bs"]
    starts = torch.tensor(_group_starts(case), device=_DEV)
    size = starts[1:] - starts[:-1]
    prefix = (_spread(gen, case["p_lo"], case["p_hi"], case["groups"]) // bs * bs).repeat_interleave(size)
    first_of = starts[:-1].repeat_interleave(size)
    lens = prefix + _spread(gen, 1, case["s_hi"], b)
    if b > 8:
        lens[_ints(gen, 0, b - 1, 1)] = 0  # an idle slot
    prefix_of = prefix
    # the pages of the prefix are the group's first request's (dealt to it even where that slot is idle now)
    dealt = torch.where(lens == 0, prefix + 1, lens)
    width = -(-(case["p_hi"] + case["s_hi"]) // bs)
    pages = int((-(-dealt // bs) - prefix // bs).sum()) + int((prefix // bs)[starts[:-1].clamp(max=b - 1)].sum()) + 3
    table, _, _ = _tables(gen, dealt, prefix // bs, first_of, bs, width, pages)
    ks, vs = _scales(case["cache"], hkv)
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    state = dict(case=case, q=torch.randn((b, case["hq"], d), generator=gen, device=_DEV).to(torch.bfloat16),
                 k_cache=_fill(gen, case["cache"], pages, bs, hkv, d), v_cache=_fill(gen, case["cache"], pages, bs, hkv, d),
                 k_scale=ks, v_scale=vs, table=table, lens=lens.int(), starts=starts.int(), prefix=prefix_of.int(),
                 scale=1.0 / math.sqrt(d), out=torch.empty((b, case["hq"], d), dtype=dtype, device=_DEV))
    if case["cache"] == "fp4":
        state["off"] = _offsets(d)
    if own:
        import paged_attention_decode_split_gb300 as pa
        state["desc"] = pa.make_desc(
            num_seqs=b, num_q_heads=case["hq"], num_kv_heads=hkv, head_dim=d, block_size=bs, max_pages_per_seq=width,
            max_seq_len=case["p_hi"] + case["s_hi"], num_pages=pages, scale=state["scale"],
            out_dtype=pa.PA_OUT_BF16 if case["out"] == "bf16" else pa.PA_OUT_F32)
        state["shared"] = pa.make_prefix(num_groups=case["groups"], max_group_seqs=int(size.max()),
                                         max_prefix_len=case["p_hi"], max_suffix_len=case["s_hi"])
        state["workspace"] = torch.empty(max(1, pa.shared_workspace_bytes(state["desc"], state["shared"])),
                                         dtype=torch.uint8, device=_DEV)
    return state


# -- one pass ------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "fork": _own_fork, "compact": _own_compact, "shared": _own_shared}[op](state)
    return {"rope": _plain_rope, "fork": _plain_fork, "compact": _plain_compact, "shared": _plain_shared}[op](state)


def _rope_outputs(s):
    if s["case"]["back"]:
        return dict(q=s["q_out"], k=s["k_out"])
    if s["case"]["cache"] == "e4m3":  # the codes as the values they stand for (the scales are 1)
        return dict(q=s["q_out"], k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn))
    return dict(q=s["q_out"], k=s["k_cache"], v=s["v_cache"])


def _own_rope(s):
    import paged_attention_decode_split_gb300 as pa
    opts = dict(interleaved=s["case"]["inter"], factor=s["factor"])
    if s["case"]["back"]:
        pa.rotary(s["q"], s["k"], s["pos"], s["freqs"], s["q_out"], s["k_out"], inverse=True, **opts)
    elif s["case"]["cache"] == "e4m3":
        pa.rotary_and_cache_fp8(s["q"], s["k"], s["v"], s["pos"], s["freqs"], s["q_out"], s["k_cache"], s["v_cache"],
                                s["slots"], s["one"], s["one"], **opts)
    else:
        pa.rotary_and_cache(s["q"], s["k"], s["v"], s["pos"], s["freqs"], s["q_out"], s["k_cache"], s["v_cache"],
                            s["slots"], **opts)
    return _rope_outputs(s)


def _own_copy(s, tokens):
    import paged_attention_decode_split_gb300 as pa
    call = pa.copy_cache_pages_fp4 if s["case"]["cache"] == "fp4" else pa.copy_cache_pages
    call(s["caches"], s["src"], s["dst"], tokens)


def _fork_outputs(s):
    return dict(table=s["table"], free=s["free"], lens=s["lens_out"], shares=s["shares_out"], num_free=s["num_out"],
                src=s["src"], dst=s["dst"], tokens=s["tokens"], caches=s["caches"])


def _own_fork(s):
    import paged_attention_decode_split_gb300 as pa
    bs, lens, shares, num = s["case"]["bs"], s["lens"], s["shares"], s["num_free"]
    if s["case"]["finished"]:
        pa.release_shared_block_tables(lens, s["finished"], s["table"], s["free"], num, shares, bs, s["lens_mid"],
                                       s["shares_mid"], s["num_mid"])
        lens, shares, num = s["lens_mid"], s["shares_mid"], s["num_mid"]
    pa.fork_block_tables(lens, s["parent"], s["table"], s["free"], num, shares, bs, s["lens_out"], s["shares_out"],
                         s["src"], s["dst"], s["tokens"], s["num_out"])
    _own_copy(s, s["tokens"])
    return _fork_outputs(s)


def _compact_outputs(s):
    return dict(table=s["table"], free=s["free_out"], num_free=s["num_out"], shares=s["shares_out"], map=s["page_map"],
                src=s["src"], dst=s["dst"], extent=s["extent"], caches=s["caches"])


def _own_compact(s):
    import paged_attention_decode_split_gb300 as pa
    pa.compact_block_tables(s["lens"], s["table"], s["free"], s["num_free"], s["shares"], s["case"]["bs"], s["free_out"],
                            s["num_out"], s["shares_out"], s["page_map"], s["src"], s["dst"], s["extent"])
    _own_copy(s, None)
    return _compact_outputs(s)


def _own_shared(s):
    import paged_attention_decode_split_gb300 as pa
    call = {"bf16": pa.paged_attention_decode_shared, "e4m3": pa.paged_attention_decode_shared_fp8,
            "fp4": pa.paged_attention_decode_shared_fp4}[s["case"]["cache"]]
    scales = () if s["case"]["cache"] == "bf16" else (s["k_scale"], s["v_scale"])
    call(s["q"], s["k_cache"], s["v_cache"], *scales, s["table"], s["lens"], s["starts"], s["prefix"], s["desc"],
         s["shared"], s["out"], s["workspace"])
    return dict(out=s["out"])


def _rotated(x, cos, sin, r, inter):
    """Rows [n, heads, d], the first r dims of each head rotated, fp32."""
    x = x.float()
    part = x[..., :r]
    a, b = (part[..., ::2], part[..., 1::2]) if inter else (part[..., :r // 2], part[..., r // 2:])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rope(s):
    case = s["case"]
    angle = s["pos"].double()[:, None] * s["freqs"]
    if case["back"]:
        angle = -angle
    cos, sin = [(f * s["factor"]).float()[:, None] for f in (angle.cos(), angle.sin())]
    s["q_out"].copy_(_rotated(s["q"], cos, sin, case["r"], case["inter"]))
    k = _rotated(s["k"], cos, sin, case["r"], case["inter"]).to(torch.bfloat16)
    if case["back"]:
        s["k_out"].copy_(k)
        return _rope_outputs(s)
    live = s["slots"] >= 0
    at, k, v = s["slots"][live], k[live], s["v"][live]
    if case["cache"] == "e4m3":
        k, v = [x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v)]
    s["k_cache"].flatten(0, 1)[at] = k
    s["v_cache"].flatten(0, 1)[at] = v
    return _rope_outputs(s)


def _plain_copy(s, tokens):
    """Copies pages src -> dst in every cache: the whole 16-token chunks that hold the first tokens[i] tokens of a page."""
    chunks = s["case"]["bs"] // 16
    want = torch.full_like(s["src"], chunks) if tokens is None else (tokens + 15) // 16
    src, dst = s["src"].long(), s["dst"].long()
    c = torch.arange(chunks, device=_DEV)
    take = (c < want[:, None]) & (src >= 0)[:, None]
    moves = ((src[:, None] * chunks + c)[take], (dst[:, None] * chunks + c)[take])
    [_move_chunks(x, chunks, *moves) for x in s["caches"]]


def _move_chunks(cache, chunks, src, dst):
    if cache.shape[2] == chunks and cache.shape[3] % 9 == 0:  # fp4 records [pages, heads, chunks, 9 d]
        cache[dst // chunks, :, dst % chunks] = cache[src // chunks, :, src % chunks]
    else:  # rows [pages, tokens, heads, d]
        rows = cache.flatten(0, 1).unflatten(0, (-1, 16))
        rows[dst] = rows[src]


def _plain_fork(s):
    bs, (b, width), pages = s["case"]["bs"], s["table"].shape, s["free"].numel()
    lens, shares, n_free, table, free = s["lens"].long(), s["shares"].long(), s["num_free"].long(), s["table"].long(), s["free"]
    lp = torch.arange(width, device=_DEV)[None]
    if s["case"]["finished"]:
        done = s["finished"] != 0
        drop = torch.bincount(table[done[:, None] & (lp < -(-lens // bs)[:, None])], minlength=pages)
        shares = shares - drop
        back = torch.nonzero((drop > 0) & (shares < 0))[:, 0]
        shares = shares.clamp(min=0)
        free[torch.arange(len(back), device=_DEV) + n_free] = back.int()
        n_free = n_free + len(back)
        lens = torch.where(done, 0, lens)
    child = s["parent"] >= 0
    a = s["parent"].long().clamp(min=0)
    full, rem = torch.where(child, lens[a] // bs, 0), torch.where(child, lens[a] % bs, 0)
    want = (rem > 0).long()
    upto = want.cumsum(0)
    served = child & ((want == 0) | (upto <= n_free))
    new = free.long()[(n_free - upto).clamp(0, pages - 1)]
    shared = served[:, None] & (lp < full[:, None])
    parts = served & (want > 0)
    shares = shares + torch.bincount(table[a][shared], minlength=pages)
    table = torch.where(shared, table[a], table)
    table = torch.where(parts[:, None] & (lp == full[:, None]), new[:, None], table)
    s["src"].copy_(torch.where(parts, table[a].gather(1, full[:, None])[:, 0], -1))
    s["dst"].copy_(torch.where(parts, new, -1))
    s["tokens"].copy_(torch.where(parts, rem, 0))
    s["table"].copy_(table)
    s["lens_out"].copy_(torch.where(served, lens[a], lens))
    s["shares_out"].copy_(shares)
    s["num_out"].copy_(n_free - torch.where(parts, upto, 0).amax())
    _plain_copy(s, s["tokens"])
    return _fork_outputs(s)


def _plain_compact(s):
    bs, pages, most = s["case"]["bs"], s["free"].numel(), s["case"]["moves"]
    number = torch.arange(pages, device=_DEV)
    listed_free = s["free"].long()[number < s["num_free"]]
    live = torch.ones(pages, dtype=torch.bool, device=_DEV)
    live[listed_free] = False
    used, holes = torch.nonzero(live)[:, 0], torch.nonzero(~live)[:, 0]
    n = len(used)
    src = used[used >= n].flip(0)[:most]
    dst = holes[:len(src)]
    page_map = number.clone()
    page_map[src] = dst
    for_good = live.clone()
    for_good[src], for_good[dst] = False, True
    left = torch.nonzero(~for_good)[:, 0].flip(0)
    s["free_out"].fill_(-1)[:len(left)] = left.int()
    s["num_out"].fill_(len(left))
    shares = s["shares"].clone()
    shares[dst], shares[src] = s["shares"][src], 0
    s["shares_out"].copy_(shares)
    s["page_map"].copy_(page_map)
    s["src"].fill_(-1)[:len(src)] = src.int()
    s["dst"].fill_(-1)[:len(src)] = dst.int()
    s["extent"].copy_(torch.where(for_good, number + 1, 0).amax())
    lp = torch.arange(s["table"].shape[1], device=_DEV)[None]
    in_use = lp < -(-s["lens"] // bs)[:, None]
    s["table"].copy_(torch.where(in_use, page_map[s["table"].long().clamp(min=0)], s["table"]))
    _plain_copy(s, None)
    return _compact_outputs(s)


def _plain_dense(s, cache, which):
    """The cached rows of every sequence, fp32 [b, hkv, tokens, d], without the head scales."""
    table = s["table"].clamp(min=0).long()
    if s["case"]["cache"] != "fp4":
        rows = cache if s["case"]["cache"] == "bf16" else cache.view(torch.float8_e4m3fn).float()
        return rows[table].flatten(1, 2).transpose(1, 2).float()
    off = s["off"][which]
    rec = cache[table].transpose(1, 2).flatten(2, 3)                                # [b, hkv, chunks, 9 d]
    codes = rec[..., off[0].flatten()].unflatten(-1, (16, -1)).flatten(2, 3)
    scales = rec[..., off[1].flatten()].unflatten(-1, (16, -1)).flatten(2, 3)
    e = torch.tensor(_E2M1, device=_DEV)
    e = torch.cat([e, -e])
    byte = torch.arange(256, device=_DEV)
    pair = torch.stack([e[byte % 16], e[byte // 16]], -1)
    x = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    x *= scales.view(torch.float8_e4m3fn).float()[..., None]
    return x.flatten(-2)


def _plain_shared(s):
    case = s["case"]
    b, hq, hkv, d = case["b"], case["hq"], case["hkv"], case["d"]
    one = torch.ones(hkv, device=_DEV)
    ks, vs = (one, one) if case["cache"] == "bf16" else (s["k_scale"], s["v_scale"])
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    x = torch.matmul(q, _plain_dense(s, s["k_cache"], 0).transpose(2, 3))
    x *= (s["scale"] * ks)[:, None, None]
    hidden = (torch.arange(x.shape[-1], device=_DEV) >= s["lens"][:, None])[:, None, None]
    x.masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == -math.inf, 0.0, top)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    v = _plain_dense(s, s["v_cache"], 1)
    v.masked_fill_(hidden.transpose(2, 3), 0.0)
    o = torch.matmul(x, v) * vs[:, None, None]
    s["out"].copy_(torch.where(total > 0, o / total, 0.0).reshape(b, hq, d))
    return dict(out=s["out"])


# -- what a pass cannot do without ---------------------------------------------------------------

_BYTES = {"bf16": 2.0, "e4m3": 1.0, "fp4": 9 / 16}


def work(case):
    if case["op"] == "rope":
        q, k = case["n"] * case["hq"] * case["d"], case["n"] * case["hkv"] * case["d"]
        moved = 4 * q + 4 * k if case["back"] else 4 * q + 4 * k + 2 * _BYTES[case["cache"]] * k
        return {"bytes": moved + 12 * case["n"], "flops": 3 * case["n"] * (case["hq"] + case["hkv"]) * case["r"]}
    row = case["hkv"] * case["d"] * _BYTES[case["cache"]]
    if case["op"] == "fork":
        kids, bs = case["parents"] * case["kids"], case["bs"]
        copied = kids * min(bs, case["len_hi"]) / 2 * row * 2 * case["layers"]
        entries = (kids + case["finished"]) * (case["len_hi"] / 2 / bs + 1)
        return {"bytes": 2 * copied + 8 * entries + 32 * case["b"], "flops": entries}
    if case["op"] == "compact":
        used = case["b"] * max(1, min(case["len_hi"], case["pages"] // (2 * case["b"]) * case["bs"])) / 2 / case["bs"]
        moved = min(case["moves"], used / 2)
        return {"bytes": 4 * moved * case["bs"] * row + 24 * case["pages"] + 8 * used, "flops": 4 * case["pages"]}
    starts = _group_starts(case)
    prefix, suffix = (case["p_lo"] + case["p_hi"]) / 2 // case["bs"] * case["bs"], (1 + case["s_hi"]) / 2
    groups = sum(1 for a, e in zip(starts, starts[1:]) if e > a)
    rows = case["b"] * case["hq"] * case["d"]
    return {"bytes": 2 * row * (groups * prefix + case["b"] * suffix) + rows * (4 if case["out"] == "bf16" else 6),
            "flops": 4 * rows * (prefix + suffix)}


# -- the operators by definition, in 64 bits -----------------------------------------------------

def _exact_turns(case):
    """Radians per position of each pair, by the published definitions, pair by pair."""
    r, f, n, kind = case["r"], case["factor"], case["orig"], case["scaling"]
    base = 10000.0 if case["pmax"] <= 32768 else 1000000.0
    got = []
    for j in range(r // 2):
        if kind == "ntk" and r > 2:
            w = 1.0 / math.exp(2 * j / r * (math.log(base) + r / (r - 2) * math.log(f)))
        else:
            w = 1.0 / math.exp(2 * j / r * math.log(base))
        if kind == "linear":
            w = w / f
        elif kind == "yarn":
            # pairs that turn more than 32 times over the original length stay, those under one turn are stretched
            edge = [r / 2 * (math.log(n) - math.log(2 * math.pi * t)) / math.log(base) for t in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(r - 1, math.ceil(edge[1]))
            share = min(1.0, max(0.0, (j - lo) / (hi - lo if hi > lo else 0.001)))
            w = (1 - share) * w + share * w / f
        elif kind == "bands":
            wave = 2 * math.pi / w
            if wave > n / 1.0:
                w = w / f
            elif wave >= n / 4.0:
                keep = (n / wave - 1.0) / 3.0
                w = (1 - keep) * w / f + keep * w
        got.append(w)
    return got, (1 + math.log(f) / 10 if kind == "yarn" else 1.0)


def _exact_rotate(x, pos, turns, m, case):
    out = x.double().clone()
    r = case["r"]
    for j, w in enumerate(turns):
        t = pos.double()[:, None] * (-w if case["back"] else w)
        i0, i1 = (2 * j, 2 * j + 1) if case["inter"] else (j, j + r // 2)
        z = torch.complex(x[..., i0].double(), x[..., i1].double()) * torch.polar(torch.full_like(t, m), t)
        out[..., i0], out[..., i1] = z.real, z.imag
    return out


def _exact_e4m3(code):
    """e4m3 bytes -> float64, by the definition of the format."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def _exact_fp4(rec, which, d):
    """Records [n, 9 d] -> rows [16 n, d] in float64, without the head scale."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=_DEV)
    lut = torch.cat([lut, -lut])
    rows = torch.empty((rec.shape[0], 16, d), dtype=torch.float64, device=_DEV)
    for t in range(16):
        codes, scales = [], []
        for m in range(d // 2):
            blk, w = divmod(m, 8)
            if which == 0:
                codes.append((blk // 8 * 2 + t // 8) * 512 + (t % 8) * 64 + w // 2 * 16 + blk % 8 * 2 + w % 2)
            else:
                codes.append((t // 8 * 2 + t % 2) * 2 * d + (w * 4 + t % 8 // 2) * (d // 16) + blk)
        for blk in range(d // 16):
            scales.append(8 * d + (t * (d // 16) + blk if which == 0 else
                                   blk // 4 * 64 + t % 8 // 2 * 16 + blk % 4 * 4 + t // 8 * 2 + t % 2))
        byte, sc = rec[:, codes].long(), _exact_e4m3(rec[:, scales]).repeat_interleave(16, 1)
        rows[:, t, 0::2], rows[:, t, 1::2] = lut[byte & 15], lut[byte >> 4]
        rows[:, t] *= sc
    return rows.flatten(0, 1)


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        turns, m = _exact_turns(case)
        q, k = _exact_rotate(s["q"], s["pos"], turns, m, case), _exact_rotate(s["k"], s["pos"], turns, m, case)
        if case["back"]:
            return {"q": q, "k": k}
        caches = [torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=_DEV) for _ in range(2)]
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        page, at = s["slots"][keep] // case["bs"], s["slots"][keep] % case["bs"]
        caches[0][page, at], caches[1][page, at] = k[keep], s["v"][keep].double()
        return {"q": q, "k": caches[0], "v": caches[1]}
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    grp = hq // hkv
    out = torch.zeros((case["b"], hq, d), dtype=torch.float64, device=_DEV)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // bs)].long()
        for h in range(hkv):
            kv = []
            for which, (cache, g) in enumerate(((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))):
                if case["cache"] == "fp4":
                    rows = _exact_fp4(cache[ids, h].flatten(0, 1), which, d) * g[h].double()
                elif case["cache"] == "e4m3":
                    rows = _exact_e4m3(cache[ids, :, h].flatten(0, 1)) * g[h].double()
                else:
                    rows = cache[ids, :, h].flatten(0, 1).double()
                kv.append(rows[:n])
            q = s["q"][b, h * grp:(h + 1) * grp].double()
            out[b, h * grp:(h + 1) * grp] = torch.softmax(q @ kv[0].T * s["scale"], -1) @ kv[1]
    return {"out": out}
