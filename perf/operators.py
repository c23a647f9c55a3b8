"""The operators of a 4-bit KV cache, and the block tables and slot maps that
every call of this library takes, as cases that can be run and timed.

Each case runs one pass through one operator, in one of two forms:

* the plain form (``own`` false): elementary torch operations in 32 bits,
  rounded once at the end;
* the library's own calls (``own`` true), as a serving loop makes them.

The fp4 cache holds, per (token, KV head), e2m1 codes with one e4m3 scale for
every 16 dims and one binary32 scale per KV head.  Sixteen tokens of a KV head
form one record of 9 * head_dim bytes; `_offsets` says where in a record each
byte stands.  A cache tensor is uint8 [pages, kv_heads, block_size / 16,
9 * head_dim].
"""
import math

import torch

own = False

_DEV = "cuda"
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# -- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # one new token of one request enters the cache: the smallest write, all launch latency
        dict(name="write_token", op="write", tokens=1, hkv=4, d=256, bs=784, out="bf16"),
        # the prompt chunks of a batch, 8-head dense model, 16-token pages, some padding rows: bandwidth
        dict(name="write_prompt", op="write", tokens=16411, hkv=8, d=128, bs=16, out="bf16"),
        # the decode step of a short chat: the new token is written and read in one call
        dict(name="step_512", op="attn", b=1, lo=512, hi=512, hq=24, hkv=4, d=256, bs=16, ql=1, out="f32",
             window=0, append=True),
        # one long conversation of the hybrid model, the context split over the whole GPU
        dict(name="decode_32k", op="attn", b=1, lo=32768, hi=32768, hq=24, hkv=4, d=256, bs=784, ql=1, out="f32",
             window=0, append=False),
        # a full serving batch of ragged lengths: the largest decode, cache bandwidth
        dict(name="decode_batch", op="attn", b=32, lo=1024, hi=32768, hq=24, hkv=4, d=256, bs=784, ql=1, out="bf16",
             window=0, append=False),
        # the dense model on small pages with a sliding window, odd lengths, one idle slot of length 0
        dict(name="decode_dense_window", op="attn", b=7, lo=0, hi=9001, hq=32, hkv=8, d=128, bs=16, ql=1, out="f32",
             window=4095, append=False),
        # speculative verify of 16 drafted rows for each of 8 requests
        dict(name="verify_draft", op="attn", b=8, lo=8208, hi=8208, hq=24, hkv=4, d=256, bs=832, ql=16, out="f32",
             window=0, append=False),
        # verify of 5 rows in the wide-group model (12 heads per KV head), ragged contexts
        dict(name="verify_wide", op="attn", b=32, lo=700, hi=2048, hq=48, hkv=4, d=256, bs=784, ql=5, out="bf16",
             window=0, append=False),
        # one chunk of a long prompt: 2048 new rows over 14336 cached tokens, tensor-core work
        dict(name="prefill_chunk", op="attn", b=1, lo=16384, hi=16384, hq=24, hkv=4, d=256, bs=832, ql=2048,
             out="bf16", window=0, append=False),
        # the table update of one decode step: every request grows by one token
        dict(name="tables_step", op="tables", b=32, bs=784, pages=42, prompt=1, short=0.0, churn=False),
        # a wave of prompts on 16-token pages: about a million slots, a pool that runs short near the end
        dict(name="tables_prompts", op="tables", b=509, bs=16, pages=512, prompt=4099, short=0.02, churn=False),
        # a scheduler step that frees finished requests and admits others in their place
        dict(name="tables_churn", op="tables", b=256, bs=16, pages=600, prompt=1500, short=0.0, churn=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "verify", "verify", "tables"])
    hq, hkv, d = rng.choice([(24, 4, 256), (48, 4, 256), (32, 8, 128), (6, 1, 256), (8, 8, 128), (20, 4, 256),
                             (32, 2, 128), (10, 2, 256)])
    bs = rng.choice([16, 48, 64, 784, 832])
    out = rng.choice(["f32", "bf16"])
    if op == "write":
        return dict(op="write", tokens=_log_int(rng, 1, 16000), hkv=hkv, d=d, bs=bs, out=out)
    if op == "tables":
        b = _log_int(rng, 1, 1000)
        return dict(op="tables", b=b, bs=bs, pages=_log_int(rng, 4, 512), prompt=_log_int(rng, 1, 4000),
                    short=rng.choice([0.0, 0.0, 0.1]), churn=rng.random() < 0.4)
    window = _log_int(rng, 1, 8000) if rng.random() < 0.25 else 0
    hi = _log_int(rng, 20, 32768)
    if op == "decode":
        b = min(_log_int(rng, 1, 64), max(1, 500_000 * 4 * 256 // (hi * hkv * d)))
        return dict(op="attn", b=b, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, hq=hq, hkv=hkv, d=d, bs=bs, ql=1,
                    out=out, window=window, append=rng.random() < 0.4)
    ql = min(_log_int(rng, 2, 700), hi)
    b = min(_log_int(rng, 1, 32), max(1, 500_000 * 4 * 256 // (hi * hkv * d)), max(1, 400_000_000 // (ql * hq * hi)))
    return dict(op="attn", b=b, lo=max(ql, rng.choice([ql, hi // 2, hi])), hi=hi, hq=hq, hkv=hkv, d=d, bs=bs,
                ql=max(2, ql), out=out, window=window, append=False)


# -- the cache format in plain torch -------------------------------------------------------------

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


def _quantise(x, g):
    """Rows [..., hkv, d] (bf16) and head scales [hkv] -> code bytes [..., d / 2]
    and scale bytes [..., d / 16]."""
    x = x.float().unflatten(-1, (-1, 16))
    g = g[:, None]
    nan = x.isnan().any(-1)
    a = x.abs().amax(-1)
    s8 = (a / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    v = x * (1.0 / (s * g))[..., None]
    w = v.abs()
    code = ((w > 0.25).byte() + (w >= 0.75).byte() + (w > 1.25).byte() + (w >= 1.75).byte() + (w > 2.5).byte()
            + (w >= 3.5).byte() + (w > 5.0).byte()) | (torch.signbit(v).byte() << 3)
    dead = (nan | (s == 0))[..., None]
    code = torch.where(dead, torch.zeros_like(code), code).flatten(-2)
    s8 = torch.where(nan, torch.full_like(s8.view(torch.uint8), 0x7F), s8.view(torch.uint8))
    return code[..., ::2] | (code[..., 1::2] << 4), s8


def _values(code_bytes, scale_bytes):
    """Code bytes [..., d / 2] and scale bytes [..., d / 16] -> code * scale, fp32 [..., d]."""
    e = torch.tensor(_E2M1, device=_DEV)
    e = torch.cat([e, -e])
    byte = torch.arange(256, device=_DEV)
    pair = torch.stack([e[byte % 16], e[byte // 16]], -1)
    x = pair[code_bytes.int()].flatten(-2).unflatten(-1, (-1, 16))
    x *= scale_bytes.view(torch.float8_e4m3fn).float()[..., None]
    return x.flatten(-2)


def _records(codes, scales, off, d):
    """Codes and scales of whole chunks [n, 16, hkv, ...] -> records [n, hkv, 9 d]."""
    n, _, hkv, _ = codes.shape
    rec = torch.empty((n, hkv, 9 * d), dtype=torch.uint8, device=_DEV)
    rec[..., off[0].flatten()] = codes.transpose(1, 2).flatten(2)
    rec[..., off[1].flatten()] = scales.transpose(1, 2).flatten(2)
    return rec


def _row_index(slots, bs, hkv, d, off):
    """Flat byte positions in a cache of the code and scale bytes of the rows at `slots`: [n, hkv, ...]."""
    page, pos = slots // bs, slots % bs
    head = torch.arange(hkv, device=_DEV)
    rec = ((page[:, None] * hkv + head) * (bs // 16) + (pos // 16)[:, None]) * (9 * d)
    return [rec[..., None] + o[pos % 16][:, None, :] for o in off]


# -- inputs --------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed)


def _rows(gen, shape):
    """bf16 K or V rows: normal, with every 32nd channel eight times as large, as K caches have them."""
    x = torch.randn(shape, generator=gen, device=_DEV)
    x[..., 7::32] *= 8.0
    return x.to(torch.bfloat16)


def _head_scales(hkv):
    h = torch.arange(hkv, device=_DEV, dtype=torch.float32)
    return (1 + h / 4) / 96, (1 + h / 8) / 80


def _cache(gen, pages, bs, hkv, d, g, off):
    chunks, step = pages * bs // 16, max(1, (1 << 26) // (16 * hkv * d))
    rec = torch.empty((chunks, hkv, 9 * d), dtype=torch.uint8, device=_DEV)
    for c in range(0, chunks, step):
        n = min(step, chunks - c)
        rec[c:c + n] = _records(*_quantise(_rows(gen, (n, 16, hkv, d)), g), off, d)
    return rec.unflatten(0, (pages, bs // 16)).transpose(1, 2).contiguous()


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device=_DEV)


def prepare(case, seed):
    return {"write": _prepare_write, "attn": _prepare_attn, "tables": _prepare_tables}[case["op"]](case, seed)


def _prepare_write(case, seed):
    gen, n, hkv, d, bs = _gen(seed), case["tokens"], case["hkv"], case["d"], case["bs"]
    pages = -(-n * 5 // (4 * bs)) + 2
    # whole pages in random order, filled front to back, as prompts fill them
    slots = (torch.randperm(pages, generator=gen, device=_DEV)[:, None] * bs
             + torch.arange(bs, device=_DEV)).flatten()[3:n + 3].contiguous()
    if n > 64:
        slots[_ints(gen, 0, n - 1, 5)] = -1  # padding rows
    ks, vs = _head_scales(hkv)
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    shape = (pages, hkv, bs // 16, 9 * d)
    return dict(case=case, k_new=_rows(gen, (n, hkv, d)), v_new=_rows(gen, (n, hkv, d)), slots=slots, k_scale=ks,
                v_scale=vs, k_cache=torch.zeros(shape, dtype=torch.uint8, device=_DEV),
                v_cache=torch.zeros(shape, dtype=torch.uint8, device=_DEV),
                k_out=torch.empty((n, hkv, d), dtype=dtype, device=_DEV),
                v_out=torch.empty((n, hkv, d), dtype=dtype, device=_DEV), off=_offsets(d))


def _prepare_attn(case, seed):
    gen, b, hkv, d, bs = _gen(seed), case["b"], case["hkv"], case["d"], case["bs"]
    lens = _ints(gen, case["lo"], case["hi"], b)
    lens[0] = case["hi"]
    if b > 1:
        lens[1] = case["lo"]
    width = -(-case["hi"] // bs)
    used = -(-lens // bs)
    pages = max(1, -(-int(used.sum()) * 11 // 10))
    order = torch.randperm(pages, generator=gen, device=_DEV)
    lp = torch.arange(width, device=_DEV)[None]
    first = (used.cumsum(0) - used)[:, None]
    table = torch.where(lp < used[:, None], order[(first + lp).clamp(max=pages - 1)], -1).int()
    ks, vs = _head_scales(hkv)
    off = _offsets(d)
    rows = b * case["ql"]
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    state = dict(case=case, q=torch.randn((rows, case["hq"], d), generator=gen, device=_DEV).to(torch.bfloat16),
                 k_cache=_cache(gen, pages, bs, hkv, d, ks, off[0]), v_cache=_cache(gen, pages, bs, hkv, d, vs, off[1]),
                 k_scale=ks, v_scale=vs, table=table, lens=lens.int(), scale=1.0 / math.sqrt(d), off=off,
                 out=torch.empty((rows, case["hq"], d), dtype=dtype, device=_DEV),
                 workspace=torch.empty(64 << 20, dtype=torch.uint8, device=_DEV))
    if case["append"]:
        last = (lens - 1).clamp(min=0)
        page = table.long().gather(1, (last // bs)[:, None])[:, 0]
        state |= dict(k_new=_rows(gen, (b, hkv, d)), v_new=_rows(gen, (b, hkv, d)),
                      slots=torch.where(lens > 0, page * bs + last % bs, -1),
                      k_out=torch.empty((b, hkv, d), dtype=torch.bfloat16, device=_DEV),
                      v_out=torch.empty((b, hkv, d), dtype=torch.bfloat16, device=_DEV))
    if own:
        import paged_attention_decode_split_gb300 as pa
        state["desc"] = pa.make_desc(
            num_seqs=b, q_len=case["ql"], num_q_heads=case["hq"], num_kv_heads=hkv, head_dim=d, block_size=bs,
            max_pages_per_seq=width, max_seq_len=case["hi"], num_pages=pages, scale=state["scale"],
            out_dtype=pa.PA_OUT_BF16 if case["out"] == "bf16" else pa.PA_OUT_F32, window=case["window"])
    return state


def _prepare_tables(case, seed):
    gen, b, bs, width = _gen(seed), case["b"], case["bs"], case["pages"]
    room, order = width * bs, torch.randperm(b, generator=gen, device=_DEV)
    # prompt lengths spread evenly over 1 .. prompt, in random order
    new = 1 + order * (min(case["prompt"], room) - 1) // max(1, b - 1)
    finished = torch.zeros(b, dtype=torch.int32, device=_DEV)
    if case["churn"]:  # of four requests one is finished, one admitted, two go on by a token
        new = torch.where(order % 4 == 0, 0, torch.where(order % 4 == 1, new, 1))
        finished = (order % 4 == 0).int()
    context = (torch.rand(b, generator=gen, device=_DEV) * (room - new + 1)).long()
    if case["churn"]:
        context = torch.where(order % 4 == 1, 0, context)
    held, need = -(-context // bs), -(-(context + new) // bs) - -(-context // bs)
    total_held, total_need = int(held.sum()), int(need.sum())
    pages = b * width + 16
    spare = max(1, int(total_need * (1 - case["short"]))) + (0 if case["short"] else 9)
    pool = torch.randperm(pages, generator=gen, device=_DEV).int()
    lp = torch.arange(width, device=_DEV)[None]
    first = (held.cumsum(0) - held)[:, None]
    table = torch.where(lp < held[:, None], pool[(first + lp).clamp(max=pages - 1)], -1).int()
    free = torch.full((pages,), -1, dtype=torch.int32, device=_DEV)
    free[:spare] = pool[total_held:total_held + spare]
    n = int(new.sum())
    n += n // 64 + 3  # the batch is padded
    i32 = dict(dtype=torch.int32, device=_DEV)
    return dict(case=case, context=context.int(), new=new.int(), finished=finished, table=table, free=free, tokens=n,
                num_free=torch.tensor([spare], **i32), lens_mid=torch.empty(b, **i32), free_mid=torch.empty(1, **i32),
                lens=torch.empty(b, **i32), free_out=torch.empty(1, **i32),
                slots=torch.empty(n, dtype=torch.int64, device=_DEV))


# -- one pass ------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"write": _own_write, "attn": _own_attn, "tables": _own_tables}[op](state)
    return {"write": _plain_write, "attn": _plain_attn, "tables": _plain_tables}[op](state)


def _own_write(s):
    import paged_attention_decode_split_gb300 as pa
    pa.reshape_and_cache_fp4(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["slots"], s["k_scale"], s["v_scale"])
    pa.gather_cache_fp4(s["k_cache"], s["v_cache"], s["slots"], s["k_scale"], s["v_scale"], s["k_out"], s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def _own_attn(s):
    import paged_attention_decode_split_gb300 as pa
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if s["case"]["append"]:
        pa.paged_attention_decode_append_fp4(s["q"], s["k_new"], s["v_new"], *cache, s["table"], s["lens"], s["desc"],
                                             s["out"], s["workspace"])
        pa.gather_cache_fp4(s["k_cache"], s["v_cache"], s["slots"], s["k_scale"], s["v_scale"], s["k_out"], s["v_out"])
        return dict(out=s["out"], k=s["k_out"], v=s["v_out"])
    call = pa.paged_attention_decode_fp4 if s["case"]["ql"] == 1 else pa.paged_attention_verify_fp4
    call(s["q"], *cache, s["table"], s["lens"], s["desc"], s["out"], s["workspace"])
    return dict(out=s["out"])


def _own_tables(s):
    import paged_attention_decode_split_gb300 as pa
    bs, lens, free = s["case"]["bs"], s["context"], s["num_free"]
    if s["case"]["churn"]:
        pa.release_block_tables(lens, s["finished"], s["table"], s["free"], free, bs, s["lens_mid"], s["free_mid"])
        lens, free = s["lens_mid"], s["free_mid"]
    pa.extend_block_tables(lens, s["new"], s["table"], s["free"], free, bs, s["lens"], s["slots"], s["free_out"])
    return dict(table=s["table"], lens=s["lens"], slots=s["slots"], num_free=s["free_out"], free=s["free"])


def _plain_store(s):
    """Quantises the new rows into their slots and reads them back."""
    bs, (n, hkv, d) = s["case"]["bs"], s["k_new"].shape
    back = []
    live = s["slots"] >= 0
    for x, cache, g, off in ((s["k_new"], s["k_cache"], s["k_scale"], s["off"][0]),
                             (s["v_new"], s["v_cache"], s["v_scale"], s["off"][1])):
        codes, scales = _quantise(x, g)
        at_codes, at_scales = _row_index(s["slots"].clamp(min=0), bs, hkv, d, off)
        flat = cache.view(-1)
        flat[at_codes[live]] = codes[live]
        flat[at_scales[live]] = scales[live]
        rows = _values(flat[at_codes], flat[at_scales]) * g[:, None]
        back.append(torch.where(live[:, None, None], rows, 0.0).to(s["k_out"].dtype))
    return back


def _plain_write(s):
    k, v = _plain_store(s)
    return dict(k=k, v=v)


def _plain_dense(cache, table, off, hkv, d):
    """The cached rows of every sequence, fp32 [b, hkv, tokens, d], without the head scales."""
    rec = cache[table.clamp(min=0).long()]                                  # [b, pages, hkv, chunks, 9 d]
    rec = rec.transpose(1, 2).flatten(2, 3)                                 # [b, hkv, chunks, 9 d]
    codes = rec[..., off[0].flatten()].unflatten(-1, (16, -1)).flatten(2, 3)
    scales = rec[..., off[1].flatten()].unflatten(-1, (16, -1)).flatten(2, 3)
    return _values(codes, scales)


def _plain_attn(s):
    case = s["case"]
    ql, hq, hkv, d = case["ql"], case["hq"], case["hkv"], case["d"]
    new = _plain_store(s) if case["append"] else None
    b, grp = case["b"], hq // hkv
    lens = s["lens"].long()
    q = s["q"].float().view(b, ql, hkv, grp, d).transpose(1, 2).flatten(2, 3)  # [b, hkv, ql * grp, d]
    k = _plain_dense(s["k_cache"], s["table"], s["off"][0], hkv, d)
    x = torch.matmul(q, k.transpose(2, 3))
    del k
    x *= (s["scale"] * s["k_scale"])[:, None, None]
    key = torch.arange(x.shape[-1], device=_DEV)
    pos = (lens[:, None] - ql + torch.arange(ql, device=_DEV)).repeat_interleave(grp, 1)[:, None, :, None]
    hidden = key > pos
    if case["window"]:
        hidden |= key <= pos - case["window"]
    x.masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == -math.inf, 0.0, top)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    v = _plain_dense(s["v_cache"], s["table"], s["off"][1], hkv, d)
    v.masked_fill_((key >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x, v) * s["v_scale"][:, None, None]
    o = torch.where(total > 0, o / total, 0.0)
    out = o.view(b, hkv, ql, grp, d).transpose(1, 2).reshape(b * ql, hq, d).to(s["out"].dtype)
    return dict(out=out, k=new[0], v=new[1]) if new else dict(out=out)


def _plain_tables(s):
    bs, (b, width), pages = s["case"]["bs"], s["table"].shape, s["free"].numel()
    table, free, n_free = s["table"].long(), s["free"].long(), s["num_free"].long()
    lens = s["context"].long()
    lp = torch.arange(width, device=_DEV)[None]
    if s["case"]["churn"]:
        held = torch.where(s["finished"] != 0, -(-lens // bs), 0)
        at = (n_free + held.cumsum(0) - held)[:, None] + lp
        mine = lp < held[:, None]
        free = free.scatter(0, torch.where(mine, at, pages).flatten()[mine.flatten()], table[mine])
        n_free = n_free + held.sum()
        lens = torch.where(s["finished"] != 0, 0, lens)
    new = s["new"].long()
    end = new.cumsum(0)
    have, want = -(-lens // bs), -(-(lens + new) // bs)
    fits = lens + new <= width * bs
    need = torch.where(fits, want - have, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= n_free))
    last = (n_free - 1 - (upto - need))[:, None] - (lp - have[:, None])  # stack entry of page lp of a request
    grown = served[:, None] & (lp >= have[:, None]) & (lp < want[:, None])
    table = torch.where(grown, free[last.clamp(0, pages - 1)], table)
    i = torch.arange(s["tokens"], device=_DEV)
    r = torch.searchsorted(end, i, right=True).clamp(max=b - 1)
    p = lens[r] + i - (end - new)[r]
    slot = table[r, (p // bs).clamp(max=width - 1)] * bs + p % bs
    slots = torch.where((i < end[-1]) & served[r], slot, -1)
    left = n_free - torch.where(served & (need > 0), upto, 0).amax()  # (upto counts refused requests' pages too)
    return dict(table=table.int(), lens=torch.where(served, lens + new, lens).int(), slots=slots, num_free=left.int(),
                free=free.int())


# -- what a pass cannot do without ---------------------------------------------------------------

def _mean_keys(case):
    return (case["lo"] + case["hi"]) / 2 if case["b"] > 2 else (case["hi"] + (case["lo"] if case["b"] > 1 else 0)) / case["b"]


def work(case):
    if case["op"] == "write":
        elems = 2 * case["tokens"] * case["hkv"] * case["d"]
        return {"bytes": elems * (2 + 9 / 16 + (2 if case["out"] == "bf16" else 4)) + 8 * case["tokens"], "flops": 4 * elems}
    if case["op"] == "tables":
        mean = case["prompt"] / 2 + 0.5
        tokens = case["b"] * (mean / 4 + 0.5 if case["churn"] else mean)
        return {"bytes": 16 * case["b"] + 8 * tokens + 8 * tokens / case["bs"], "flops": 2 * tokens}
    keys, rows = _mean_keys(case), case["b"] * case["ql"]
    seen = keys - (case["ql"] - 1) / 2
    if case["window"]:
        seen, keys = min(seen, case["window"]), min(keys, case["window"] + case["ql"] - 1)
    o = 2 if case["out"] == "bf16" else 4
    return {"bytes": case["b"] * keys * case["hkv"] * case["d"] * 9 / 8 + rows * case["hq"] * case["d"] * (2 + o),
            "flops": 4 * rows * case["hq"] * case["d"] * seen}


# -- the operators by definition, in 64 bits -----------------------------------------------------

_CODE64 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _exact_e4m3(code):
    """e4m3 bytes -> float64, by the definition of the format."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def _exact_row_bytes(kind, t, d):
    """Where code byte of dims (2m, 2m + 1) and scale byte of block blk stand for the t-th token of a record."""
    codes, scales = [], []
    for m in range(d // 2):
        blk, w = divmod(m, 8)
        if kind == "k":
            codes.append((blk // 8 * 2 + t // 8) * 512 + (t % 8) * 64 + w // 2 * 16 + blk % 8 * 2 + w % 2)
        else:
            codes.append((t // 8 * 2 + t % 2) * 2 * d + (w * 4 + t % 8 // 2) * (d // 16) + blk)
    for blk in range(d // 16):
        if kind == "k":
            scales.append(8 * d + t * (d // 16) + blk)
        else:
            scales.append(8 * d + blk // 4 * 64 + t % 8 // 2 * 16 + blk % 4 * 4 + t // 8 * 2 + t % 2)
    return codes, scales


def _exact_chunks(rec, kind, d):
    """Records [n, 9 d] -> rows [16 n, d] in float64, without the head scale."""
    lut = torch.tensor(_CODE64, dtype=torch.float64, device=_DEV)
    rows = torch.empty((rec.shape[0], 16, d), dtype=torch.float64, device=_DEV)
    for t in range(16):
        codes, scales = _exact_row_bytes(kind, t, d)
        byte, s = rec[:, codes].long(), _exact_e4m3(rec[:, scales]).repeat_interleave(16, 1)
        rows[:, t, 0::2], rows[:, t, 1::2] = lut[byte & 15], lut[byte >> 4]
        rows[:, t] *= s
    return rows.flatten(0, 1)


def _exact_stored(x, g):
    """The values that rows [n, hkv, d] stand for once stored: nearest points by
    distance, ties to the even code; single steps rounded to binary32 as defined."""
    to32 = lambda v: v.float().double()  # noqa: E731
    x = x.double().unflatten(-1, (-1, 16))
    g = g.double()[:, None]
    want = to32(x.abs().amax(-1) / to32(6 * g)).clamp(max=448)
    points = _exact_e4m3(torch.arange(127, device=_DEV))
    hi = torch.searchsorted(points, want).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    near = torch.where(want - points[lo] == points[hi] - want, torch.where(lo % 2 == 0, lo, hi),
                       torch.where(want - points[lo] < points[hi] - want, lo, hi))
    s = points[near]
    v = to32(x * to32(1 / to32(s * g))[..., None])
    mags = torch.tensor(_CODE64[:8], dtype=torch.float64, device=_DEV)
    w = v.abs().clamp(max=6.0)
    hi = torch.searchsorted(mags, w).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    down, up = w - mags[lo], mags[hi] - w
    pick = torch.where(down == up, torch.where(lo % 2 == 0, lo, hi), torch.where(down < up, lo, hi))
    rows = torch.where(s[..., None] == 0, 0.0, torch.sign(v) * mags[pick]) * s[..., None] * g[..., None]
    return rows.flatten(-2)


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "write":
        pad = (s["slots"] < 0)[:, None, None]
        return {"k": _exact_stored(s["k_new"], s["k_scale"]).masked_fill(pad, 0.0),
                "v": _exact_stored(s["v_new"], s["v_scale"]).masked_fill(pad, 0.0)}
    ql, hq, hkv, d, bs = case["ql"], case["hq"], case["hkv"], case["d"], case["bs"]
    grp, window = hq // hkv, case["window"]
    if case["b"] * ql * hq * case["hi"] * d > 1.5e12:
        return None
    out = torch.zeros((case["b"] * ql, hq, d), dtype=torch.float64, device=_DEV)
    result = {"out": out}
    if case["append"]:
        result["k"] = _exact_stored(s["k_new"], s["k_scale"])
        result["v"] = _exact_stored(s["v_new"], s["v_scale"])
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            if case["append"]:
                result["k"][b], result["v"][b] = 0.0, 0.0
            continue
        ids = s["table"][b, :-(-n // bs)].long()
        for h in range(hkv):
            k = _exact_chunks(s["k_cache"][ids, h].flatten(0, 1), "k", d)[:n] * s["k_scale"][h].double()
            v = _exact_chunks(s["v_cache"][ids, h].flatten(0, 1), "v", d)[:n] * s["v_scale"][h].double()
            if case["append"]:
                k[n - 1], v[n - 1] = result["k"][b, h], result["v"][b, h]
            key = torch.arange(n, device=_DEV)
            for r0 in range(0, ql, 64):
                rows = torch.arange(r0, min(ql, r0 + 64), device=_DEV)
                q = s["q"][b * ql + rows, h * grp:(h + 1) * grp].double()
                x = torch.einsum("rgd,td->rgt", q, k) * s["scale"]
                pos = (n - ql + rows)[:, None, None]
                seen = key <= pos
                if window:
                    seen = seen & (key > pos - window)
                w = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
                out[b * ql + rows, h * grp:(h + 1) * grp] = torch.einsum("rgt,td->rgd", w, v)
    return result
