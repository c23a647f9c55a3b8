"""Decode over shared prefixes without a GPU: its plan, the calls that are refused
before a launch, and the reference that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests.shared_ref import KINDS, Batch

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def desc(**kw):
    base = dict(num_seqs=64, num_q_heads=24, num_kv_heads=4, head_dim=256, block_size=784, max_pages_per_seq=50,
                max_seq_len=34000, num_pages=200, scale=1 / 16, num_sms=152)
    return pa.make_desc(**(base | kw))


def prefix(**kw):
    return pa.make_prefix(**(dict(num_groups=1, max_group_seqs=64, max_prefix_len=32768, max_suffix_len=1500) | kw))


def records(d, x):
    """Split records per row that the workspace holds (exact: a record is head_dim floats and two)."""
    rows = d.num_seqs * d.num_q_heads
    n = pa.shared_workspace_bytes(d, x)
    for s in range(1, 2000):
        if (rows * s * d.head_dim * 4 + 255) // 256 * 256 + rows * s * 8 == n:
            return s


def test_plan(lib):
    # 64 sequences of 6 heads: 3 row blocks of 4 KV heads, 0.7 of the SMs; own parts of 1500 tokens in one split
    assert records(desc(), prefix()) == 9 + 1
    # prefixes next to which the own parts are short get nearly all, and no second wave
    assert records(desc(), prefix(max_suffix_len=64)) == 12 + 1
    # 16 groups of 4 KV heads, their prefixes taken for shorter than the longest on average
    assert records(desc(), prefix(num_groups=16, max_group_seqs=4)) == 3 + 1
    # 32: several waves, at most 4096 tokens for a CTA
    assert records(desc(), prefix(num_groups=32, max_group_seqs=2)) == 8 + 1
    # short prefixes are not cut below 128 tokens; own parts are cut while SMs are left
    assert records(desc(), prefix(max_prefix_len=512, max_suffix_len=4000)) == 4 + 1
    # sharing that saves little is left: 4 sequences of 552 tokens, 35 chunks, split as a decode of that length
    small = dict(max_group_seqs=4, max_prefix_len=512, max_suffix_len=40)
    assert records(desc(num_seqs=4), prefix(**small)) == 7
    assert records(desc(num_seqs=4), prefix(prefix_splits=3, **small)) == 3 + 1
    # so is a batch without groups; one split of it needs no records
    assert pa.shared_workspace_bytes(desc(num_splits=1), prefix(num_groups=64, max_group_seqs=1)) == 0
    # forced
    assert records(desc(num_splits=7), prefix(prefix_splits=5)) == 5 + 7
    # the hints bound nothing, and 0 stands for max_seq_len
    assert records(desc(), prefix(max_prefix_len=0)) == records(desc(), prefix(max_prefix_len=10 ** 9))
    assert pa.shared_workspace_bytes(desc(num_seqs=0), prefix(num_groups=0, max_group_seqs=0)) == 0


@pytest.mark.parametrize("kw,xw,code", [
    (dict(head_dim=64), {}, pa.PA_ERR_UNSUPPORTED), (dict(num_q_heads=40), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(q_len=2), {}, pa.PA_ERR_INVALID_ARG), (dict(window=100), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=20, max_pages_per_seq=2000), {}, pa.PA_ERR_UNSUPPORTED), (dict(flags=2), {}, pa.PA_ERR_INVALID_ARG),
    ({}, dict(num_groups=0), pa.PA_ERR_INVALID_ARG), ({}, dict(num_groups=-1), pa.PA_ERR_INVALID_ARG),
    ({}, dict(max_group_seqs=0), pa.PA_ERR_INVALID_ARG), ({}, dict(max_prefix_len=-1), pa.PA_ERR_INVALID_ARG),
    ({}, dict(max_suffix_len=-1), pa.PA_ERR_INVALID_ARG), ({}, dict(prefix_splits=-1), pa.PA_ERR_INVALID_ARG),
    ({}, dict(num_groups=65536), pa.PA_ERR_UNSUPPORTED)])
def test_calls_refuse_descriptions(lib, kw, xw, code):
    d, x = desc(**kw), prefix(**xw)
    args = (FAKE, FAKE, ctypes.byref(d), ctypes.byref(x), FAKE, FAKE, 1 << 40, None, None)
    assert lib.pa_paged_attention_decode_shared(FAKE, FAKE, FAKE, FAKE, FAKE, *args) == code
    for name in ("fp8", "fp4"):
        fn = getattr(lib, "pa_paged_attention_decode_shared_" + name)
        assert fn(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, *args) == code
    with pytest.raises(pa.PagedAttnError):
        pa.shared_workspace_bytes(d, x)


def test_calls_refuse_pointers_and_workspace(lib):
    d, x = desc(), prefix()
    need = pa.shared_workspace_bytes(d, x)

    def call(name="", ks=FAKE, ws=FAKE, size=need, d=d, x=x, **at):
        v = [at.get(k, FAKE) for k in ("q", "k", "v", "table", "lens", "starts", "prefix", "out")]
        scales = (ks, FAKE) if name else ()
        return getattr(lib, "pa_paged_attention_decode_shared" + name)(
            *v[:3], *scales, *v[3:7], ctypes.byref(d) if d else None, ctypes.byref(x) if x else None, v[7], ws, size, None, None)
    for k in ("q", "k", "v", "table", "lens", "starts", "prefix", "out"):
        assert call(**{k: None}) == pa.PA_ERR_INVALID_ARG, k
        assert call(**{k: FAKE + 2}) == pa.PA_ERR_INVALID_ARG, k
    assert call(d=None) == call(x=None) == pa.PA_ERR_INVALID_ARG
    assert call(size=need - 1) == call(ws=None) == call(ws=FAKE + 8) == pa.PA_ERR_WORKSPACE
    for name in ("_fp8", "_fp4"):
        assert call(name, ks=None) == call(name, ks=FAKE + 2) == pa.PA_ERR_INVALID_ARG
    empty = desc(num_seqs=0)
    assert lib.pa_paged_attention_decode_shared(*[None] * 7, ctypes.byref(empty), ctypes.byref(prefix(num_groups=0)), None, None, 0,
                                                None, None) == pa.PA_OK


def test_binding_refuses(lib):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    d = desc(num_seqs=2, block_size=16, max_pages_per_seq=4, max_seq_len=64, num_pages=8)
    x = prefix(num_groups=2, max_group_seqs=2)
    cache, codes, rec = z(8, 16, 4, 256), z(8, 16, 4, 256, t=torch.uint8), z(*pa.fp4_cache_shape(8, 16, 4, 256), t=torch.uint8)
    good = dict(q=z(2, 24, 256), k_cache=cache, v_cache=cache, block_table=i(2, 4), seq_lens=i(2), group_starts=i(3),
                prefix_lens=i(2), desc=d, prefix=x, out=z(2, 24, 256, t=torch.float32), workspace=z(64, t=torch.uint8))
    for kw, msg in ((dict(group_starts=i(2)), "group_starts: shape"), (dict(prefix_lens=i(3)), "prefix_lens: shape"),
                    (dict(group_starts=i(3).long()), "group_starts: dtype"), (dict(prefix_lens=z(2)), "prefix_lens: dtype"),
                    (dict(group_starts=None), "both are required"), (dict(k_cache=codes), "k_cache: dtype"),
                    (dict(q=z(3, 24, 256)), "q: shape"), (dict(), "q: a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            pa.paged_attention_decode_shared(**(good | kw))
    g = torch.ones(4)
    quant = good | dict(k_scale=g, v_scale=g)
    for fn, c, kw, msg in ((pa.paged_attention_decode_shared_fp8, cache, {}, "k_cache: dtype"),
                           (pa.paged_attention_decode_shared_fp8, codes, dict(k_scale=None), "an e4m3 cache needs both"),
                           (pa.paged_attention_decode_shared_fp4, codes, {}, "k_cache: shape"),
                           (pa.paged_attention_decode_shared_fp4, rec, dict(v_scale=g[:3]), "v_scale: shape"),
                           (pa.paged_attention_decode_shared_fp4, rec, {}, "q: a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            fn(**(quant | dict(k_cache=c, v_cache=c) | kw))


@pytest.mark.parametrize("kind", KINDS)
def test_reference_against_the_oracle(kind, oracle_mod):
    """The float64 reference of the GPU tests equals the oracle over every sequence's own table."""
    b = Batch(3, [(64, [1, 20, None]), (0, [9]), (32, [0, 40])], 12, 2, 128, 16, kind)
    ref, tol = b.reference()
    if kind == "fp4":
        vals = [b.rows(w, np.arange(b.pages * b.bs)).astype(np.float32).reshape(b.pages, b.bs, 2, 128) for w in (0, 1)]
        k, v = (torch.from_numpy(x).to(torch.bfloat16) for x in vals)  # (rounds the head scale's product)
        want = oracle_mod.paged_attention(b.q, k, v, b.table, b.lens, b.scale)
        assert np.abs(want - ref).max() < 0.05
        return
    if kind == "bf16":
        want = oracle_mod.paged_attention(b.q, b.k, b.v, b.table, b.lens, b.scale)
    else:
        want = oracle_mod.paged_attention_fp8(b.q, torch.from_numpy(b.k), torch.from_numpy(b.v), torch.from_numpy(b.g[0]),
                                              torch.from_numpy(b.g[1]), b.table, b.lens, b.scale)
    # (the scale is binary32 there)
    assert np.abs(want - ref).max() < 1e-6
