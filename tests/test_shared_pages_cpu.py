"""Pages with several holders without a GPU: the calls that are refused before
a launch, and the plain forms of perf/more_operators.py against the
request-by-request model that the GPU tests compare the calls with."""
import ctypes
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import shared_pages_model as model


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


@pytest.fixture(scope="module")
def operators():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators_on_cpu", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod._DEV = "cpu"
    return mod


def by_model(s):
    """The outputs of a pass over a prepared fork or compact case, by walking the requests."""
    bs, a = s["case"]["bs"], {k: v.numpy().copy() for k, v in s.items() if isinstance(v, torch.Tensor)}
    num_free = int(s["num_free"])
    if s["case"]["op"] == "compact":
        return model.compact(a["lens"], a["table"], a["free"], num_free, a["shares"], bs, s["case"]["moves"])[0]
    free = a["free"]
    if s["case"]["finished"]:
        r, _ = model.release(a["lens"], a["finished"], a["table"], free, num_free, a["shares"], bs)
        a, free, num_free = a | r, r["free"], r["num_free"]
    return model.fork(a["lens"], a["parent"], a["table"], free, num_free, a["shares"], bs)[0] | dict(free=free)


def copied(s, src, dst, tokens):
    """The caches after the listed copies, by walking the chunks."""
    bs, caches = s["case"]["bs"], [c.clone() for c in s["caches"]]
    for i, (a, b) in enumerate(zip(src, dst)):
        for c in range(bs // 16 if tokens is None else model.pages_of(int(tokens[i]), 16)):
            for x, old in zip(caches, s["caches"]):
                if a >= 0 and s["case"]["cache"] == "fp4":
                    x[b, :, c] = old[a, :, c]
                elif a >= 0:
                    x[b, 16 * c:16 * c + 16] = old[a, 16 * c:16 * c + 16]
    return caches


def check(operators, case, seed):
    s = operators.prepare(case, seed)
    want = by_model(s)
    caches = copied(s, want["src"], want["dst"], want.get("tokens"))
    got = operators.run(s)
    for name in set(got) - {"caches"}:
        assert np.array_equal(got[name].numpy().reshape(np.shape(want[name])), want[name]), name
    for g, w in zip(got["caches"], caches):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


FORK = dict(op="fork", hkv=1, d=128, layers=1)
COMPACT = dict(op="compact", hkv=1, d=128)


@pytest.mark.parametrize("case", [
    FORK | dict(b=8, parents=1, kids=4, bs=16, cache="bf16", len_hi=90, finished=0, short=False),
    FORK | dict(b=30, parents=4, kids=5, bs=16, cache="e4m3", len_hi=200, finished=3, short=True),
    FORK | dict(b=40, parents=3, kids=2, bs=48, cache="fp4", len_hi=48, finished=30, short=False),
    COMPACT | dict(b=9, bs=16, cache="e4m3", pages=70, len_hi=100, moves=100),
    COMPACT | dict(b=9, bs=16, cache="fp4", pages=70, len_hi=100, moves=3),
    COMPACT | dict(b=50, bs=32, cache="bf16", pages=40, len_hi=300, moves=7)])
@pytest.mark.parametrize("seed", range(4))
def test_plain_forms_follow_the_model(operators, case, seed):
    check(operators, case, seed)


def test_plain_forms_of_drawn_cases(operators):
    rng, done = random.Random(1), 0
    while done < 10:
        case = operators.draw(rng)
        if case["op"] in ("fork", "compact"):
            case |= dict(hkv=1, d=128, len_hi=min(case["len_hi"], 900))
            case |= dict(pages=min(case["pages"], 200), moves=min(case["moves"], 50)) if case["op"] == "compact" else {}
            check(operators, case, done)
            done += 1


B, WIDTH, BS, PAGES, MOVES = 2, 4, 16, 8, 3
SIZES = {
    "fork": dict(lens=B, parent=B, table=B * WIDTH, free=PAGES, num_free=1, shares=PAGES, lens_out=B, shares_out=PAGES,
                 src=B, dst=B, tokens=B, num_out=1),
    "release": dict(lens=B, finished=B, table=B * WIDTH, free=PAGES, num_free=1, shares=PAGES, lens_out=B,
                    shares_out=PAGES, num_out=1),
    "compact": dict(lens=B, table=B * WIDTH, free=PAGES, num_free=1, shares=PAGES, free_out=PAGES, num_out=1,
                    shares_out=PAGES, map=PAGES, src=MOVES, dst=MOVES, extent=1)}
WRITTEN = {"fork": {"table", "lens_out", "shares_out", "src", "dst", "tokens", "num_out"},
           "release": {"free", "lens_out", "shares_out", "num_out"},
           "compact": {"table", "free_out", "num_out", "shares_out", "map", "src", "dst", "extent"}}


def call(lib, name, at, B=B, width=WIDTH, bs=BS, pages=PAGES, moves=MOVES):
    """`at`: fake addresses, never dereferenced."""
    v = [at[k] for k in SIZES[name]]
    if name == "fork":
        return lib.pa_fork_block_tables(*v[:6], B, width, bs, pages, *v[6:], None, None)
    if name == "release":
        return lib.pa_release_shared_block_tables(*v[:6], B, width, bs, pages, *v[6:], None, None)
    return lib.pa_compact_block_tables(*v[:5], B, width, bs, pages, moves, *v[5:], None, None)


@pytest.mark.parametrize("name", list(SIZES))
def test_table_calls_refuse(lib, name):
    apart = {k: 0x10000 + 0x1000 * i for i, k in enumerate(SIZES[name])}
    for k in apart:
        assert call(lib, name, apart | {k: None}) == pa.PA_ERR_INVALID_ARG, k
        assert call(lib, name, apart | {k: apart[k] + 2}) == pa.PA_ERR_INVALID_ARG, k
    for kw in (dict(B=-1), dict(width=-1), dict(bs=0), dict(pages=0), dict(moves=-1)):
        if name == "compact" or "moves" not in kw:
            assert call(lib, name, apart, **kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(B=65536), dict(pages=1 << 31), dict(width=1 << 20, bs=4096)):
        assert call(lib, name, apart, **kw) == pa.PA_ERR_UNSUPPORTED, kw
    sizes = {k: 4 * n for k, n in SIZES[name].items()}
    for w in WRITTEN[name]:
        for other in set(sizes) - {w}:
            # the same address, the last element of the one, the first of the other
            for off in {0, sizes[other] - 4, 4 - sizes[w]}:
                assert call(lib, name, apart | {w: apart[other] + off}) == pa.PA_ERR_INVALID_ARG, (w, other, off)


def test_copies_refuse(lib):
    F = 0x10000
    ptrs = (ctypes.c_void_p * 2)(F, 2 * F)
    good = dict(caches=ptrs, n=2, src=F, dst=F, tokens=None, pairs=3, parts=1, chunk=4096, bs=16, pages=9)
    def copy(**kw):
        a = good | kw
        return lib.pa_copy_cache_pages(a["caches"], a["n"], a["src"], a["dst"], a["tokens"], a["pairs"], a["parts"],
                                       a["chunk"], a["bs"], a["pages"], None, None)
    for kw in (dict(n=-1), dict(pairs=-1), dict(parts=0), dict(chunk=0), dict(bs=0), dict(pages=0), dict(caches=None),
               dict(src=None), dict(dst=None), dict(src=F + 2), dict(tokens=F + 1), dict(caches=(ctypes.c_void_p * 2)(F, None)),
               dict(caches=(ctypes.c_void_p * 2)(F, F + 8))):
        assert copy(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(n=pa.PA_MAX_COPY_CACHES + 1), dict(bs=24), dict(chunk=24), dict(pages=1 << 31), dict(chunk=1 << 40),
               dict(chunk=1 << 30, bs=1 << 25, parts=1 << 20)):
        assert copy(**kw) == pa.PA_ERR_UNSUPPORTED, kw
    assert copy(n=0) == pa.PA_OK and copy(pairs=0) == pa.PA_OK  # nothing to copy


def test_binding_refuses(lib):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = dict(block_table=i(2, 4), free_pages=i(8), num_free=i(1), share_counts=i(8), block_size=16,
                share_counts_out=i(8), num_free_out=i(1))
    fork = pool | dict(seq_lens=i(2), parent=i(2), seq_lens_out=i(2), copy_src=i(2), copy_dst=i(2), copy_tokens=i(2))
    rel = pool | dict(seq_lens=i(2), finished=i(2), seq_lens_out=i(2))
    comp = pool | dict(seq_lens=i(2), free_pages_out=i(8), page_map=i(8), copy_src=i(5), copy_dst=i(5), extent=i(1))
    for fn, good, bads in (
            (pa.fork_block_tables, fork, ((dict(parent=i(3)), "parent: shape"), (dict(copy_dst=i(1)), "copy_dst: shape"),
                                          (dict(copy_tokens=i(2).long()), "copy_tokens: dtype"))),
            (pa.release_shared_block_tables, rel, ((dict(finished=i(3)), "finished: shape"),)),
            (pa.compact_block_tables, comp, ((dict(copy_dst=i(4)), "copy_dst: shape"), (dict(page_map=i(7)), "page_map: shape"),
                                             (dict(free_pages_out=i(9)), "free_pages_out: shape"), (dict(extent=i(2)), "extent: shape")))):
        for bad, msg in bads + ((dict(share_counts=i(7)), "share_counts: shape"), (dict(share_counts_out=i(9)), "share_counts_out: shape"),
                                (dict(num_free=i(2)), "num_free: shape"), (dict(block_table=i(8)), "block_table: a"),
                                (dict(seq_lens=i(3)), "seq_lens: shape"), (dict(block_size=0), "block_size"),
                                (dict(), "seq_lens: a CUDA tensor")):
            with pytest.raises(ValueError, match=msg):
                fn(**(good | bad))
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    bf, codes = z(8, 16, 2, 128), z(8, 16, 2, 128, t=torch.uint8)
    for args, msg in ((([], i(1), i(1)), "caches: at least"), (([bf] * 129, i(1), i(1)), "caches: at most"),
                      (([bf, codes], i(1), i(1)), "caches: dtype"), (([bf, bf[:4]], i(1), i(1)), "caches: shape"),
                      (([bf.float()], i(1), i(1)), "caches: dtype"), (([bf], i(1), i(2)), "copy_dst: shape"),
                      (([bf], i(1).long(), i(1)), "copy_src: dtype"), (([bf], i(1), i(1), i(2)), "copy_tokens: shape"),
                      (([bf[0]], i(1), i(1)), "caches: 4"), (([bf], i(1), i(1)), "caches: a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            pa.copy_cache_pages(*args)
    with pytest.raises(ValueError, match="caches: dtype"):
        pa.copy_cache_pages_fp4([bf], i(1), i(1))
