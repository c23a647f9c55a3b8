"""Rotary positions without a GPU: the frequency table against the published
definitions, and the calls that are refused before a launch."""
import ctypes
import math

import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build

FAKE = 0x100000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def radians(r, base, scaling, factor, orig, low, high):
    """Radians per position of each pair, pair by pair."""
    got = []
    for j in range(r // 2):
        b = base * factor ** (r / (r - 2)) if scaling == "ntk" and r > 2 else base
        w = b ** (-2 * j / r)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            def pair_of(turns):  # the (real) pair that makes so many turns over the original length
                return r / 2 * math.log(orig / (2 * math.pi * turns)) / math.log(base)
            lo, hi = max(math.floor(pair_of(high)), 0), min(math.ceil(pair_of(low)), r - 1)
            mix = min(1, max(0, (j - lo) / max(hi - lo, 0.001)))
            w = w * (1 - mix) + w / factor * mix
        if scaling == "bands":
            mix = min(1, max(0, (orig * w / (2 * math.pi) - low) / (high - low)))
            w = w * mix + w / factor * (1 - mix)
        got.append(w)
    return got


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
@pytest.mark.parametrize("r", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("base,factor,orig", [(10000.0, 1.0, 2048), (10000.0, 8.0, 8192), (1e6, 4.0, 32768), (1.5, 2.5, 100)])
def test_frequencies_follow_their_definitions(lib, scaling, r, base, factor, orig):
    low, high = 1.0, 4.0 if scaling == "bands" else 32.0
    freqs, rows = pa.rotary_frequencies(r, base=base, scaling=scaling, factor=factor, original_len=orig, device="cpu")
    assert freqs.dtype == torch.int64 and freqs.shape == (r // 2,)
    for f, w in zip(freqs.tolist(), radians(r, base, scaling, factor, orig, low, high)):
        # a dozen operations in 64 bits, each off by half a step; pow and log by a few
        assert abs(f - w / (2 * math.pi) * 2 ** 64) <= 2 ** 64 * w * 2 ** -46 + 1
    assert rows == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=2 ** -23)


def test_frequencies_by_hand(lib):
    freqs, _ = pa.rotary_frequencies(4, base=100.0, device="cpu")
    assert freqs.tolist() == [round(2 ** 64 / (2 * math.pi)), pytest.approx(2 ** 64 / (20 * math.pi), rel=1e-15)]
    # a pair with more turns than high stays, one with fewer than low is stretched
    freqs, _ = pa.rotary_frequencies(128, base=1e4, scaling="bands", factor=8.0, original_len=8192, device="cpu")
    plain, _ = pa.rotary_frequencies(128, base=1e4, device="cpu")
    assert freqs[0] == plain[0] and abs(int(freqs[-1]) * 8 - int(plain[-1])) <= int(plain[-1]) * 2 ** -50 + 8


def test_frequencies_refuse(lib):
    for kw in (dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(scaling="linear", factor=0.5),
               dict(scaling="yarn", factor=2.0, original_len=0), dict(scaling="ntk", factor=float("nan")),
               dict(scaling="bands", factor=2.0, original_len=100, low_turns=4.0, high_turns=4.0),
               dict(scaling="bands", factor=2.0, original_len=100, low_turns=0.0)):
        with pytest.raises(pa.PagedAttnError):
            pa.rotary_frequencies(64, device="cpu", **kw)
    for bad in (0, 7, -2):
        with pytest.raises(ValueError):
            pa.rotary_frequencies(bad, device="cpu")
    with pytest.raises(ValueError, match="scaling"):
        pa.rotary_frequencies(64, scaling="stretch", device="cpu")
    factor = ctypes.c_float()
    assert lib.pa_rotary_frequencies(None, FAKE, ctypes.byref(factor)) == pa.PA_ERR_INVALID_ARG


class Desc(ctypes.Structure):  # pa_rotary_desc
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_tokens", "num_q_heads", "num_kv_heads", "head_dim", "rotary_dim",
                                               "flags", "position_offset")] + [("factor", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride", "k_out_stride")])


def desc(**kw):
    d = dict(num_tokens=3, num_q_heads=8, num_kv_heads=2, head_dim=128, rotary_dim=64, flags=0, position_offset=0,
             factor=1.0, q_stride=1024, k_stride=256, v_stride=256, q_out_stride=1024, k_out_stride=256)
    return Desc(**(d | kw))


# q 3 x 2048 bytes, k and v 3 x 512
Q, K, V, QO, KO = (FAKE + 0x100000 * i for i in range(5))
BAD = [(dict(num_tokens=-1), "arg"), (dict(rotary_dim=144), "arg"), (dict(rotary_dim=0), "arg"), (dict(flags=4), "arg"),
       (dict(factor=float("nan")), "arg"), (dict(num_q_heads=0, num_kv_heads=0), "arg"), (dict(rotary_dim=24), "no"),
       (dict(head_dim=24, rotary_dim=16), "no"), (dict(head_dim=16, rotary_dim=16), "no"), (dict(head_dim=2048), "no"),
       (dict(q_stride=1028), "arg"), (dict(q_out_stride=1016), "arg"), (dict(k_stride=-256), "arg"),
       (dict(q_stride=1 << 31), "no"), (dict(v_stride=1 << 40, q_out_stride=1 << 61), "no")]
CODE = {"arg": pa.PA_ERR_INVALID_ARG, "no": pa.PA_ERR_UNSUPPORTED}


@pytest.mark.parametrize("kw,code", BAD)
def test_calls_refuse_descriptions(lib, kw, code):
    d = desc(**kw)
    assert lib.pa_rotary(Q, K, FAKE, FAKE, QO, KO, ctypes.byref(d), None) == CODE[code]
    assert lib.pa_rotary_and_cache(Q, K, V, FAKE, FAKE, QO, FAKE, FAKE, FAKE, ctypes.byref(d), 16, 4, None,
                                   None) == CODE[code]


def test_calls_refuse_pointers_and_overlaps(lib):
    d = desc()
    call = lambda q=Q, k=K, pos=FAKE, f=FAKE, qo=QO, ko=KO, d=d: lib.pa_rotary(  # noqa: E731
        q, k, pos, f, qo, ko, ctypes.byref(d), None)
    for kw in (dict(q=None), dict(k=None), dict(pos=None), dict(f=None), dict(qo=None), dict(ko=None), dict(q=Q + 8),
               dict(ko=KO + 2), dict(pos=FAKE + 2), dict(f=FAKE + 4)):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert lib.pa_rotary(Q, K, FAKE, FAKE, QO, KO, None, None) == pa.PA_ERR_INVALID_ARG
    # what is written overlaps another argument: a row on, the last vector, another stride, each other
    for kw in (dict(qo=Q + 2048), dict(qo=Q - 2048), dict(qo=Q + 3 * 2048 - 16), dict(qo=K), dict(ko=Q), dict(ko=K + 16),
               dict(ko=QO), dict(ko=QO + 3 * 2048 - 16), dict(qo=K - 3 * 2048 + 16)):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert call(qo=Q, d=desc(q_out_stride=2048)) == pa.PA_ERR_INVALID_ARG
    # one buffer of q, k, v rows: k_out over v's place is refused only where it reaches q or k
    rows = desc(q_stride=1536, k_stride=1536, q_out_stride=1536, k_out_stride=1536)
    assert call(k=Q + 2048, qo=Q, ko=Q + 2048 - 16, d=rows) == pa.PA_ERR_INVALID_ARG
    assert call(k=Q + 2048, qo=Q + 512, ko=Q + 2048, d=rows) == pa.PA_ERR_INVALID_ARG
    # nothing to do
    assert lib.pa_rotary(None, None, None, None, None, None, ctypes.byref(desc(num_tokens=0)), None) == pa.PA_OK
    assert lib.pa_rotary_and_cache(None, None, None, None, None, None, None, None, None,
                                   ctypes.byref(desc(num_tokens=0)), 16, 4, None, None) == pa.PA_OK


def test_cache_calls_refuse(lib):
    def call(fn="", d=desc(), bs=16, pages=4, v=V, kc=FAKE, slots=FAKE, ks=FAKE):
        scales = (ks, FAKE) if fn else ()
        return getattr(lib, "pa_rotary_and_cache" + fn)(Q, K, v, FAKE, FAKE, QO, kc, FAKE, slots, *scales,
                                                       ctypes.byref(d), bs, pages, None, None)
    for fn in ("", "_fp8", "_fp4"):
        for kw in (dict(bs=0), dict(pages=0), dict(v=None), dict(kc=None), dict(kc=FAKE + 8), dict(slots=None),
                   dict(slots=FAKE + 4), dict(d=desc(flags=pa.PA_ROPE_INVERSE)), dict(d=desc(num_kv_heads=0))):
            assert call(fn, **kw) == pa.PA_ERR_INVALID_ARG, (fn, kw)
        assert call(fn, pages=1 << 31) == pa.PA_ERR_UNSUPPORTED
    for fn in ("_fp8", "_fp4"):
        assert call(fn, ks=None) == pa.PA_ERR_INVALID_ARG and call(fn, ks=FAKE + 2) == pa.PA_ERR_INVALID_ARG
    assert call("_fp4", bs=24) == pa.PA_ERR_UNSUPPORTED
    assert call("_fp4", d=desc(head_dim=64, q_stride=512, q_out_stride=512)) == pa.PA_ERR_UNSUPPORTED
    assert call("_fp4", d=desc(num_kv_heads=128, k_stride=1 << 14, v_stride=1 << 14)) == pa.PA_ERR_UNSUPPORTED


def test_binding_refuses(lib):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    q, k, pos, freqs, slots, g = z(3, 8, 128), z(3, 2, 128), z(3, t=torch.int32), z(32, t=torch.int64), z(3, t=torch.int64), torch.ones(2)
    for kw, msg in ((dict(q=z(3, 1024)), "q: a .tokens"), (dict(k=z(2, 2, 128)), "k: shape"), (dict(q=q.float()), "q: dtype"),
                    (dict(k=z(3, 2, 64)), "k: shape"), (dict(positions=slots), "positions: dtype"),
                    (dict(positions=pos[:2]), "positions: shape"), (dict(freqs=freqs.int()), "freqs: dtype"),
                    (dict(q_out=z(3, 8, 64)), "q_out: shape"), (dict(k_out=z(3, 3, 128)), "k_out: shape"),
                    (dict(k_out=None), "k, k_out: both"), (dict(position_offset=1 << 31), "position_offset"),
                    (dict(), "q: a CUDA tensor")):
        args = dict(q=q, k=k, positions=pos, freqs=freqs, q_out=q, k_out=k) | kw
        if torch.cuda.is_available() and not kw:
            continue
        with pytest.raises(ValueError, match=msg):
            pa.rotary(**args)
    cache, codes, rec = z(4, 16, 2, 128), z(4, 16, 2, 128, t=torch.uint8), z(4, 2, 1, 9 * 128, t=torch.uint8)
    base = dict(q=q, k=k, v=k, positions=pos, freqs=freqs, q_out=q, slot_mapping=slots)
    for fn, caches, scales, msg in ((pa.rotary_and_cache, (codes, cache), {}, "k_cache: dtype"),
                                    (pa.rotary_and_cache, (cache, cache[:3]), {}, "v_cache: shape"),
                                    (pa.rotary_and_cache_fp8, (cache, codes), dict(k_scale=g, v_scale=g), "k_cache: dtype"),
                                    (pa.rotary_and_cache_fp8, (codes, codes), dict(k_scale=g, v_scale=None), "needs both"),
                                    (pa.rotary_and_cache_fp8, (codes, codes), dict(k_scale=g[:1], v_scale=g), "k_scale: shape"),
                                    (pa.rotary_and_cache_fp4, (codes, codes), dict(k_scale=g, v_scale=g), "k_cache: shape"),
                                    (pa.rotary_and_cache_fp4, (rec, rec), dict(k_scale=g, v_scale=g.double()), "v_scale: dtype")):
        with pytest.raises(ValueError, match=msg):
            fn(**base, k_cache=caches[0], v_cache=caches[1], **scales)
    with pytest.raises(ValueError, match="v: shape"):
        pa.rotary_and_cache(**(base | dict(v=k[:2])), k_cache=cache, v_cache=cache)
    with pytest.raises(ValueError, match="slot_mapping: dtype"):
        pa.rotary_and_cache(**(base | dict(slot_mapping=pos)), k_cache=cache, v_cache=cache)
