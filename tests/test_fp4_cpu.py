"""Host-side checks of the fp4 cache and block-table entry points (nothing here
launches a kernel), and pins of the reference the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import fp4_ref as ref

FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def desc(**kw):
    base = dict(num_seqs=1, num_q_heads=24, num_kv_heads=4, head_dim=256, block_size=16, max_pages_per_seq=4,
                max_seq_len=64, num_pages=8, scale=1 / 16, num_sms=152)
    base.update(kw)
    return pa.make_desc(**base)


# -- the reference --------------------------------------------------------------------------------

@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_record_places_fill_the_record_once(kind, d):
    places = np.concatenate([np.concatenate(ref.byte_places(kind, t, d)) for t in range(16)])
    assert np.array_equal(np.sort(places), np.arange(9 * d))


def test_reference_conversions_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(ref.e4m3_value(codes.numpy()), codes.view(torch.float8_e4m3fn).float().double().numpy(),
                          equal_nan=True)
    x = torch.linspace(0, 448, 9001)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_even(x.double().numpy(), ref._E4M3_POS), want)


def test_reference_quantiser_by_hand():
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5]
    x[0, 0, 16:19] = [1e9, -1e9, 1.0]
    x[0, 0, 40] = np.nan
    codes, scales = ref.quantise(x, np.ones(1, np.float32))
    assert scales[0, 0].tolist() == [0x38, 0x7E, 0x7F, 0, 0, 0, 0, 0]  # 1, 448, NaN, zeros
    assert codes[0, 0, :16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 15, 8, 10, 10, 12, 12, 14, 14]  # ties to even
    assert codes[0, 0, 16:19].tolist() == [7, 15, 0] and not codes[0, 0, 32:].any()


def test_reference_rows_round_trip():
    rng = np.random.default_rng(0)
    for kind in "kv":
        cache = rng.integers(0, 256, (2, 2, 3, 9 * 128), dtype=np.uint8)
        before, slots = cache.copy(), [95, 0, 17, 33, -1, 96]
        x = rng.integers(-3, 4, (6, 2, 128)).astype(np.float32) * 2
        x[..., ::16] = 6.0  # every block's scale is g
        ref.write_rows(kind, x, np.array([1.0, 0.5], np.float32), cache, slots)
        got = ref.read_rows(kind, cache, slots, np.array([1.0, 0.5], np.float32))
        assert np.array_equal(got[:4], x[:4]) and not got[4:].any()
        others = [s for s in range(96) if s not in slots]
        assert np.array_equal(ref.read_rows(kind, cache, others), ref.read_rows(kind, before, others), equal_nan=True)


# -- refusals -------------------------------------------------------------------------------------

def test_attention_entries_refuse(lib):
    for name in ("pa_paged_attention_decode_fp4", "pa_paged_attention_verify_fp4"):
        fn = getattr(lib, name)
        q_len = 1 if "decode" in name else 4
        args = lambda ks, vs, dd, kc=FAKE: (FAKE, kc, FAKE, ks, vs, FAKE, FAKE, ctypes.byref(dd), FAKE, FAKE, 1 << 30,  # noqa: E731
                                            None, None)
        ok = desc(q_len=q_len)
        assert fn(*args(None, FAKE, ok)) == pa.PA_ERR_INVALID_ARG
        assert fn(*args(FAKE, None, ok)) == pa.PA_ERR_INVALID_ARG
        assert fn(*args(FAKE, FAKE + 2, ok)) == pa.PA_ERR_INVALID_ARG
        assert fn(*args(FAKE, FAKE, ok, None)) == pa.PA_ERR_INVALID_ARG
        assert fn(*args(FAKE, FAKE, ok, FAKE + 8)) == pa.PA_ERR_INVALID_ARG
        assert fn(*args(FAKE, FAKE, desc(q_len=q_len, head_dim=64))) == pa.PA_ERR_UNSUPPORTED
        assert fn(*args(FAKE, FAKE, desc(q_len=q_len, block_size=24, max_pages_per_seq=9))) == pa.PA_ERR_UNSUPPORTED
        assert fn(*args(FAKE, FAKE, desc(q_len=q_len, flags=2))) == pa.PA_ERR_INVALID_ARG
    big = desc(block_size=784, max_pages_per_seq=42, max_seq_len=32768, num_pages=46)
    need = pa.workspace_bytes(big)
    assert lib.pa_paged_attention_decode_fp4(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(big), FAKE, FAKE,
                                             need - 1, None, None) == pa.PA_ERR_WORKSPACE
    app = lib.pa_paged_attention_decode_append_fp4
    tail = (FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(desc()), FAKE, FAKE, 1 << 30, None, None)
    assert app(FAKE, None, FAKE, *tail) == pa.PA_ERR_INVALID_ARG
    assert app(FAKE, FAKE, FAKE + 4, *tail) == pa.PA_ERR_INVALID_ARG
    assert app(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, ctypes.byref(desc()), FAKE, FAKE, 1 << 30, None,
               None) == pa.PA_ERR_INVALID_ARG


def test_row_entries_refuse(lib):
    def write(n=1, hkv=4, d=256, bs=16, p=8, k=FAKE, slots=FAKE, ks=FAKE):
        return lib.pa_reshape_and_cache_fp4(k, FAKE, FAKE, FAKE, slots, ks, FAKE, n, hkv, d, bs, p, None, None)

    def read(n=1, hkv=4, d=256, bs=16, p=8, out=FAKE, slots=FAKE, dtype=0):
        return lib.pa_gather_cache_fp4(FAKE, FAKE, slots, FAKE, FAKE, out, FAKE, dtype, n, hkv, d, bs, p, None, None)

    for fn in (write, read):
        assert fn(n=-1) == fn(hkv=0) == fn(p=0) == fn(bs=0) == pa.PA_ERR_INVALID_ARG
        assert fn(d=64) == fn(d=192) == fn(bs=20) == pa.PA_ERR_UNSUPPORTED
        assert fn(slots=None) == fn(slots=FAKE + 4) == pa.PA_ERR_INVALID_ARG
        assert fn(n=0, slots=None) == pa.PA_OK
    assert write(k=FAKE + 8) == write(ks=None) == write(ks=FAKE + 2) == pa.PA_ERR_INVALID_ARG
    assert read(out=None) == read(out=FAKE + 8) == read(dtype=2) == pa.PA_ERR_INVALID_ARG


def test_table_entries_refuse(lib):
    def extend(lens=FAKE, new=FAKE, table=FAKE, free=FAKE, num=FAKE, B=2, width=4, bs=16, P=8, N=5, out=FAKE + 64,
               slots=FAKE, num_out=FAKE + 64):
        return lib.pa_extend_block_tables(lens, new, table, free, num, B, width, bs, P, N, out, slots, num_out, None,
                                          None)

    def release(lens=FAKE, done=FAKE, table=FAKE, free=FAKE, num=FAKE, B=2, width=4, bs=16, P=8, out=FAKE + 64,
                num_out=FAKE + 64):
        return lib.pa_release_block_tables(lens, done, table, free, num, B, width, bs, P, out, num_out, None, None)

    for fn in (extend, release):
        for bad in (dict(B=-1), dict(width=-1), dict(bs=0), dict(P=0), dict(lens=None), dict(free=None),
                    dict(table=None), dict(num=None), dict(num_out=None), dict(out=None), dict(lens=FAKE + 2),
                    dict(out=FAKE), dict(num_out=FAKE)):
            assert fn(**bad) == pa.PA_ERR_INVALID_ARG, bad
        assert fn(B=65536) == fn(P=2 ** 31) == fn(width=2 ** 27, bs=16) == pa.PA_ERR_UNSUPPORTED
    assert extend(N=-1) == extend(slots=None) == extend(slots=FAKE + 4) == extend(new=None) == pa.PA_ERR_INVALID_ARG


def test_binding_refuses(lib):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    shape = pa.fp4_cache_shape(8, 16, 4, 256)
    assert shape == (8, 4, 1, 2304)
    with pytest.raises(ValueError):
        pa.fp4_cache_shape(8, 20, 4, 256)
    q, out, g = z(1, 24, 256), z(1, 24, 256, t=torch.float32), torch.ones(4)
    rec, codes = z(*shape, t=torch.uint8), z(8, 16, 4, 256, t=torch.uint8)
    bt, sl = z(1, 4, t=torch.int32), z(1, t=torch.int32)
    for args, msg in (((q, codes, codes, g, g), "k_cache: shape"), ((q, z(*shape), rec, g, g), "k_cache: dtype"),
                      ((q, rec, codes, g, g), "v_cache: shape"), ((q, rec, rec, None, g), "an fp4 cache needs both"),
                      ((q, rec, rec, g, torch.ones(3)), "v_scale: shape"), ((q, rec, rec, g, g), "q: a CUDA tensor")):
        for fn in (pa.paged_attention_decode_fp4, pa.paged_attention_verify_fp4):
            with pytest.raises(ValueError, match=msg):
                fn(*args, bt, sl, desc(), out)
    with pytest.raises(ValueError, match="k_new: shape"):
        pa.paged_attention_decode_append_fp4(q, z(1, 2, 256), z(1, 4, 256), rec, rec, g, g, bt, sl, desc(), out)
    with pytest.raises(ValueError, match="k_cache: dtype"):  # an fp4 cache is no fp8 or bf16 cache
        pa.paged_attention_decode(q, rec, rec, bt, sl, desc(), out)
    slots, rows = z(3, t=torch.int64), z(3, 4, 256)
    for args, msg in (((rows, rows, rec, rec, slots.int(), g, g), "slot_mapping: dtype"),
                      ((rows[:2], rows, rec, rec, slots, g, g), "k_new: shape"),
                      ((rows.float(), rows, rec, rec, slots, g, g), "k_new: dtype"),
                      ((rows, rows, rec, rec[:4], slots, g, g), "v_cache: shape"),
                      ((rows, rows, codes, codes, slots, g, g), "k_cache: a .pages"),
                      ((rows, rows, rec, rec, slots, g.double(), g), "k_scale: dtype"),
                      ((rows, rows, rec, rec, slots, g, g), "k_new: a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            pa.reshape_and_cache_fp4(*args)
    with pytest.raises(ValueError, match="v_out: dtype"):
        pa.gather_cache_fp4(rec, rec, slots, g, g, rows, rows.float())
    with pytest.raises(ValueError, match="k_out: shape"):
        pa.gather_cache_fp4(rec, rec, slots, g, g, rows[:1], rows)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(context_lens=i(2), num_new=i(2), block_table=i(2, 4), free_pages=i(8), num_free=i(1), block_size=16,
                seq_lens=i(2), slot_mapping=slots, num_free_out=i(1))
    for bad, msg in ((dict(context_lens=i(3)), "context_lens: shape"), (dict(num_new=slots[:2]), "num_new: dtype"),
                     (dict(block_table=i(8)), "block_table: a"), (dict(num_free=i(2)), "num_free: shape"),
                     (dict(slot_mapping=i(3)), "slot_mapping: dtype"), (dict(block_size=0), "block_size"),
                     (dict(), "context_lens: a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            pa.extend_block_tables(**(good | bad))
    rel = dict(seq_lens=i(2), finished=i(2), block_table=i(2, 4), free_pages=i(8), num_free=i(1), block_size=16,
               seq_lens_out=i(2), num_free_out=i(1))
    for bad, msg in ((dict(finished=i(3)), "finished: shape"), (dict(seq_lens_out=i(1)), "seq_lens_out: shape"),
                     (dict(), "seq_lens: a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            pa.release_block_tables(**(rel | bad))
