"""Plain reference of the fp4 cache and of attention over it: numpy, written
from the format's definition, byte by byte, with attention in float64."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
CODE_VALUE = np.concatenate([E2M1, -E2M1])


def e4m3_value(code):
    code = np.asarray(code, dtype=np.int64)
    e, m, s = (code >> 3) & 15, code & 7, np.where(code & 128, -1.0, 1.0)
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return s * np.where((code & 127) == 127, np.nan, v)


_E4M3_POS = e4m3_value(np.arange(127))


def nearest_even(x, points):
    """Index of the nearest of ascending points, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(points, x), 0, len(points) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up = x - points[lo], points[hi] - x
    return np.where(down == up, np.where(lo % 2 == 0, lo, hi), np.where(down < up, lo, hi))


def quantise(x, g):
    """Rows [n, hkv, d] float32 and head scales [hkv] float32 -> codes [n, hkv, d]
    (0..15) and scale codes [n, hkv, d / 16]."""
    f32 = np.float32
    x = np.asarray(x, f32).reshape(*x.shape[:2], -1, 16)
    g = np.asarray(g, f32)[None, :, None]
    nan = np.isnan(x).any(-1)
    with np.errstate(all="ignore"):
        want = np.abs(np.where(nan[..., None], f32(0), x)).max(-1) / (f32(6) * g)
        scale = nearest_even(np.minimum(want.astype(np.float64), 448.0), _E4M3_POS)
        s = _E4M3_POS[scale].astype(f32)
        v = x * (f32(1) / (s * g))[..., None]
        codes = nearest_even(np.minimum(np.abs(v.astype(np.float64)), 6.0), E2M1) + 8 * np.signbit(v)
    codes = np.where((nan | (s == 0))[..., None], 0, codes)
    return codes.reshape(*codes.shape[:2], -1), np.where(nan, 0x7F, scale)


def byte_places(kind, t, d):
    """Where the code bytes (dims 0-1, 2-3, ...) and the scale bytes of the t-th
    token stand in a record."""
    codes, scales = [], []
    for dim in range(0, d, 2):
        blk = dim // 16
        if kind == "k":
            codes.append((blk // 8 * 2 + t // 8) * 512 + t % 8 * 64 + dim % 16 // 4 * 16 + blk % 8 * 2 + dim % 4 // 2)
        else:
            u = t // 8 * 2 + t % 2
            codes.append(u * 2 * d + (dim % 16 // 2 * 4 + t % 8 // 2) * (d // 16) + blk)
    for blk in range(d // 16):
        if kind == "k":
            scales.append(8 * d + t * (d // 16) + blk)
        else:
            scales.append(8 * d + blk // 4 * 64 + t % 8 // 2 * 16 + blk % 4 * 4 + t // 8 * 2 + t % 2)
    return np.array(codes), np.array(scales)


def write_rows(kind, rows, g, cache, slots):
    """reshape_and_cache: quantise bf16/float rows [n, hkv, d] into the uint8
    cache [p, hkv, bs / 16, 9 d], in place."""
    pages, hkv, chunks, rec = cache.shape
    d, bs = rec // 9, chunks * 16
    codes, scales = quantise(rows, g)
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    for i, s in enumerate(slots):
        if s < 0 or s >= pages * bs:
            continue
        page, pos = divmod(int(s), bs)
        at_c, at_s = byte_places(kind, pos % 16, d)
        for h in range(hkv):
            cache[page, h, pos // 16][at_c] = packed[i, h]
            cache[page, h, pos // 16][at_s] = scales[i, h].astype(np.uint8)


def read_rows(kind, cache, slots, g=None):
    """The values at the given slots, float64 [n, hkv, d]: code * S (* g)."""
    pages, hkv, chunks, rec = cache.shape
    d, bs = rec // 9, chunks * 16
    out = np.zeros((len(slots), hkv, d))
    slots = np.asarray(slots, dtype=np.int64)
    places = [byte_places(kind, t, d) for t in range(16)]
    for t in range(16):
        mine = np.nonzero((slots >= 0) & (slots < pages * bs) & (slots % 16 == t))[0]
        if not len(mine):
            continue
        rows = cache[slots[mine] // bs, :, slots[mine] % bs // 16]  # [m, hkv, rec]
        byte, sc = rows[..., places[t][0]], e4m3_value(rows[..., places[t][1]])
        v = np.stack([CODE_VALUE[byte & 15], CODE_VALUE[byte >> 4]], -1).reshape(*byte.shape[:2], d)
        out[mine] = v * np.repeat(sc, 16, -1)
    return out if g is None else out * np.asarray(g, np.float64)[None, :, None]


def random_cache(rng, pages, block_size, hkv, d, g):
    """A cache of N(0, 1) rows quantised with head scales g (one numpy Generator)."""
    k = np.empty((pages, hkv, block_size // 16, 9 * d), np.uint8)
    v = np.empty_like(k)
    for kind, cache, scale in (("k", k, g[0]), ("v", v, g[1])):
        codes, scales = quantise(rng.standard_normal((pages * block_size, hkv, d)).astype(np.float32), scale)
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
        for t in range(16):
            at_c, at_s = byte_places(kind, t, d)
            rows = packed[t::16].reshape(pages, block_size // 16, hkv, -1).transpose(0, 2, 1, 3)
            cache[..., at_c] = rows
            cache[..., at_s] = scales[t::16].reshape(pages, block_size // 16, hkv, -1).transpose(0, 2, 1, 3)
    return k, v


def slots_of(table_row, length, block_size):
    t = np.arange(length)
    return np.asarray(table_row, np.int64)[t // block_size] * block_size + t % block_size


def attention(q, k_cache, v_cache, g, table, lens, scale, q_len=1, window=0):
    """Softmax attention in float64 over the cached values: (out, weighted |v|,
    largest sum |q k| scale), each [rows, hq, ...]."""
    rows, hq, d = q.shape
    hkv, bs = k_cache.shape[1], k_cache.shape[2] * 16
    grp = hq // hkv
    out, mag, reach = np.zeros((rows, hq, d)), np.zeros((rows, hq, d)), np.zeros((rows, hq))
    q = np.asarray(q, np.float64)
    for b, n in enumerate(lens):
        if n < max(1, q_len):
            continue
        s = slots_of(table[b], n, bs)
        k, v = read_rows("k", k_cache, s, g[0]), read_rows("v", v_cache, s, g[1])
        for i in range(q_len):
            pos = n - q_len + i
            lo = max(0, pos - window + 1) if window else 0
            for h in range(hq):
                kk, vv = k[lo:pos + 1, h // grp], v[lo:pos + 1, h // grp]
                qr = q[b * q_len + i, h]
                x = kk @ qr * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b * q_len + i, h] = w @ vv
                mag[b * q_len + i, h] = w @ np.abs(vv)
                reach[b * q_len + i, h] = (np.abs(kk) @ np.abs(qr)).max() * abs(scale)
    return out, mag, reach


def tolerance(mag, reach, d, keys, out_bf16, ref):
    """How far a correct kernel's output may be, element by element.

    A score is a sum of d products in binary32: each addition is off by at most
    one step, 2^-23 of sum |q k| (the tensor core may truncate), so a score is
    off by at most e = (d + 4) 2^-23 reach, a weight by a factor within
    1 +- 1.01 e (natural units) +- 2^-21 (exp2 and the f16 head + residual of
    P), and so is their sum; the weighted sum over the keys adds one step per
    16-key product and per merge, at most keys / 16 + 64 of them.  bf16 outputs
    add half a step, 2^-8 relative."""
    e = (d + 4) * 2.0 ** -23 * reach
    rel = 2.02 * e + 2 * 2.0 ** -21 + (keys / 16 + 64) * 2.0 ** -23
    tol = rel[..., None] * mag + 1e-30
    return tol + (np.abs(ref) * 2.0 ** -8 if out_bf16 else 0.0)


def vanished(q, k_cache, v_cache, g, table, lens, scale, q_len=1, window=0):
    """What small weights may lose, element by element.  A weight enters the
    product as two f16 numbers, relative to a reference that gives the largest
    weight of its split 2^7 or more, so its error ends at half the smallest f16,
    2^-25, or at itself: at most min(w, 2^-32 of the largest w) |v|, summed."""
    rows, hq, d = q.shape
    hkv, bs = k_cache.shape[1], k_cache.shape[2] * 16
    off = np.zeros((rows, hq, d))
    q = np.asarray(q, np.float64)
    for b, n in enumerate(lens):
        if n < max(1, q_len):
            continue
        s = slots_of(table[b], n, bs)
        k, v = read_rows("k", k_cache, s, g[0]), np.abs(read_rows("v", v_cache, s, g[1]))
        for i in range(q_len):
            pos = n - q_len + i
            lo = max(0, pos - window + 1) if window else 0
            for h in range(hq):
                x = k[lo:pos + 1, h * hkv // hq] @ q[b * q_len + i, h] * scale
                w = np.exp(x - x.max())
                off[b * q_len + i, h] = np.minimum(w, 2.0 ** -32) @ v[lo:pos + 1, h * hkv // hq] / w.sum()
    return off


def head_scales(hkv):
    """Scales that are no powers of two, one per KV head."""
    h = np.arange(hkv, dtype=np.float32)
    return ((1 + h / 4) / 96).astype(np.float32), ((1 + h / 8) / 80).astype(np.float32)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()
