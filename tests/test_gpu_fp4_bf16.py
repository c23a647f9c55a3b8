"""bf16 outputs over an fp4 cache: these are kernels of their own (the weights
enter the second product as one f16), at the shapes, masks and values where the
fp32 ones are tested.

Tolerance: that of fp32 outputs (fp4_ref.tolerance, fp4_ref.vanished), half a
step of the bf16 output (in fp4_ref.tolerance), and half a step of f16, 2^-11,
for each weight: 2^-11 of the sum of |weight v| at most."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import fp4_ref as ref
from tests.test_gpu_fp4 import Problem

pytestmark = pytest.mark.gpu

BF16 = dict(out_dtype=pa.PA_OUT_BF16)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def check(p, runs, window=0):
    args = (p.q.float().numpy(), p.k, p.v, p.g, p.table, p.lens, p.scale, p.q_len, window)
    with np.errstate(invalid="ignore"):
        want, mag, reach = ref.attention(*args)
        off = ref.vanished(*args)
    mag, reach, off = (np.where(np.isfinite(x), x, 0.0) for x in (mag, reach, off))
    tol = ref.tolerance(mag, reach, p.d, max(p.lens), True, want) + off + 2.0 ** -11 * mag
    live = np.isfinite(want)
    for kw in runs:
        out, status = p.run(window=window, **BF16, **kw)
        assert status == 0
        assert np.array_equal(np.isnan(out), ~live)
        worst = (np.abs(out - want)[live] / tol[live]).max()
        assert worst <= 1, (kw, worst)


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("gap", [6, 14, 20])
@pytest.mark.parametrize("hq,hkv,d", [(6, 1, 256), (16, 1, 256), (4, 2, 128), (24, 2, 128)])
def test_small_weights_and_small_scales(hq, hkv, d, gap, q_len):
    """A first key that takes nearly all of the weight and has no value, beside
    keys with 2^-gap of its weight whose block scales are 2^-9 to 2^-4: their
    sum is the output."""
    p = Problem(gap + d + q_len, [600, 90], hq, hkv, d, 16, q_len=q_len)
    rng = np.random.default_rng(gap)
    p.q = torch.from_numpy(1 + 0.1 * rng.standard_normal(p.q.shape).astype(np.float32)).to(torch.bfloat16)
    for b, n in enumerate(p.lens):
        first = [int(p.table[b, 0]) * 16]
        ref.write_rows("k", np.full((1, hkv, d), gap * np.log(2) / np.sqrt(d), np.float32), p.g[0], p.k, first)
        ref.write_rows("v", np.zeros((1, hkv, d), np.float32), p.g[1], p.v, first)
        for t in range(1, n):
            places = ref.byte_places("v", t % 16, d)[1]
            p.v[p.table[b, t // 16], :, 0, places] = rng.integers(1, 0x19, (len(places), hkv))
    check(p, (dict(num_splits=1), dict()))
