"""NaN over an fp4 cache where a whole split sees nothing else: a NaN in q, and
NaN scales in every key of a split.  The splits' records are merged by two
kernels (up to 8 splits, and more); either has to pass the NaN on."""
import numpy as np
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build
from tests import fp4_ref as ref
from tests.test_gpu_fp4 import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    pa.load_library()


def check_nan(p, **kw):
    """NaN where the formula has it, and nowhere else; the rest within the tolerance."""
    with np.errstate(invalid="ignore"):
        want, mag, reach = ref.attention(p.q.float().numpy(), p.k, p.v, p.g, p.table, p.lens, p.scale, p.q_len)
    clean = [np.where(np.isfinite(x), x, 0.0) for x in (mag, reach)]
    bf = kw.get("out_dtype") == pa.PA_OUT_BF16
    # bf16 outputs: each weight off by half a step of f16, 2^-11
    tol = ref.tolerance(*clean, p.d, max(p.lens), bf, want) + (2.0 ** -11 * clean[0] if bf else 0.0)
    assert np.isnan(want).any() and np.isfinite(want).any()
    out, status = p.run(**kw)
    assert status == 0
    assert np.array_equal(np.isnan(out), np.isnan(want))
    live = np.isfinite(want)
    assert (np.abs(out - want)[live] <= tol[live]).all()


@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("splits", [1, 4, 12])
@pytest.mark.parametrize("q_len", [1, 3])
def test_nan_in_q_fills_its_rows(q_len, splits, bf):
    p = Problem(71 + q_len, [1600, 61, 790], 8, 2, 128, 16, q_len=q_len)
    p.q[0, 3, 17] = float("nan")
    p.q[q_len, 0, 0] = float("nan")
    p.q[-1, 6, 5] = float("inf")  # scores of both infinities: NaN by the formula
    check_nan(p, num_splits=splits, out_dtype=pa.PA_OUT_BF16 if bf else pa.PA_OUT_F32)


@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("splits", [4, 12])
@pytest.mark.parametrize("q_len", [1, 3])
def test_a_split_of_nan_keys_fills_its_heads(q_len, splits, bf):
    """Every key of the second split, for one KV head, has a NaN."""
    p = Problem(81 + q_len, [1600, 790], 8, 2, 128, 16, q_len=q_len)
    p.run(num_splits=splits)
    plan = pa.last_plan()
    assert (plan["num_splits"] > 8) == (splits > 8)
    for t in range(16 * plan["chunks_per_split"], 32 * plan["chunks_per_split"]):
        p.k[p.table[0, t // 16], 0, 0, ref.byte_places("k", t % 16, 128)[1]] = 0x7F
    check_nan(p, num_splits=splits, out_dtype=pa.PA_OUT_BF16 if bf else pa.PA_OUT_F32)
