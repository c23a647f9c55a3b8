"""Block-table calls whose buffers overlap are refused before a launch."""
import pytest
import torch

import paged_attention_decode_split_gb300 as pa
from paged_attention_decode_split_gb300 import _build

B, WIDTH, BS, PAGES, ROWS = 2, 4, 16, 8, 5
SIZES = dict(lens=4 * B, count=4 * B, table=4 * B * WIDTH, free=4 * PAGES, num_free=4, lens_out=4 * B, slots=8 * ROWS,
             num_free_out=4)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def call(lib, name, at):
    """`at`: fake addresses, never dereferenced (an overlap is refused on the host)."""
    if name == "extend":
        return lib.pa_extend_block_tables(at["lens"], at["count"], at["table"], at["free"], at["num_free"], B, WIDTH, BS,
                                          PAGES, ROWS, at["lens_out"], at["slots"], at["num_free_out"], None, None)
    return lib.pa_release_block_tables(at["lens"], at["count"], at["table"], at["free"], at["num_free"], B, WIDTH, BS, PAGES,
                                       at["lens_out"], at["num_free_out"], None, None)


@pytest.mark.parametrize("name", ["extend", "release"])
def test_overlapping_buffers_are_refused(lib, name):
    apart = {k: 0x10000 + 0x1000 * i for i, k in enumerate(SIZES)}
    written = {"lens_out", "num_free_out"} | ({"table", "slots"} if name == "extend" else {"free"})
    used = set(SIZES) - (set() if name == "extend" else {"slots"})
    for w in written:
        for other in used - {w}:
            unit = 8 if "slots" in (w, other) else 4
            # the same address, the last element of the one, the first of the other
            for off in {0, SIZES[other] - unit, unit - SIZES[w]}:
                if off % unit == 0 and -SIZES[w] < off < SIZES[other]:
                    assert call(lib, name, apart | {w: apart[other] + off}) == pa.PA_ERR_INVALID_ARG, (w, other, off)


@pytest.mark.gpu
def test_empty_buffers_overlap_nothing():
    """No rows, their address inside another buffer; no requests, no addresses."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    free, out, left, status = i32(*range(8)), i32(-9), i32(-9), i32(0)
    slots = free.view(torch.int64)[1:1]
    table = torch.full((1, 4), 5, dtype=torch.int32, device="cuda")
    pa.extend_block_tables(i32(17), i32(0), table, free, i32(8), 16, out, slots, left, status)
    assert (out.item(), left.item(), status.item()) == (17, 8, 0) and free.tolist() == list(range(8))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    pa.release_block_tables(none, none, table[:0], free, i32(3), 16, none.clone(), left, status)
    assert (left.item(), status.item()) == (3, 0)
