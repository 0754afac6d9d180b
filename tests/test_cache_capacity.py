"""The largest capacity: row arrays of 2^31 - 1 entries are written to their ends."""
import numpy as np
import pytest
import torch

import verify_sampling_gb300 as vs


def _blocks(rows, chunk=1024):
    """First row and rows of each of the last blocks, in 32-bit sums as the kernel forms them."""
    n = max(1, (rows + chunk - 1) // chunk)
    for x in range(max(0, n - 3), n):
        b0 = np.int32(x * chunk)
        k = min(chunk, int(np.int32(rows) - b0))
        yield int(b0), k, int(b0) + k


@pytest.mark.parametrize("rows", [0, 1, 1023, 1024, 1025, 2 ** 31 - 1025, 2 ** 31 - 1024, 2 ** 31 - 2, 2 ** 31 - 1])
def test_block_bounds_stay_in_32_bits(rows):
    at = None
    for b0, k, b1 in _blocks(rows):
        assert 0 <= k <= 1024 and b1 < 2 ** 31 and (at is None or b0 == at)
        at = b1
    assert at == rows


@pytest.mark.gpu
def test_every_row_of_the_largest_capacity_is_written():
    rows, off = 2 ** 31 - 1, [0, 3, 5]
    c = vs.cache_tables(2, 10, 4, 5)
    out = {k: torch.full((rows,), 9, dtype=torch.int32, device="cuda") for k in ("position", "request", "slot")}
    out["new_len"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    out["ring_pos"] = torch.zeros(2, dtype=torch.int64, device="cuda")
    vs.cache_reserve(c, torch.tensor(off, dtype=torch.int32, device="cuda"), rows, out=out)
    assert out["request"][:5].tolist() == [0, 0, 0, 1, 1] and out["slot"][:5].tolist() == [0, 1, 2, 4, 5]
    for k in ("position", "request", "slot"):
        for part in out[k][5:].split(1 << 28):
            assert torch.all(part == -1)
    del out
    torch.cuda.empty_cache()
