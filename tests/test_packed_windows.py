"""Calls of more than 2^20 query rows over a cache in 4 bits, which run in windows: by the narrow kernel alone, with 8 and with 16 query
rows an item, and by both kernels where segments of up to 16 query rows and of more meet."""
import pytest
import torch

import verify_sampling_gb300 as vs
from test_packed_attention import BF, Case

pytestmark = pytest.mark.gpu


def _run(c, pick):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(c.q, 3.0)
    got, lse = c.call(want_lse=True, status=st, out=out)
    assert st.item() == 0
    c.check(got, lse, sorted(set(pick)))
    assert bool(torch.isfinite(got.float()).all()) and torch.all(got[c.off[-1]:] == 3)


def _near_border(off, rows, Hq):
    """Requests on both sides of each window's border."""
    most = (1 << 20) // Hq
    windows = -(-rows // most)
    step = -(-rows // windows)
    at = [int((torch.tensor(off) <= step * w).sum()) - 1 for w in range(1, windows)]
    return [r + d for r in at for d in (-2, -1, 0, 1, 2) if 0 <= r + d < len(off) - 1]


def _lengths(R, each):
    """Own keys: short, and now and then of several tiles."""
    return [each + (i * 37) % 20 + (650 if i % 499 == 3 else 0) for i in range(R)]


@pytest.mark.parametrize("each,Hq,Hk,D", [(1, 64, 16, 64), (1, 64, 16, 128), (3, 64, 16, 64), (1, 128, 16, 128), (2, 128, 16, 64)])
def test_few_rows_a_request(each, Hq, Hk, D):
    """At most 12 to 16 query rows of a key head a request, and so one kernel: the first two with items of 8 rows."""
    R = (1 << 20) // Hq // each + 700
    n = [each] * R
    if each * Hq // Hk == 16:
        n[R // 3] = 0  # makes room for the row of no request
    kv = _lengths(R, each)
    c = Case(n, kv, Hq, Hk, D, 8, BF)
    assert c.rows * Hq > 1 << 20 and c.rows * (Hq // Hk) <= 16 * R
    _run(c, _near_border(c.off, c.rows, Hq) + [0, 1, 3, R // 3, R // 3 + 1, R - 1] + [(i * 7919) % R for i in range(40)] + [3 + 499 * i for i in range(R // 499)][:12])


@pytest.mark.parametrize("D,groups", [(64, True), (128, True), (64, False)])
def test_segments_of_few_and_of_many_rows(D, groups):
    Hq, Hk, each = 64, 8, 2
    R = (1 << 20) // Hq // each + 100
    n = [40 if i % 61 == 7 else 17 if i % 61 == 30 else each for i in range(R)]
    if not groups:
        n = [max(2, v) if i % 2 else 3 for i, v in enumerate(n)]
    kv = [max(a, b) for a, b in zip(n, _lengths(R, each))]
    c = Case(n, kv, Hq, Hk, D, 16, BF, ((R // 3, 130), (2, 300), (1, 700)) if groups else ())
    assert c.rows * Hq > 1 << 20
    many = [i for i in range(R) if n[i] > 2][:8]
    _run(c, _near_border(c.off, c.rows, Hq) + [0, 1, R // 3 - 1, R // 3, R // 3 + 2, R // 3 + 3, R - 1] + many + [(i * 7919) % R for i in range(40)])
