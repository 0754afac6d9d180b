"""The attention's workspace is bounded: calls of many rows run in windows of packed rows, with the same results."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import verify_sampling_gb300 as vs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32
PIECES = (2 << 20) + (1 << 16)  # rows of partial results at most: D + 2 floats each


@pytest.fixture(scope="module")
def built():
    if not os.path.exists(vs.LIB_PATH):
        from verify_sampling_gb300 import build
        build.build()


@pytest.mark.parametrize("rows,R,Hq,D", [(497011, 250, 64, 128), (32768, 1, 64, 128), (2 ** 31 // 1024 - 1, 65535, 1024, 256),
                                         (2 ** 30, 1, 1, 64), (2 ** 31 - 1, 65535, 1, 256), (1 << 20, 1, 1, 128)])
def test_workspace_of_many_rows_is_bounded(built, rows, R, Hq, D):
    assert 0 < vs.attention_workspace_bytes(rows, R, Hq, D) <= PIECES * (D + 2) * 4 + (2 * R + 2) * 8 + 768


@pytest.mark.parametrize("rows,R,Hq,D", [(1, 1, 32, 128), (1664, 256, 64, 128), (4096, 512, 64, 128)])
def test_workspace_of_few_rows_is_as_it_was(built, rows, R, Hq, D):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    pieces = 2 * rows * Hq + (1 << 16)
    assert vs.attention_workspace_bytes(rows, R, Hq, D) == up(pieces * D * 4) + up(pieces * 8) + up((2 * R + 2) * 8)


def _case(*args, **kw):
    spec = importlib.util.spec_from_file_location("prefix_cases", os.path.join(ROOT, "tests", "test_prefix_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.Case(*args, **kw), m


# rows * Hq above 2^20: two windows or three, cut inside requests, between them, and where nothing is
WINDOWS = [
    # n, kv, Hq, Hk, D, P, groups
    ([700, 1, 0, 420, 3, 300], [900, 77, 5, 420, 200, 250], 1024, 8, 64, 16, ((2, 130), (3, 300))),
    ([1100, 50], [1100, 700], 1024, 16, 128, 64, ()),
    ([2, 5, 3] * 300, [1 + (i * 37) % 90 for i in range(900)], 512, 4, 64, 16, ((450, 70), (400, 200))),
    ([4500], [4500], 256, 2, 64, 128, ((1, 33),)),
    ([600, 700], [700, 400], 1020, 4, 64, 32, ((1, 64),)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("n,kv,Hq,Hk,D,P,groups", WINDOWS)
def test_rows_of_several_windows_match_64_bits(n, kv, Hq, Hk, D, P, groups):
    c, m = _case(n, kv, Hq, Hk, D, P, BF, groups)
    assert c.rows * Hq > 1 << 20
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(c.q, 3.0)
    got, lse = c.call(want_lse=True, status=st, out=out)
    assert st.item() == 0
    few = sorted(set(np.linspace(0, len(n) - 1, 30).astype(int)) | {int(r) for r in np.argsort(n)[-2:]})
    for r in few:  # a request at a time, rows in parts: the check holds all their scores in 64 bits
        full, off = c.n[r], c.off.copy()
        for a in range(0, full, 100):
            b = min(full, a + 100)
            c.n[r], c.off[r], c.off[r + 1], kv_r = b - a, off[r] + a, off[r] + b, c.kv[r]
            c.kv[r] = kv_r - (full - b)
            if c.kv[r] >= 0:
                c.check(got, lse, [r])
            c.kv[r] = kv_r
        c.n[r], c.off = full, off
    assert torch.all(got[c.off[-1]:] == 3)


@pytest.mark.gpu
def test_bad_offsets_among_windows_are_left_out():
    c, _ = _case([600, 2, 2, 700], [650, 9, 8, 700], 1024, 8, 64, 16, BF, ())
    want, lse = c.call(want_lse=True)
    off = c.off.copy()
    for bad in (-5, 10 ** 9):
        c.off = off.copy()
        c.off[2] = bad  # requests 1 and 2 have no rows then
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(c.q, 3.0)
        got, l2 = c.call(want_lse=True, status=st, out=out)
        assert st.item() == vs.STATUS_BAD_LEN
        assert torch.all(got[600:604] == 3)
        # the cuts between blocks lie elsewhere without those rows: bf16 results of sums that differ by rounding
        for a, b in ((0, 600), (604, 1304)):
            x, y = got[a:b].float(), want[a:b].float()
            assert torch.all((x - y).abs() <= 2 * torch.finfo(BF).eps * (1 + x.abs()))
            assert torch.all((l2[a:b] - lse[a:b]).abs() <= 1e-4)
    c.off = off


@pytest.mark.gpu
def test_windows_in_a_graph_and_with_a_given_workspace():
    c, m = _case([1100, 3], [1100, 50], 1024, 8, 64, 16, BF, ((2, 40),))
    need = vs.attention_workspace_bytes(c.rows, 2, 1024, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want, lse = c.call(want_lse=True, workspace=ws)
    args = (c.q, c.k, c.v, m._i32(c.off), m._i32(c.kv), c.block_table)
    kw = dict(scale=c.scale, group_off=m._i32(c.goff), prefix_len=m._i32([40]), prefix_table=c.prefix_table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = vs.prefix_attention(*args, **kw, workspace=ws)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[:c.off[-1]], want[:c.off[-1]])


@pytest.mark.gpu
def test_generic_sizes_of_many_rows():
    c, _ = _case([900, 40, 400], [950, 300, 400], 1024, 8, 24, 16, BF, ((2, 65),))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = c.call(want_lse=True, status=st)
    assert st.item() == 0
    c.check(got, lse, [1])
