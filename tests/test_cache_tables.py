"""Cache tables on the GPU against a plain loop over requests: equal whole numbers,
over rounds that take pages, keep some tokens and give pages back."""
import numpy as np
import pytest
import torch

import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu


class Plain:
    """The same bookkeeping with Python lists."""

    def __init__(self, R, n_pages, P, width):
        self.kv, self.table, self.P, self.width = [0] * R, [[] for _ in range(R)], P, width
        self.free = list(range(n_pages))

    def reserve(self, n, base, rows):
        P, short = self.P, False
        position, request, slot = [], [], []
        self.new, asked = [], 0
        avail = len(self.free)
        granted = []
        for kv, k in zip(self.kv, n):
            have, want = -(-kv // P), -(-(kv + k) // P)
            need = want - have
            ok = want <= self.width
            if ok:
                ok = need == 0 or asked + need <= avail
                asked += need
            granted.append((ok, need))
            short |= not ok
        for r, (ok, need) in enumerate(granted):
            kv = self.kv[r]
            del self.table[r][-(-kv // P):]
            if ok:
                self.table[r] += [self.free.pop(0) for _ in range(need)]
            for j in range(n[r]):
                p = kv + j
                position.append(base[r] + p if ok else -1)
                request.append(r if ok else -1)
                slot.append(self.table[r][p // P] * P + p % P if ok else -1)
            self.new.append(kv + n[r] if ok else kv)
        pad = [-1] * (rows - len(slot))
        return position + pad, request + pad, slot + pad, short

    def commit(self, keep):
        for r, k in enumerate(keep):
            kept = 0 if k < 0 else min(self.kv[r] + k, self.new[r])
            self.free += self.table[r][-(-kept // self.P):-(-self.new[r] // self.P)]
            self.kv[r] = kept


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


@pytest.mark.parametrize("R,P,n_pages,width,new,pad", [
    (1, 16, 40, 20, 1, 0), (3, 1, 50, 30, 4, 5), (64, 16, 300, 9, 12, 100), (300, 8, 4000, 40, 30, 0),
    (700, 24, 900, 6, 13, 31), (2, 64, 200, 90, 2500, 7), (257, 7, 333, 12, 9, 1025), (5, 16, 6, 50, 20, 3)])
def test_rounds_match_the_plain_bookkeeping(R, P, n_pages, width, new, pad):
    rng = np.random.RandomState(R + P)
    plain, c = Plain(R, n_pages, P, width), vs.cache_tables(R, n_pages, P, width)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for turn in range(8):
        n = rng.randint(0, new + 1, R) * (rng.rand(R) < 0.8)
        base = rng.randint(0, 100, R)
        rows = int(n.sum()) + pad
        position, request, slot, short = plain.reserve(n.tolist(), base.tolist(), rows)
        status.zero_()
        ring_before = c["ring"].clone()
        out = vs.cache_reserve(c, _i32(np.concatenate([[0], np.cumsum(n)])), rows, pos_base=_i32(base), status=status)
        assert out["position"].tolist() == position
        assert out["request"].tolist() == request
        assert out["slot"].tolist() == slot
        assert out["new_len"].tolist() == plain.new
        assert torch.equal(c["ring"], ring_before)
        assert bool(status.item() & vs.STATUS_NO_PAGES) == short and status.item() & ~vs.STATUS_NO_PAGES == 0
        table = c["block_table"].tolist()
        assert all(table[r][:len(t)] == t for r, t in enumerate(plain.table))
        keep = np.where(rng.rand(R) < 0.1, -1, rng.randint(0, new + 3, R))
        plain.commit(keep.tolist())
        done = vs.cache_commit(c, out, _i32(keep), status=status)
        c.update(done)
        assert c["kv_len"].tolist() == plain.kv
        head, tail = c["ring_pos"].tolist()
        ring = c["ring"].tolist()
        assert [ring[i % n_pages] for i in range(head, tail)] == plain.free
        assert status.item() & vs.STATUS_BAD_PAGE == 0


def test_a_repeated_call_repeats_its_outputs():
    c = vs.cache_tables(40, 200, 16, 12)
    off = _i32(np.arange(41) * 7)
    a = vs.cache_reserve(c, off, 280)
    b = vs.cache_reserve(c, off, 280)
    assert all(torch.equal(a[k], b[k]) for k in a)
    keep = _i32(np.arange(40) % 9 - 1)
    ring = [vs.cache_commit(c, a, keep) and c["ring"].clone() for _ in range(2)]
    assert torch.equal(*ring)


def test_bad_lengths_and_pages_are_flagged_and_their_rows_left_out():
    c = vs.cache_tables(4, 30, 16, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["kv_len"].copy_(_i32([5, -3, 0, 17]))
    c["block_table"][0, 0], c["block_table"][3, 0], c["block_table"][3, 1] = 3, 4, 99
    out = vs.cache_reserve(c, _i32([0, 2, 4, 6, 8]), 7, status=status)  # the last request's rows pass the capacity
    assert status.item() == vs.STATUS_BAD_LEN
    assert out["request"].tolist() == [0, 0, -1, -1, 2, 2, -1]
    assert out["new_len"].tolist() == [7, 0, 2, 17]
    status.zero_()
    out = vs.cache_reserve(c, _i32([0, 2, 4, 6, 8]), 8, status=status)
    assert status.item() == vs.STATUS_BAD_LEN | vs.STATUS_BAD_PAGE
    assert out["slot"].tolist()[6:] == [-1, -1] and out["slot"].tolist()[:2] == [3 * 16 + 5, 3 * 16 + 6]


def test_no_requests_and_no_rows():
    c = vs.cache_tables(3, 10, 4, 5)
    out = vs.cache_reserve(c, _i32([0, 0, 0, 0]), 0)
    assert out["new_len"].tolist() == [0, 0, 0] and out["ring_pos"].tolist() == [0, 10]
    out = vs.cache_reserve(c, _i32([0, 0, 0, 0]), 3)
    assert out["slot"].tolist() == [-1] * 3


def test_runs_on_another_stream_and_in_a_graph():
    c = vs.cache_tables(20, 100, 16, 8)
    off, keep = _i32(np.arange(21) * 3), _i32([2] * 20)
    want = vs.cache_reserve(c, off, 64)
    done = vs.cache_commit(c, want, keep)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vs.cache_reserve(c, off, 64, stream=side)
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = vs.cache_reserve(c, off, 64)
        b = vs.cache_commit(c, a, keep)
    c["block_table"].fill_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], want[k]) for k in want) and all(torch.equal(b[k], done[k]) for k in done)


def test_refusals():
    c = vs.cache_tables(4, 10, 16, 3)
    with pytest.raises(TypeError):
        vs.cache_reserve(c, torch.zeros(5, dtype=torch.int64, device="cuda"), 4)
    with pytest.raises(ValueError):
        vs.cache_reserve(c, _i32([0, 1, 2]), 4)
    with pytest.raises(TypeError):
        vs.cache_reserve(c, torch.zeros(5, dtype=torch.int32), 4)
    with pytest.raises(vs.SpecError):
        vs.cache_reserve(c, _i32([0] * 5), 4, out={**vs.cache_reserve(c, _i32([0] * 5), 4), "ring_pos": c["ring_pos"]})


@pytest.mark.parametrize("R,n", [(40, 30), (100, 3), (200, 1700)])
def test_a_wide_capacity_gives_the_same_rows_and_pads_the_rest(R, n):
    off, width = np.arange(R + 1) * n, 2 * (n // 16 + 2)
    few, many = [vs.cache_tables(R, R * width, 16, width) for _ in range(2)]
    for _ in range(2):
        a, b = vs.cache_reserve(few, _i32(off), R * n), vs.cache_reserve(many, _i32(off), R * n + 330000)
        for key in ("position", "request", "slot"):
            assert torch.equal(b[key][:R * n], a[key]) and torch.all(b[key][R * n:] == -1)
        assert torch.equal(a["new_len"], b["new_len"]) and torch.equal(few["block_table"], many["block_table"])
        assert a["slot"].min() >= 0 and a["slot"].unique().numel() == R * n
        for c, p in ((few, a), (many, b)):
            c.update(vs.cache_commit(c, p, _i32(np.full(R, n - 1))))
        assert torch.equal(few["kv_len"], many["kv_len"]) and torch.equal(few["ring"], many["ring"])
