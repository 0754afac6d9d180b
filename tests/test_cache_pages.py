"""Page ids outside the cache never reach the ring of free pages: whoever reserves next gets pages that exist."""
import numpy as np
import pytest
import torch

import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


@pytest.mark.parametrize("R,most,share", [(1, 1, 1.0), (1, 5, 0.5), (3, 40, 0.3), (33, 3, 0.1), (128, 2, 0.05), (129, 30, 0.5),
                                          (300, 9, 0.02), (1500, 4, 0.2), (2500, 2, 0.0), (5, 3000, 0.01), (140, 70, 1.0)])
def test_commit_gives_back_the_pages_that_exist(R, most, share):
    r, P = np.random.RandomState(R * 7 + most), 8
    held = r.randint(0, most + 1, R)
    held[-1] = most
    n_pages = int(held.sum()) + 6
    table = np.full((R, most + 2), 10 ** 9)
    at = r.permutation(n_pages)
    for i in range(R):
        table[i, :held[i]], at = at[:held[i]], at[held[i]:]
    strange = r.rand(R, most + 2) < share
    table = np.where(strange, r.choice([-1, n_pages, n_pages + 7, 2 ** 31 - 1, -2 ** 31], table.shape), table)
    kv = np.maximum(held * P - r.randint(0, P, R), 0) * (held > 0)
    keep = np.where(r.rand(R) < 0.6, -1, r.randint(0, 3, R))
    before = (kv * r.rand(R)).astype(np.int64)  # the rest of kv is new
    before = np.where(r.rand(R) < 0.3, kv, before)
    kept = np.where(keep < 0, 0, np.minimum(before + np.maximum(keep, 0), kv))
    back = [int(p) for i in range(R) for p in table[i, -(-kept[i] // P):-(-kv[i] // P)]]
    good = [p for p in back if 0 <= p < n_pages]
    head = 3
    c = {"kv_len": _i32(before), "block_table": _i32(table), "ring": _i32(np.full(n_pages, -5)), "page_size": P,
         "ring_pos": torch.tensor([head, head], dtype=torch.int64, device="cuda")}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    done = vs.cache_commit(c, {"new_len": _i32(kv), "ring_pos": c["ring_pos"]}, _i32(keep), status=status)
    assert status.item() == (vs.STATUS_BAD_PAGE if len(good) < len(back) else 0)
    assert done["kv_len"].tolist() == kept.tolist()
    assert done["ring_pos"].tolist() == [head, head + len(good)]
    ring = c["ring"].tolist()
    assert [ring[(head + i) % n_pages] for i in range(len(good))] == good
    assert sum(p == -5 for p in ring) == n_pages - len(good)
    # what the ring holds serves the next requests
    c.update(done)
    c["kv_len"].zero_()
    n = np.full(R, P) * (np.arange(R) < len(good))
    status.zero_()
    out = vs.cache_reserve(c, _i32(np.concatenate([[0], np.cumsum(n)])), int(n.sum()), status=status)
    assert status.item() == 0
    assert out["slot"].tolist() == [p * P + j for p in good[:R] for j in range(P)]


def test_a_strange_id_taken_from_the_ring_does_not_come_back():
    """reserve reports it and gives its rows no slot; after the commit it is gone."""
    c = vs.cache_tables(2, 4, 4, 4)
    c["ring"].copy_(_i32([2, 77, 1, 0]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = vs.cache_reserve(c, _i32([0, 8, 12]), 12, status=status)
    assert status.item() == vs.STATUS_BAD_PAGE and out["slot"].tolist() == [8, 9, 10, 11] + [-1] * 4 + [4, 5, 6, 7]
    status.zero_()
    done = vs.cache_commit(c, out, _i32([-1, -1]), status=status)
    assert status.item() == vs.STATUS_BAD_PAGE and done["ring_pos"].tolist() == [3, 6]
    ring = c["ring"].tolist()
    assert [ring[i % 4] for i in range(3, 6)] == [0, 2, 1]
