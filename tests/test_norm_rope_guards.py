"""Rows that are left out, slots outside the cache, far positions, and calls in place or without queries or keys, in every
kernel of the head norms and for both kinds of cache.  The caches are the middle of larger buffers, so that what a slot outside
them would reach is there to be looked at."""
import pytest
import torch

import packed_ref
import verify_sampling_gb300 as vs
from test_norm_rope import _check, _freq, _near, _normed, _turned

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
P, GUARD = 16, 3  # tokens of a page, pages before and behind the cache

# rows, Hq, Hk, D, rot, type: the ring with one token a stage, with two and four and a remainder, with more stages than it
# holds; a warp a part of a short row; pairs off the vectors; heads longer than a warp's vectors
SHAPES = [(9, 32, 8, 128, 128, BF), (700, 32, 8, 128, 64, BF), (1001, 24, 4, 64, 64, BF), (2003, 24, 4, 64, 32, BF), (9001, 24, 4, 64, 64, BF),
          (1001, 12, 2, 64, 64, F32), (5003, 12, 2, 64, 32, F32), (60, 2, 1, 64, 64, F32), (300, 5, 3, 96, 64, BF), (60, 6, 2, 96, 22, BF),
          (40, 3, 2, 512, 512, BF), (40, 3, 2, 256, 256, F32)]


class Guarded:
    """A cache of either kind between pages that nothing may write."""

    def __init__(self, packed, pages, Hk, D, dt):
        n = pages + 2 * GUARD
        self.packed, self.pages = packed, pages
        if packed:
            data, scale = vs.packed_cache(n, P, Hk, D)
            self.whole = (data.fill_(0x5A), scale.fill_(0xA5))
            self.cache = tuple(t[GUARD:-GUARD] for t in self.whole)
        else:
            self.whole = (torch.full((n, P, Hk, D), 7.0, dtype=dt, device="cuda"),)
            self.cache = self.whole[0][GUARD:-GUARD]
        self.before = [t.clone() for t in self.whole]

    def values(self):
        """What the slots hold [slots, Hk, D]."""
        return (packed_ref.decode(self.cache) if self.packed else self.cache).flatten(0, 1)

    def changed_slots(self):
        """Slots whose bytes changed, counted from the first guard page."""
        out = torch.zeros((self.pages + 2 * GUARD) * P, dtype=torch.bool, device="cuda")
        for t, b in zip(self.whole, self.before):
            d = t != b
            if self.packed:  # [pages, Hk, groups, P, 16] and [pages, Hk, P, groups]
                d = d.permute(0, 3, 1, 2, 4) if d.dim() == 5 else d.permute(0, 2, 1, 3)
            out |= d.flatten(0, 1).flatten(1).any(1)
        return out


def _inputs(rows, Hq, Hk, D, dt, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    qkv = torch.randn(rows, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
    position = torch.randint(0, 100000, (rows,), generator=g, device="cuda", dtype=torch.int32)
    pages = -(-rows // P) + 1
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:rows].to(torch.int32)
    w = [1 + 0.5 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    return qkv, position, slot, pages, w


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot,dt", SHAPES)
def test_what_is_left_out_stays_as_it_was(rows, Hq, Hk, D, rot, dt, packed, interleaved):
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, Hq, Hk, D, dt)
    row = torch.arange(rows, device="cuda")
    # every kind of row at every place of a stage of 2, 4 or 8, and two whole stages of 8 left out
    position[(row % 11 == 3) | (row // 8 == 5) | (row == rows - 1)] = -1
    position[row % 37 == 1] = -(1 << 31)
    far = row % 13 == 6
    position[far] = (1 << 24) + row[far].to(torch.int32)
    for i, bad in enumerate((-1, -2 * P, pages * P, pages * P + 2 * P + 1)):
        slot[(row % 17 == 2 + 3 * i) | (row // 8 == 7)] = bad
    live = position >= 0
    written = live & (slot >= 0) & (slot < pages * P)
    kc, vc = (Guarded(packed, pages, Hk, D, dt) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((rows + 2, Hq, D), 5.0, dtype=dt, device="cuda")
    freq = _freq(rot)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    vs.norm_rope_cache(q, k, v, freq, position, slot, kc.cache, vc.cache, q_weight=qw, k_weight=kw, interleaved=interleaved, scale=1.25,
                       q_out=q_out[1:-1], status=status)
    assert status.item() == (vs.STATUS_BAD_PAGE if bool((slot >= pages * P).any()) else 0) | (vs.STATUS_BAD_POSITION if bool(far.any()) else 0)
    at = position.clamp(max=(1 << 24) - 1)[live]
    want, size = _turned(_normed(q[live], qw, 1e-6), at, freq, 1.25, interleaved)
    _check(q_out[1:-1][live], want, size, _near(D))
    assert torch.all(q_out[1:-1][~live] == 5) and torch.all(q_out[0] == 5) and torch.all(q_out[-1] == 5)
    to = slot[written].long()
    for c in (kc, vc):
        allowed = torch.zeros((pages + 2 * GUARD) * P, dtype=torch.bool, device="cuda")
        allowed[to + GUARD * P] = True
        assert torch.equal(c.changed_slots(), allowed)
    at = position.clamp(max=(1 << 24) - 1)[written]
    want, size = (t.cuda() for t in _turned(_normed(k[written], kw, 1e-6), at, freq, 1.25, interleaved))
    have = kc.values()[to]
    if not packed:
        _check(have, want.cpu(), size.cpu(), _near(D))
        assert torch.equal(vc.values()[to], v[written])
        return
    step = packed_ref.scales(kc.cache[1].transpose(1, 2).flatten(0, 1)[to]).repeat_interleave(32, -1)
    assert torch.all((want - have).abs() <= step / 2 + _near(D) * size + 2.0 ** -22 * want.abs())
    step = packed_ref.scales(vc.cache[1].transpose(1, 2).flatten(0, 1)[to]).repeat_interleave(32, -1)
    x = v[written].double()
    assert torch.all((x - vc.values()[to]).abs() <= step / 2 + 2.0 ** -22 * x.abs())


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot,dt", [s for s in SHAPES if s[0] < 5000] + [(700, 4, 16, 128, 128, BF)])
def test_in_place_and_without_queries_or_keys(rows, Hq, Hk, D, rot, dt, packed):
    """The bits of the whole call."""
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, Hq, Hk, D, dt, seed=1)
    position[::5] = -1
    freq = _freq(rot)
    k, v = (qkv[:, a:a + Hk].contiguous() for a in (Hq, Hq + Hk))
    q = qkv[:, :Hq].contiguous()
    whole = [Guarded(packed, pages, Hk, D, dt) for _ in range(2)]
    out = q.clone()  # rows that are left out, too
    vs.norm_rope_cache(q, k, v, freq, position, slot, *(c.cache for c in whole), q_weight=qw, k_weight=kw, q_out=out)
    # in place, with the keys
    caches = [Guarded(packed, pages, Hk, D, dt) for _ in range(2)]
    here = q.clone()
    assert vs.norm_rope_cache(here, k, v, freq, position, slot, *(c.cache for c in caches), q_weight=qw, k_weight=kw, q_out=here) is here
    assert torch.equal(here, out) and all(torch.equal(a, b) for c, d in zip(caches, whole) for a, b in zip(c.whole, d.whole))
    # in place where queries, keys and values lie in one projection
    caches = [Guarded(packed, pages, Hk, D, dt) for _ in range(2)]
    one = qkv.clone()
    view = one[:, :Hq]
    vs.norm_rope_cache(view, one[:, Hq:Hq + Hk], one[:, Hq + Hk:], freq, position, slot, *(c.cache for c in caches), q_weight=qw, k_weight=kw, q_out=view)
    assert torch.equal(view, out) and torch.equal(one[:, Hq:], qkv[:, Hq:])
    assert all(torch.equal(a, b) for c, d in zip(caches, whole) for a, b in zip(c.whole, d.whole))
    # queries alone
    here = q.clone()
    vs.norm_rope_cache(here, None, None, freq, position, None, None, None, q_weight=qw, q_out=here)
    assert torch.equal(here, out)
    # keys and values alone
    caches = [Guarded(packed, pages, Hk, D, dt) for _ in range(2)]
    assert vs.norm_rope_cache(q[:, :0], k, v, freq, position, slot, *(c.cache for c in caches), k_weight=kw).shape == (rows, 0, D)
    assert all(torch.equal(a, b) for c, d in zip(caches, whole) for a, b in zip(c.whole, d.whole))
