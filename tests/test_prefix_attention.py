"""Shared-prefix attention on the GPU against softmax sums in 64 bits, request by request."""
import math

import numpy as np
import pytest
import torch

import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


class Case:
    """Requests with ``n`` rows and ``kv`` own keys each, in ``groups`` [(requests, prefix keys)]; every place of the
    cache that no key names is NaN."""

    def __init__(self, n, kv, Hq, Hk, D, P, dt, groups=(), seed=0, row0=0, spread=1.0):
        r = np.random.RandomState(seed)
        self.n, self.kv, self.groups, self.P, self.D, self.Hk = list(n), list(kv), list(groups), P, D, Hk
        R = len(self.n)
        self.off = (np.concatenate([[0], np.cumsum(self.n)]) + row0).astype(int)
        self.rows = int(self.off[-1]) + 1  # a row of no request at the end
        pages = [-(-k // P) for k in self.kv]
        ppages = [-(-p // P) for _, p in self.groups]
        total = sum(pages) + sum(ppages) + 2
        perm = list(r.permutation(total))
        take = lambda c: [perm.pop() for _ in range(c)]  # noqa: E731
        self.tab, self.ptab = [take(c) for c in pages], [take(c) for c in ppages]
        full = lambda t, w: _i32([x + [0] * (w - len(x)) for x in t])  # noqa: E731
        self.block_table = full(self.tab, max(pages + [1]) + 1)
        self.prefix_table = full(self.ptab, max(ppages + [1])) if self.groups else None
        g = torch.Generator("cuda").manual_seed(seed)
        self.q = (spread * torch.randn(self.rows, Hq, D, generator=g, device="cuda")).to(dt)
        self.k = torch.full((total, P, Hk, D), math.nan, dtype=dt, device="cuda")
        self.v = self.k.clone()
        for tab, m in list(zip(self.tab, self.kv)) + list(zip(self.ptab, [p for _, p in self.groups])):
            s = self._slots(tab, m)
            for c in (self.k, self.v):
                c.view(-1, Hk, D)[s] = torch.randn(m, Hk, D, generator=g, device="cuda").to(dt)
        self.scale = 1 / math.sqrt(D)
        self.goff = np.concatenate([[0], np.cumsum([c for c, _ in self.groups])]) if self.groups else None
        assert R >= sum(c for c, _ in self.groups)

    def _slots(self, table, m):
        at = np.arange(m)
        return torch.tensor(np.asarray(table, dtype=np.int64)[at // self.P] * self.P + at % self.P if m else at, device="cuda")

    def call(self, **kw):
        g = dict(group_off=_i32(self.goff), prefix_len=_i32([p for _, p in self.groups]), prefix_table=self.prefix_table) if self.groups else {}
        return vs.prefix_attention(self.q, self.k, self.v, _i32(self.off), _i32(self.kv), self.block_table, scale=self.scale, **g, **kw)

    def want(self, r):
        """out, lse, sum of |weighted values| and of |score terms| of request r's rows in 64 bits."""
        s = self._slots(self.tab[r], self.kv[r])
        shared = 0
        for g, (_, p) in enumerate(self.groups):
            if self.goff[g] <= r < self.goff[g + 1]:
                s, shared = torch.cat([self._slots(self.ptab[g], p), s]), p
        k, v = (c.view(-1, self.Hk, self.D)[s].double() for c in (self.k, self.v))
        q = self.q[self.off[r]:self.off[r + 1]].double()
        q = q.view(q.shape[0], self.Hk, -1, self.D)
        z = torch.einsum("nhgd,lhd->nhgl", q, k) * self.scale
        size = (torch.einsum("nhgd,lhd->nhgl", q.abs(), k.abs()) * self.scale).amax(-1) if len(s) else z.new_zeros(z.shape[:3])
        last = shared + self.kv[r] - self.n[r] + torch.arange(self.n[r], device="cuda")
        hide = torch.arange(len(s), device="cuda")[None, :] > last[:, None]
        hide[:, :shared] = False
        z = z.masked_fill(hide[:, None, None, :], -math.inf)
        lse = torch.logsumexp(z, -1)
        w = torch.where(lse[..., None] == -math.inf, 0.0, torch.exp(z - lse[..., None]))
        o, a = torch.einsum("nhgl,lhd->nhgd", w, v), torch.einsum("nhgl,lhd->nhgd", w, v.abs())
        return [t.flatten(1, 2) for t in (o, lse, a, size)]

    def check(self, got, lse, requests=None):
        for r in range(len(self.n)) if requests is None else requests:
            if self.n[r] == 0:
                continue
            o, l, a, size = self.want(r)
            at = slice(self.off[r], self.off[r + 1])
            keys = self.kv[r] + max([0] + [p for _, p in self.groups])
            # a score is off by D + 3 roundings of its terms (the tensor cores may cut where others round: twice), a power of
            # two by 2^-21, sums by a rounding a term; bf16 adds the weights' and the result's rounding
            dz = 2 * (self.D + 3) * 2.0 ** -24 * size
            rel = 2 * dz + 2.0 ** -20 + (keys / 4 + 200) * 2.0 ** -24
            tol = a * rel[..., None]
            if self.q.dtype == BF:
                half = torch.finfo(BF).eps / 2
                tol = tol + 1.01 * half * (a + o.abs())
            err = (got[at].double() - o).abs()
            assert torch.all(err <= tol + 1e-30), (r, float((err - tol).max()))
            none = l == -math.inf
            assert torch.equal(lse[at] == -math.inf, none) and torch.all(got[at][none] == 0)
            le = (lse[at].double() - l).abs()[~none]
            assert torch.all(le <= (rel + l.abs() * 2.0 ** -22 + 2.0 ** -20)[~none]), (r, float(le.max()))


def _run(c, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(c.q, 3.0)
    got, lse = c.call(want_lse=True, status=st, out=out, **kw)
    assert st.item() == 0
    c.check(got, lse)
    assert torch.all(got[c.off[-1]:] == 3) and torch.all(got[:c.off[0]] == 3)
    return got, lse


GENERIC = [
    # n, kv, Hq, Hk, D, P, groups
    ([1], [1], 1, 1, 1, 1, ()),
    ([1], [700], 4, 4, 64, 16, ()),
    ([2, 0, 3], [5, 7, 3], 6, 2, 33, 5, ()),
    ([1, 4, 2], [40, 4, 9], 8, 2, 80, 16, ((2, 50), (1, 7))),
    ([3, 1], [100, 30], 5, 1, 256, 24, ((2, 333),)),
    ([7, 5, 9, 1, 2], [90, 5, 200, 33, 64], 3, 3, 96, 8, ((1, 0), (3, 65))),
]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("n,kv,Hq,Hk,D,P,groups", GENERIC)
def test_generic_sizes(n, kv, Hq, Hk, D, P, groups, dt):
    _run(Case(n, kv, Hq, Hk, D, P, dt, groups))


TENSOR = [
    ([1], [1], 1, 1, 64, 16, ()),
    ([1], [128], 8, 1, 128, 128, ()),
    ([1], [129], 8, 1, 128, 16, ()),
    ([1], [5000], 32, 8, 128, 16, ()),
    ([3], [3], 4, 2, 128, 8, ()),
    ([2, 0, 5, 1], [700, 30, 300, 1], 16, 4, 128, 32, ()),
    ([1, 4, 2, 3], [40, 4, 9, 300], 16, 2, 128, 64, ((2, 500), (2, 130))),
    ([12] * 9, [100 + 37 * i for i in range(9)], 24, 3, 128, 64, ((9, 1000),)),
    ([5] * 30, [5 + 11 * i for i in range(30)], 40, 8, 64, 16, ((10, 257), (0, 40), (15, 4000))),
    ([300, 1, 70], [300, 900, 500], 12, 4, 128, 256, ()),
    ([130, 64], [1000, 64], 5, 1, 64, 128, ((2, 384),)),
    ([1, 1, 0, 0, 1], [0, 10, 0, 5, 3], 8, 8, 128, 16, ((3, 0), (2, 100))),
    ([4, 4], [2, 6], 8, 2, 128, 16, ()),
    ([2] * 70, [2 + (i * 53) % 400 for i in range(70)], 64, 8, 128, 64, ((35, 700), (35, 128))),
    ([1] * 400, [1 + (i * 29) % 300 for i in range(400)], 2, 1, 64, 32, ((400, 90),)),
]


@pytest.mark.parametrize("n,kv,Hq,Hk,D,P,groups", TENSOR)
def test_tensor_core_sizes(n, kv, Hq, Hk, D, P, groups):
    _run(Case(n, kv, Hq, Hk, D, P, BF, groups))


@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 40), (BF, 128)])
def test_rising_scores_rescale_and_large_ones_stay_finite(dt, D):
    c = Case([3, 2], [900, 40], 8, 2, D, 16, dt, ((2, 600),), spread=3.0)
    for tab, m in list(zip(c.tab, c.kv)) + list(zip(c.ptab, [600])):  # later keys score higher and higher
        s = c._slots(tab, m)
        ramp = torch.linspace(0.1, 8.0, m, device="cuda").to(dt)[:, None, None]
        c.k.view(-1, c.Hk, c.D)[s] = c.k.view(-1, c.Hk, c.D)[s] * ramp
    _run(c)


def test_strided_queries_and_output_give_the_same():
    c = Case([2, 3], [50, 300], 8, 2, 128, 16, BF, ((2, 140),))
    want, lse = _run(c)
    wide = torch.zeros(c.rows, 14, 136, dtype=BF, device="cuda")
    q = c.q
    c.q = wide[:, 3:11, :128]
    c.q.copy_(q)
    assert torch.equal(c.call()[:c.off[-1]], want[:c.off[-1]])
    out = torch.zeros(c.rows, 9, 130, dtype=BF, device="cuda")
    c.call(out=out[:, 1:, 2:])
    assert torch.equal(out[:c.off[-1], 1:, 2:], want[:c.off[-1]]) and torch.all(out[:, 0] == 0) and torch.all(out[..., :2] == 0)
    # off 16 bytes: the generic kernel
    odd = torch.zeros(c.rows, 8, 129, dtype=BF, device="cuda")
    c.q = odd[..., 1:]
    c.q.copy_(q)
    got, l2 = c.call(want_lse=True)
    c.check(got, l2)


@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 128)])
def test_bad_lengths_and_pages_are_flagged(dt, D):
    c = Case([2, 2, 2], [40, 50, 60], 4, 2, D, 16, dt, ((3, 33),))
    c.k.nan_to_num_(0.0)
    c.v.nan_to_num_(0.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, table = c.kv, c.block_table.clone()
    c.kv = [40, -5, 10 ** 6]
    out, lse = torch.zeros_like(c.q), torch.zeros(c.rows, 4, device="cuda")
    c.call(status=st, out=out, lse=lse)
    assert st.item() == vs.STATUS_BAD_LEN
    c.kv = kv
    c.check(out, lse, [0])
    c.call(out=out, lse=lse)
    c.check(out, lse)
    st.zero_()
    c.block_table = table.clone()
    c.block_table[1, 1] = c.k.shape[0]
    c.block_table[2, 0] = -1
    c.call(status=st, out=out, lse=lse)
    assert st.item() == vs.STATUS_BAD_PAGE
    c.check(out, lse, [0])
    st.zero_()
    c.block_table = table
    c.off = np.array([0, 2, 4, c.rows + 1])  # the last request's rows leave the batch
    c.n = [2, 2, 2]
    c.groups = []
    c.call(status=st, out=out)
    assert st.item() == vs.STATUS_BAD_LEN


def test_same_bits_again_on_another_stream_and_in_a_graph():
    c = Case([3, 1, 8], [500, 20, 1000], 16, 2, 128, 32, BF, ((3, 600),))
    want, lse = _run(c)
    args = (c.q, c.k, c.v, _i32(c.off), _i32(c.kv), c.block_table)
    kw = dict(scale=c.scale, group_off=_i32(c.goff), prefix_len=_i32([600]), prefix_table=c.prefix_table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vs.prefix_attention(*args, **kw, stream=side)
    side.synchronize()
    live = slice(0, c.off[-1])
    assert torch.equal(got[live], want[live])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = vs.prefix_attention(*args, **kw)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[live], want[live])


def test_refusals():
    c = Case([1], [5], 4, 2, 64, 16, BF)
    args = lambda: [c.q, c.k, c.v, _i32(c.off), _i32(c.kv), c.block_table]  # noqa: E731
    for i, bad, err in ((0, c.q.float(), TypeError), (0, c.q.half(), TypeError), (1, c.k[..., :32], ValueError), (2, c.v[:1], ValueError),
                        (3, _i32([0]), ValueError), (4, _i32([5]).long(), TypeError), (5, c.block_table.float(), TypeError),
                        (0, c.q.transpose(1, 2), ValueError), (1, c.k.transpose(1, 2), ValueError)):
        a = args()
        a[i] = bad
        with pytest.raises(err):
            vs.prefix_attention(*a)
    with pytest.raises(ValueError):
        vs.prefix_attention(*args(), prefix_len=_i32([3]))
    with pytest.raises(vs.SpecError):
        vs.prefix_attention(*args(), scale=-1.0)
    with pytest.raises(vs.SpecError):
        vs.prefix_attention(*args(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert vs.prefix_attention(c.q[:0], c.k, c.v, _i32([0, 0]), _i32([5]), c.block_table).shape == (0, 4, 64)
