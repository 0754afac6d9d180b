"""Attention over a cache in 4 bits against softmax sums in 64 bits of what the cache stands for, request by request."""
import math

import numpy as np
import pytest
import torch

import packed_ref
import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


class Case:
    """Requests with ``n`` rows and ``kv`` own keys each, in ``groups`` [(requests, prefix keys)]; every place of the
    cache that no key names holds the largest values there are."""

    def __init__(self, n, kv, Hq, Hk, D, P, dt, groups=(), seed=0, row0=0, spread=1.0, ramp=None):
        r = np.random.RandomState(seed)
        self.n, self.kv, self.groups, self.P, self.D, self.Hk = list(n), list(kv), list(groups), P, D, Hk
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
        self.caches, self.values = [], []
        for c in range(2):
            x = torch.randn(total, P, Hk, D, generator=g, device="cuda").double()
            if ramp and c == 0:
                for tab, m in list(zip(self.tab, self.kv)) + list(zip(self.ptab, [p for _, p in self.groups])):
                    s = self._slots(tab, m)
                    x.view(-1, Hk, D)[s] *= torch.linspace(*ramp, m, device="cuda", dtype=torch.float64)[:, None, None]
            code, num = packed_ref.encode(x)
            named = torch.zeros(total * P, dtype=torch.bool, device="cuda")
            for tab, m in list(zip(self.tab, self.kv)) + list(zip(self.ptab, [p for _, p in self.groups])):
                named[self._slots(tab, m)] = True
            named = named.view(total, P)
            code[~named], num[~named] = 255, 7
            self.caches.append(packed_ref.pack(code, num))
            self.values.append(packed_ref.decode(self.caches[-1]).flatten(0, 1))
        self.scale = 1 / math.sqrt(D)
        self.goff = np.concatenate([[0], np.cumsum([c for c, _ in self.groups])]) if self.groups else None

    def _slots(self, table, m):
        at = np.arange(m)
        return torch.tensor(np.asarray(table, dtype=np.int64)[at // self.P] * self.P + at % self.P if m else at, device="cuda")

    def args(self):
        g = dict(group_off=_i32(self.goff), prefix_len=_i32([p for _, p in self.groups]), prefix_table=self.prefix_table) if self.groups else {}
        return (self.q, *self.caches, _i32(self.off), _i32(self.kv), self.block_table), dict(scale=self.scale, **g)

    def call(self, **kw):
        a, k = self.args()
        return vs.prefix_attention_packed(*a, **k, **kw)

    def want(self, r):
        """out, lse, sum of |weighted values| and of |score terms| of request r's rows in 64 bits."""
        s = self._slots(self.tab[r], self.kv[r])
        shared = 0
        for g, (_, p) in enumerate(self.groups):
            if self.goff[g] <= r < self.goff[g + 1]:
                s, shared = torch.cat([self._slots(self.ptab[g], p), s]), p
        k, v = (c[s] for c in self.values)
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
    ([1], [1], 1, 1, 32, 1, ()),
    ([1], [700], 4, 4, 64, 16, ()),
    ([2, 0, 3], [5, 7, 3], 6, 2, 96, 5, ()),
    ([1, 4, 2], [40, 4, 9], 8, 2, 160, 16, ((2, 50), (1, 7))),
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
    ([3], [3], 4, 2, 128, 16, ()),
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
    ([1] * 50, [100 + (i * 131) % 2000 for i in range(50)], 28, 4, 128, 32, ()),
    ([1] * 3, [3000, 20000, 1], 128, 1, 128, 64, ()),
    ([1, 2, 700, 1, 33], [900, 5, 900, 60, 33], 16, 2, 128, 16, ()),
    ([40, 1, 1], [4000, 3, 70], 1, 1, 64, 16, ((3, 200),)),
    ([3, 1, 60], [1500, 700, 2000], 16, 4, 128, 384, ((2, 800),)),
    ([1, 2, 30], [1500, 9000, 200], 12, 2, 64, 8, ((1, 3000), (2, 100))),
    ([1] * 6, [5000, 4097, 129, 1, 70, 12000], 14, 1, 128, 8, ()),
    ([1, 40], [5000, 9000], 6, 1, 64, 640, ()),
    ([1] * 30 + [200], [40 + 31 * i for i in range(31)], 2, 1, 128, 16, ()),
    ([1] * 60 + [150], [1 + 17 * i for i in range(61)], 1, 1, 128, 32, ()),
    ([1] * 20 + [90], [200] * 20 + [95], 6, 3, 64, 64, ()),
]


@pytest.mark.parametrize("n,kv,Hq,Hk,D,P,groups", TENSOR)
def test_tensor_core_sizes(n, kv, Hq, Hk, D, P, groups):
    _run(Case(n, kv, Hq, Hk, D, P, BF, groups))


@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 96), (BF, 128)])
@pytest.mark.parametrize("ramp", [(0.1, 8.0), (8.0, 0.1)])
def test_rising_and_falling_scores_rescale_and_stay_finite(dt, D, ramp):
    _run(Case([3, 2, 40], [900, 40, 700], 8, 2, D, 16, dt, ((2, 600), (1, 300)), spread=3.0, ramp=ramp))


def test_far_scales():
    """Keys near the smallest and values near the largest scale."""
    c = Case([2, 9], [300, 700], 8, 2, 128, 16, BF)
    c.caches[0][1].fill_(3)
    c.caches[1][1].fill_(250)
    c.values = [packed_ref.decode(x).flatten(0, 1) for x in c.caches]
    _run(c)


@pytest.mark.parametrize("n", [[2, 1], [30, 1]])
@pytest.mark.parametrize("power", [-90, -30, 30, 90])
def test_far_queries(n, power):
    """Queries of any size, with the scale that makes their scores ordinary; rows of zeros among them."""
    c = Case(n, [300, 700], 8, 2, 128, 16, BF, ((1, 100),))
    c.q = c.q * 2.0 ** power
    c.q[1] = 0
    c.scale = c.scale * 2.0 ** -power if power > -90 else 1e26  # (2^90 / 11 is 1.1e26)
    _run(c)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("n", [[3, 2], [30, 2]])
def test_a_row_of_nan_stays_alone(n, bad):
    c = Case(n, [300, 70], 8, 2, 128, 16, BF, ((2, 140),))
    want, lse = _run(c)
    c.q[1, 3, 5] = bad
    got = c.call()
    live = torch.ones(c.off[-1], 8, dtype=torch.bool, device="cuda")
    live[1, 3] = False
    assert torch.equal(got[:c.off[-1]][live], want[:c.off[-1]][live]) and bool(torch.isnan(got[1, 3]).any())


@pytest.mark.parametrize("each,Hq,Hk", [(4, 64, 8), (1, 256, 2), (9, 64, 16), (4, 16, 4)])
def test_calls_of_many_rows_run_in_windows(each, Hq, Hk):
    """More than 2^20 query rows: by the narrow kernel alone (16 rows a segment), or by both."""
    R = (1 << 20) // Hq // each + 700
    kv = [each + (i * 37) % 90 for i in range(R)]
    c = Case([each] * R, kv, Hq, Hk, 64, 16, BF, ((R // 2, 130),) if each == 9 else ())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = c.call(want_lse=True, status=st)
    assert st.item() == 0
    pick = sorted({0, 1, R // 3, R // 2 - 1, R // 2, R - 2, R - 1} | {(i * 7919) % R for i in range(60)} | {(1 << 19) // Hq // each + i for i in range(-3, 4)})
    c.check(got, lse, pick)
    assert bool(torch.isfinite(got[:c.off[-1]].float()).all())


def test_rows_ahead_of_the_first_request():
    _run(Case([3, 2], [300, 40], 8, 2, 128, 16, BF, ((2, 150),), row0=5))


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


@pytest.mark.parametrize("n", [[2, 2, 2], [40, 2, 30]])
@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 128)])
def test_bad_lengths_and_pages_are_flagged(dt, D, n):
    c = Case(n, [40, 50, 60], 4, 2, D, 16, dt, ((3, 33),))
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
    c.block_table[1, 1] = c.caches[0][0].shape[0]
    c.block_table[2, 0] = -1
    c.call(status=st, out=out, lse=lse)
    assert st.item() == vs.STATUS_BAD_PAGE
    c.check(out, lse, [0])
    st.zero_()
    c.block_table = table
    c.off = np.array([0, n[0], n[0] + n[1], c.rows + 1])  # the last request's rows leave the batch
    c.groups = []
    c.call(status=st, out=out)
    assert st.item() == vs.STATUS_BAD_LEN


@pytest.mark.parametrize("n", [[3, 1, 8], [3, 1, 90]])
def test_same_bits_again_on_another_stream_and_in_graphs(n):
    c = Case(n, [500, 20, 1000], 16, 2, 128, 32, BF, ((3, 600),))
    want, lse = _run(c)
    a, kw = c.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vs.prefix_attention_packed(*a, **kw, stream=side)
    side.synchronize()
    live = slice(0, c.off[-1])
    assert torch.equal(got[live], want[live])
    # two graphs that share a workspace, replayed one after the other
    ws = torch.empty(vs.attention_packed_workspace_bytes(c.rows, 3, 16, 128), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vs.prefix_attention_packed(*a, **kw, workspace=ws))
        graphs.append(g)
    for o in outs:
        o.zero_()
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[live], want[live]) for o in outs)


def test_refusals():
    c = Case([1], [5], 4, 2, 64, 16, BF)
    (k, ks), (v, vsc) = c.caches
    args = lambda: list(c.args()[0])  # noqa: E731
    for i, bad, err in ((0, c.q.float()[..., :32], ValueError), (0, c.q.half(), TypeError), (1, (k[:, :1], ks[:, :1]), ValueError),
                        (1, (k[:, :, :1], ks), ValueError), (2, (v[:1], vsc[:1]), ValueError), (2, (v.int(), vsc), TypeError),
                        (3, _i32([0]), ValueError), (4, _i32([5]).long(), TypeError), (5, c.block_table.float(), TypeError),
                        (0, c.q.transpose(1, 2), ValueError), (1, (k.transpose(1, 2), ks), ValueError), (1, (k, ks.cpu()), TypeError)):
        a = args()
        a[i] = bad
        with pytest.raises(err):
            vs.prefix_attention_packed(*a)
    with pytest.raises(ValueError):
        vs.prefix_attention_packed(*args(), prefix_len=_i32([3]))
    with pytest.raises(vs.SpecError):
        vs.prefix_attention_packed(*args(), scale=-1.0)
    with pytest.raises(vs.SpecError):
        vs.prefix_attention_packed(*args(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    a = args()
    a[0], a[3] = c.q[:0], _i32([0, 0])
    assert vs.prefix_attention_packed(*a).shape == (0, 4, 64)


@pytest.mark.parametrize("dt,n", [(BF, 1), (BF, 9), (F32, 2)])
def test_pages_past_two_gigabytes(dt, n):
    """Keys at the end of caches of 2.3 GB give the bits that they give in small ones."""
    Hq, Hk, D, P, R, kv = 16, 8, 128, 64, 3, 150
    many, few = 70001, 3 * R
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(R * kv, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
    pos = torch.arange(R * kv, dtype=torch.int32, device="cuda")
    freq, _ = vs.rope_frequencies(D)
    q = x[:R * n, :Hq].contiguous()
    place = np.arange(kv)
    outs = []
    for pages in (many, few):
        kc, vc = vs.packed_cache(pages, P, Hk, D), vs.packed_cache(pages, P, Hk, D)
        table = pages - few + np.arange(few).reshape(R, 3)
        slot = _i32(np.concatenate([table[r][place // P] * P + place % P for r in range(R)]))
        turned = vs.norm_rope_cache(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], freq, pos, slot, kc, vc)
        k, v = vs.cache_read_packed(kc, vc, slot)
        o = vs.prefix_attention_packed(q, kc, vc, _i32(np.arange(R + 1) * n), _i32([kv] * R), _i32(table))
        outs.append((turned, k, v, o))
        del kc, vc
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and float(outs[0][3].float().abs().max()) > 0


@pytest.mark.parametrize("dt,Hq,Hk,D,P", [(BF, 16, 2, 128, 16), (F32, 6, 2, 96, 24)])
def test_write_then_attend(dt, Hq, Hk, D, P):
    """Rounds as they are run: slots reserved, rows normed, turned and stored in 4 bits, attended, some of them kept; against
    64 bits from what the cache then stands for."""
    R, rounds = 5, 4
    g = torch.Generator("cuda").manual_seed(3)
    freq, _ = vs.rope_frequencies(D)
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    cache = vs.cache_tables(R, 60, P, 12)
    kc, vc = vs.packed_cache(60, P, Hk, D), vs.packed_cache(60, P, Hk, D)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(rounds):
        n = [(7 * r + 3 * t) % 6 + (30 if t == 0 else 0) for r in range(R)]
        off = np.concatenate([[0], np.cumsum(n)])
        rows = int(off[-1])
        qkv = torch.randn(rows, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
        res = vs.cache_reserve(cache, _i32(off), rows, status=st)
        q = vs.norm_rope_cache(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], freq, res["position"], res["slot"], kc, vc,
                               q_weight=qw, k_weight=kw, status=st)
        got, lse = vs.prefix_attention_packed(q, kc, vc, _i32(off), res["new_len"], cache["block_table"], want_lse=True, status=st)
        c = Case.__new__(Case)
        c.n, c.kv, c.groups, c.P, c.D, c.Hk, c.off, c.q, c.scale = n, res["new_len"].tolist(), [], P, D, Hk, off, q, D ** -0.5
        c.tab = cache["block_table"].tolist()
        c.values = [packed_ref.decode(x).flatten(0, 1) for x in (kc, vc)]
        c.check(got, lse)
        keep = _i32([max(0, x - (r % 3)) for r, x in enumerate(n)])
        cache.update(vs.cache_commit(cache, res, keep, status=st))
    assert st.item() == 0
