"""Logit adjustments on the GPU against the formula in 64 bits, one request after the other."""
import math

import numpy as np
import pytest
import torch

import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def _f32(v):
    return torch.tensor(np.asarray(v, dtype=np.float32), device="cuda")


class Case:
    """Random requests; `want` the formula's values, `named` the entries that a rule names, `size` the sum of the
    magnitudes that are rounded on the way."""

    def __init__(self, R, V, dt, new=4, hist=40, n_bias=5, n_masks=3, seed=0, offs=0, ld=None, pen=True):
        r = np.random.RandomState(seed)
        self.n = r.randint(0 if R > 1 else 1, new + 1, R)
        self.off = np.concatenate([[0], np.cumsum(self.n)]) + offs
        self.rows, self.V = int(self.off[-1]) + 2, V
        base = 4 * torch.randn(self.rows, ld or V, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        self.logits = base.to(dt)[:, :V]
        self.len = r.randint(0, hist + 1, R)
        self.prompt = r.randint(0, hist + 1, R)
        self.tok = r.randint(0, max(1, min(V, 2 * hist)), (R, hist + 3)) * 7 % V
        self.x = r.randint(0, max(1, min(V, 4)), (R, new))
        self.pen = [r.uniform(0.8, 1.5, R).astype(np.float32), r.uniform(-1, 1, R).astype(np.float32),
                    r.uniform(-1, 1, R).astype(np.float32)] if pen else None
        nb = r.randint(0, n_bias + 1, R)
        self.boff = np.concatenate([[0], np.cumsum(nb)])
        self.btok, self.bval = r.randint(0, V, int(nb.sum())), r.randn(int(nb.sum())).astype(np.float32)
        self.mask = r.randint(-(1 << 31), 1 << 31, (max(n_masks, 1), -(-V // 32) + 1)).astype(np.int64).astype(np.int32) if n_masks else None
        self.mrow = r.randint(-1, max(n_masks, 1), self.rows)
        self.R = R

    def call(self, **kw):
        p = dict(zip(("repetition", "frequency", "presence"), map(_f32, self.pen))) if self.pen else {}
        m = dict(mask=torch.from_numpy(self.mask).cuda(), mask_row=_i32(self.mrow)) if self.mask is not None else {}
        return vs.adjust_logits(self.logits, _i32(self.tok), _i32(self.prompt), _i32(self.len), row_off=_i32(self.off), x=_i32(self.x),
                                bias=(_i32(self.boff), _i32(self.btok), _f32(self.bval)), **p, **m, **kw)

    def want(self):
        z = self.logits.double().cpu().numpy()
        size, named = np.abs(z), np.zeros(z.shape, bool)
        for r in range(self.R):
            for j in range(self.n[r]):
                b = self.off[r] + j
                zb, sb, nb = z[b], size[b], named[b]
                if self.pen:
                    rep, fr, pr = (float(t[r]) for t in self.pen)
                    toks = [int(t) for t in self.tok[r, :self.len[r]]]
                    asked, said = toks[:self.prompt[r]], toks[self.prompt[r]:] + [int(t) for t in self.x[r, :j]]
                    for v in set(asked) | set(said):
                        zb[v] = zb[v] / rep if zb[v] > 0 else zb[v] * rep
                        sb[v], nb[v] = abs(zb[v]), True
                    for v in set(said):
                        c = said.count(v)
                        zb[v] -= fr * c + pr
                        sb[v] += abs(fr * c) + abs(pr)
                for v, t in {int(self.btok[i]): float(self.bval[i]) for i in range(self.boff[r], self.boff[r + 1])}.items():
                    zb[v] += t
                    sb[v] += abs(t)
                    nb[v] = True
                if self.mask is not None and self.mrow[b] >= 0:
                    bits = np.unpackbits(self.mask[self.mrow[b]].view(np.uint8), bitorder="little")[:self.V]
                    zb[bits == 0] = -math.inf
        return z, size, named

    def check(self, got):
        z, size, named = self.want()
        own = np.zeros(self.rows, bool)
        own[self.off[0]:self.off[-1]] = True
        got64, src = got.double().cpu().numpy()[own], self.logits.double().cpu().numpy()[own]
        z, size, named = z[own], size[own], named[own]
        hidden = np.isneginf(z)
        assert np.array_equal(np.isneginf(got64), hidden)
        plain = ~named & ~hidden
        assert np.array_equal(got64[plain], src[plain])
        at = named & ~hidden
        # at most five roundings to fp32 of sums no larger than `size` (it holds every term), then the stored type's
        tol = 5 * 2.0 ** -24 * 2 * size[at]
        if got.dtype == torch.bfloat16:
            tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (np.abs(z[at]) + tol)
        err = np.abs(got64[at] - z[at])
        assert np.all(err <= tol), float((err - tol).max())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,kw", [
    (1, 1, dict(hist=3)), (3, 7, dict(hist=5)), (2, 33, {}), (5, 1000, dict(hist=500)), (4, 4099, dict(new=9, hist=300, n_bias=50)),
    (40, 8192, dict(new=3)), (60, 20001, dict(new=12, hist=90)), (1, 50257, dict(new=64, hist=2000)), (7, 12345, dict(ld=12352)),
    (3, 9000, dict(n_masks=0, offs=1)), (3, 9000, dict(pen=False)), (2, 5000, dict(pen=False, n_bias=0, n_masks=1)),
    (1, 6000, dict(new=64, hist=10, seed=5))])
def test_matches_the_formula(R, V, kw, dt):
    c = Case(R, V, dt, **kw)
    c.check(c.call())


@pytest.mark.parametrize("dt,V", [(torch.float32, 5003), (torch.bfloat16, 4096)])
def test_in_place_gives_the_same_and_leaves_other_rows(dt, V):
    c = Case(6, V, dt, offs=1)
    want, src = c.call(), c.logits.clone()
    c.logits = src.clone()
    got = c.call(out=c.logits)
    assert got.data_ptr() == c.logits.data_ptr()
    a, b = int(c.off[0]), int(c.off[-1])
    assert torch.equal(got[a:b], want[a:b]) and torch.equal(got[:a], src[:a]) and torch.equal(got[b:], src[b:])


def test_rows_at_other_offsets_from_16_bytes():
    c = Case(5, 3001, torch.bfloat16)
    want = c.call()
    wide = torch.zeros(c.rows, 3016, dtype=torch.bfloat16, device="cuda")
    got = c.call(out=wide[:, 3:3004])
    a, b = int(c.off[0]), int(c.off[-1])
    assert torch.equal(got[a:b], want[a:b])
    assert torch.all(wide[:, :3] == 0) and torch.all(wide[:, 3004:] == 0)


def test_a_fixed_number_of_rows_a_request_and_many_rows_of_one():
    z = torch.randn(90, 2000, device="cuda")
    tok, length = _i32(np.arange(30).reshape(3, 10)), _i32([10, 4, 0])
    got = vs.adjust_logits(z, tok, None, length, rows_per_request=30, frequency=_f32([0.5, 0.25, 1.0]))
    want = z.clone()
    for r in range(3):
        for t in tok[r, :int(length[r])].tolist():
            want[30 * r:30 * r + 30, t] -= [0.5, 0.25, 1.0][r]
    assert torch.equal(got, want)
    one = vs.adjust_logits(z, tok[:1].contiguous(), None, length[:1].contiguous(), rows_per_request=90, frequency=_f32([0.5]))
    want = z.clone()
    want[:, :10] -= 0.5
    assert torch.equal(one, want)


def test_nothing_allowed_infinities_and_nan():
    V = 100
    z = torch.randn(4, V, device="cuda")
    z[1, 5], z[1, 6], z[1, 7], z[2, 8], z[2, 9] = math.nan, math.inf, -math.inf, math.nan, torch.finfo(torch.float32).min
    mask = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    mask[0] = 0
    mask[1, 0] = ~(7 << 5)
    got = vs.adjust_logits(z, mask=mask, mask_row=_i32([0, 1, 2, -1]))
    assert torch.all(torch.isneginf(got[0]))
    assert torch.all(torch.isneginf(got[1, 5:8])) and torch.equal(got[1, 8:], z[1, 8:]) and torch.equal(got[1, :5], z[1, :5])
    assert torch.isnan(got[2, 8]) and got[2, 9] == z[2, 9] and torch.equal(got[3], z[3])
    # where no row of masks is named, row b has mask b
    assert torch.equal(vs.adjust_logits(z[:2], mask=mask), got[:2])


def test_bad_entries_are_flagged_and_count_for_nothing():
    V, st = 50, torch.zeros(1, dtype=torch.int32, device="cuda")
    z = torch.randn(2, V, device="cuda")
    tok = _i32([[1, -5, V, 2], [3, 4, 5, 6]])
    got = vs.adjust_logits(z, tok, None, _i32([4, 99]), presence=_f32([1, 1]), bias=(_i32([0, 2, 2]), _i32([-1, 7]), _f32([9, 2])),
                           mask=torch.zeros(1, 2, dtype=torch.int32, device="cuda"), mask_row=_i32([-1, 1]), status=st)
    assert st.item() == vs.STATUS_BAD_TOKEN | vs.STATUS_BAD_LEN | vs.STATUS_BAD_ROW
    want = z.clone()
    want[0, [1, 2]] -= 1
    want[0, 7] += 2
    want[1, 3:7] -= 1
    assert torch.equal(got, want)
    st.zero_()
    out = torch.full_like(z, 3.0)
    vs.adjust_logits(z, row_off=_i32([0, 1, 9]), out=out, status=st)
    assert st.item() == vs.STATUS_BAD_LEN and torch.equal(out, z)


def test_empty_histories_and_lists():
    z = torch.randn(2, 64, device="cuda")
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    got = vs.adjust_logits(z, none, None, _i32([0, 0]), x=none, repetition=_f32([2, 2]), bias=(_i32([0, 0, 0]), _i32([]), _f32([])))
    assert torch.equal(got, z)
    assert vs.adjust_logits(z[:0]).shape == (0, 64)


def test_a_biased_token_listed_twice_takes_its_last_entry():
    z = torch.zeros(1, 64, device="cuda")
    got = vs.adjust_logits(z, bias=(_i32([0, 3]), _i32([9, 9, 9]), _f32([1, 2, 4])))
    assert got[0, 9] == 4


def test_stream_and_graph():
    c = Case(9, 5000, torch.float32)
    want = c.call()
    side = torch.cuda.Stream()
    args = dict(repetition=_f32(c.pen[0]), row_off=_i32(c.off), x=_i32(c.x))
    pos = (c.logits, _i32(c.tok), _i32(c.prompt), _i32(c.len))
    want = vs.adjust_logits(*pos, **args)
    torch.cuda.synchronize()
    got = vs.adjust_logits(*pos, **args, stream=side)
    side.synchronize()
    a, b = int(c.off[0]), int(c.off[-1])
    assert torch.equal(got[a:b], want[a:b])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = vs.adjust_logits(*pos, **args)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[a:b], want[a:b])


def test_refusals():
    z = torch.randn(4, 64, device="cuda")
    with pytest.raises(TypeError):
        vs.adjust_logits(z.half())
    with pytest.raises(TypeError):
        vs.adjust_logits(z, mask=torch.zeros(1, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        vs.adjust_logits(z, mask=torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        vs.adjust_logits(z.t())
    with pytest.raises(ValueError):
        vs.adjust_logits(z, out=z[:3])
    with pytest.raises(vs.SpecError):
        vs.adjust_logits(z, presence=_f32([1] * 4))  # a penalty without tokens
    with pytest.raises(vs.SpecError):
        vs.adjust_logits(z, length=_i32([1] * 4), rows_per_request=2)  # eight rows of four


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,kw", [
    (500, 1000, dict(new=5, hist=90)), (120, 9025, dict(new=9, offs=3)), (160, 6015, dict(new=4, n_masks=0)), (460, 7, dict(new=3)),
    (456, 3009, dict(new=2, n_bias=40)), (40, 50257, dict(new=12, hist=300, n_bias=90)), (20, 40000, dict(new=64, hist=2000)),
    (500, 3005, dict(pen=False, n_bias=0, n_masks=0)), (470, 3013, dict(new=3, ld=3019)), (230, 6008, dict(new=7, ld=6032, offs=1))])
def test_many_rows(R, V, kw, dt):
    """The formula, and the same bits as in place, where the results are written over the logits."""
    c = Case(R, V, dt, **kw)
    got = c.call()
    c.check(got)
    a, b = int(c.off[0]), int(c.off[-1])
    src, c.logits = c.logits, c.logits.clone()
    assert torch.equal(c.call(out=c.logits)[a:b], got[a:b])
    # strided results on the same offsets from 16 bytes
    c.logits = src
    wide = torch.full((c.rows, src.stride(0) + 16), 3.0, dtype=dt, device="cuda")
    assert torch.equal(c.call(out=wide[:, :V])[a:b], got[a:b])
    assert torch.all(wide[:, V:] == 3) and torch.all(wide[:a] == 3) and torch.all(wide[b:] == 3)
