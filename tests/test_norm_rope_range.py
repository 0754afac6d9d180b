"""Head norms of heads whose squares leave fp32, against 64 bits: elements from the smallest numbers to the largest, in every
kernel (heads side by side in long rows; short rows; odd heads; heads longer than a warp's vectors)."""
import math

import pytest
import torch

import packed_ref
import verify_sampling_gb300 as vs
from test_norm_rope import _check, _freq, _near, _normed, _turned

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ROWS, P = 40, 8
SHAPES = [(32, 8, 128, 128), (32, 8, 128, 64), (3, 1, 64, 32), (5, 3, 96, 96), (3, 2, 50, 22), (3, 2, 512, 512), (3, 2, 192, 64)]
POWERS = [-140, -126, -110, -75, -64, -60, -45, -30, 0, 0, 0, 20, 45, 50, 63, 64, 66, 100, 124]


def _heads(Hq, Hk, D, dt, seed=0):
    """Heads of very different sizes beside one another, and keys and values of them."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(ROWS, Hq + 2 * Hk, D, generator=g, device="cuda", dtype=torch.float64).clamp(-7, 7)
    power = torch.tensor(POWERS, dtype=torch.float64, device="cuda")[torch.randint(0, len(POWERS), (ROWS, Hq + 2 * Hk, 1), generator=g, device="cuda")]
    x = (x * torch.exp2(power)).to(dt)
    position = torch.randint(0, 1000, (ROWS,), generator=g, device="cuda", dtype=torch.int32)
    slot = torch.randperm(ROWS + P, generator=g, device="cuda")[:ROWS].to(torch.int32)
    w = [1 + 0.5 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    return x, power, position, slot, w


def _cache(packed, Hk, D, dt):
    return vs.packed_cache(ROWS // P + 1, P, Hk, D) if packed else torch.zeros(ROWS // P + 1, P, Hk, D, dtype=dt, device="cuda")


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1e30])
@pytest.mark.parametrize("Hq,Hk,D,rot", SHAPES)
def test_heads_of_any_size_match_64_bits(Hq, Hk, D, rot, eps, interleaved, dt):
    x, power, position, slot, (qw, kw) = _heads(Hq, Hk, D, dt)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], torch.ones_like(x[:, Hq + Hk:])
    freq, at = _freq(rot), slot.long()
    kwargs = dict(q_weight=qw, k_weight=kw, eps=eps, interleaved=interleaved, scale=1.25)
    kc, vc = _cache(False, Hk, D, dt), _cache(False, Hk, D, dt)
    got = vs.norm_rope_cache(q, k, v, freq, position, slot, kc, vc, **kwargs)
    eps = float(torch.tensor(eps, dtype=F32))
    # beside what fp32 leaves of a pair: results below the normal numbers, products there times at most 2^45 (a head below the
    # range in which it is taken as it is: two roundings of 2^-150 and one of the result)
    floor = 2.0 ** -104 / _near(D)
    for have, heads, w in ((got, q, qw), (kc.flatten(0, 1)[at], k, kw)):
        want, size = _turned(_normed(heads, w, eps), position, freq, 1.25, interleaved)
        none = want.isnan()  # heads of zeros (in bf16 those of 2^-140) with eps = 0
        assert torch.equal(have.isnan().cpu(), none)
        _check(have.masked_fill(none.cuda(), 0), want.masked_fill(none, 0), size.masked_fill(none, 0) + floor, _near(D))
    assert torch.equal(vc.flatten(0, 1)[at], v)
    if D % 32:
        return
    kc, vc = _cache(True, Hk, D, dt), _cache(True, Hk, D, dt)
    assert torch.equal(vs.norm_rope_cache(q, k, v, freq, position, slot, kc, vc, **kwargs).nan_to_num(), got.nan_to_num())
    want, size = (t.nan_to_num() for t in _turned(_normed(k, kw, eps), position, freq, 1.25, interleaved))  # (NaN is stored as 0)
    have = packed_ref.decode(kc).flatten(0, 1)[at].cpu()
    step = packed_ref.scales(kc[1].transpose(1, 2).flatten(0, 1)[at]).repeat_interleave(32, -1).cpu()
    assert torch.all((want - have).abs() <= step / 2 + _near(D) * size + 2.0 ** -22 * want.abs())


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("Hq,Hk,D,rot", [s for s in SHAPES if s[2] % 32 == 0])
def test_a_head_keeps_its_bits_beside_far_ones(Hq, Hk, D, rot, dt, packed):
    x, power, position, slot, (qw, kw) = _heads(Hq, Hk, D, dt)
    plain = torch.where(power == 0, x.double(), 1.0).to(dt)
    outs = []
    for y in (x, plain):
        kc, vc = _cache(packed, Hk, D, dt), _cache(packed, Hk, D, dt)
        q = vs.norm_rope_cache(y[:, :Hq], y[:, Hq:Hq + Hk], y[:, Hq + Hk:], _freq(rot), position, slot, kc, vc, q_weight=qw, k_weight=kw, eps=1e-30)
        keys = packed_ref.decode(kc) if packed else kc
        outs.append(torch.cat([q.double(), keys.flatten(0, 1)[slot.long()].double()], 1))
    same = (power[:, :Hq + Hk] == 0).expand_as(outs[0])
    assert bool(same.any()) and torch.equal(outs[0][same], outs[1][same])


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("Hq,Hk,D,rot", SHAPES)
def test_zeros_and_infinities(Hq, Hk, D, rot, dt):
    """Zeros are zeros with any eps but 0, which makes NaN of them; infinities are NaN and what is beside them zeros."""
    x, power, position, slot, (qw, _) = _heads(Hq, 0, D, dt)
    x[0] = 0
    x[1, 0] = torch.linspace(1, 2, D, device="cuda") * 3e38 / 2
    x[1, 0, 0] = math.inf
    for eps in (0.0, 1e-30, 1e-6):
        q = vs.norm_rope_cache(x, None, None, _freq(0), position, None, None, None, q_weight=qw, eps=eps)
        assert bool(torch.isnan(q[0]).all()) if eps == 0 else bool(torch.all(q[0] == 0))
        far = x[1, 0].isinf()  # (the larger half of the numbers too: their product passes fp32)
        assert torch.equal(q[1, 0].isnan(), far) and bool(torch.all(q[1, 0][~far] == 0))
        none = (x[2:] == 0).all(-1, keepdim=True).expand_as(x[2:]) & (eps == 0)
        assert torch.equal(torch.isfinite(q[2:]), ~none)
