"""Head norms with rotary positions, and keys and values written to caches of either kind, against 64 bits."""
import math

import pytest
import torch

import packed_ref
import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _normed(x, weight, eps):
    """The norm in 64 bits."""
    x = x.double().cpu()
    if weight is None:
        return x
    return x * weight.double().cpu() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def _turned(x, position, freq, scale, interleaved):
    """Turned pairs of x (64 bits, host), and the sizes |x| + |y| of each pair (an element past them: its own)."""
    n = freq.numel()
    z = torch.polar(torch.full((len(position), n), scale, dtype=torch.float64),
                    position.double().cpu()[:, None] * freq.cpu())[:, None]
    y, size = x.clone(), x.abs()
    at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    t = torch.complex(x[..., at[0]], x[..., at[1]]) * z
    y[..., at[0]], y[..., at[1]] = t.real, t.imag
    for a in at:
        size[..., a] = (x[..., at[0]].abs() + x[..., at[1]].abs()) * scale
    return y, size


def _near(D):
    """What fp32 leaves, relative to a pair's size: the sum of squares (each term a rounding, D / 32 + 5 sums in a row at
    most 16 + 5; half of it under the root), the root (2 ulp), two products: under (D / 64 + 16) roundings; angle and
    rotation 1e-6 as for rope_cache."""
    return 1e-6 + (D / 64 + 16) * 2.0 ** -24


def _check(got, want, size, near):
    err, tol = (got.double().cpu() - want).abs(), near * size
    if got.dtype == BF:
        tol = tol + torch.finfo(BF).eps / 2 * (want.abs() + tol)
    assert torch.all(err <= tol), float((err - tol).max())


def _inputs(rows, Hq, Hk, D, dt, seed=0, far=1 << 24, P=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    # heads of very different sizes: the norm takes them out
    qkv = torch.randn(rows, Hq + 2 * Hk, D, generator=g, device="cuda")
    qkv = (qkv * torch.exp(2 * torch.randn(rows, Hq + 2 * Hk, 1, generator=g, device="cuda"))).to(dt)
    position = torch.randint(0, far, (rows,), generator=g, device="cuda", dtype=torch.int32)
    if rows > 1:
        position[0], position[-1] = 0, far - 1
    pages = -(-rows // P) + 2
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:rows].to(torch.int32)
    w = [1 + 0.5 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    return qkv, position, slot, pages, w


def _freq(rot):
    return vs.rope_frequencies(rot)[0] if rot else torch.zeros(0, dtype=torch.float64, device="cuda")


def _filled_cache(pages, P, Hk, D):
    data, scale = vs.packed_cache(pages, P, Hk, D)
    return data.fill_(0x5A), scale.fill_(0xA5)


SIZES = [(1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (5, 3, 1, 80, 80), (7, 4, 2, 96, 32), (33, 6, 3, 50, 22), (2, 8, 8, 512, 512),
         (311, 40, 8, 128, 64), (700, 4, 1, 64, 64), (1300, 2, 2, 24, 16), (9, 5, 5, 33, 0), (305, 100, 4, 128, 128), (64, 7, 1, 136, 24),
         (40, 3, 2, 256, 256), (700, 40, 8, 128, 128), (2100, 32, 4, 128, 64), (1500, 70, 5, 64, 64), (1111, 9, 3, 256, 192)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot", SIZES)
def test_normed_and_turned_rows_match_64_bits(rows, Hq, Hk, D, rot, interleaved, dt):
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, Hq, Hk, D, dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    kc, vc = (torch.full((pages, 8, Hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    freq = _freq(rot)
    kwargs = dict(q_weight=qw, k_weight=kw, eps=1e-3, interleaved=interleaved, scale=1.25)
    got = vs.norm_rope_cache(q, k, v, freq, position, slot, kc, vc, **kwargs)
    _check(got, *_turned(_normed(q, qw, 1e-3), position, freq, 1.25, interleaved), _near(D))
    at = slot.long()
    _check(kc.flatten(0, 1)[at], *_turned(_normed(k, kw, 1e-3), position, freq, 1.25, interleaved), _near(D))
    assert torch.equal(vc.flatten(0, 1)[at], v)
    rest = torch.ones(pages * 8, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(kc.flatten(0, 1)[rest] == 7) and torch.all(vc.flatten(0, 1)[rest] == 7)
    # the queries alone, in place, from rows that lie apart and off 16 bytes
    wide = torch.zeros(rows, Hq + 1, D + 1, dtype=dt, device="cuda")
    view = wide[:, 1:, 1:]
    view.copy_(q)
    vs.norm_rope_cache(view, None, None, freq, position, None, None, None, q_out=view, **{**kwargs, "k_weight": None})
    _check(view, *_turned(_normed(q, qw, 1e-3), position, freq, 1.25, interleaved), _near(D))
    assert torch.all(wide[:, 0] == 0) and torch.all(wide[:, :, 0] == 0)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot", SIZES)
def test_without_weights_it_is_rope_cache(rows, Hq, Hk, D, rot, interleaved, dt):
    qkv, position, slot, pages, _ = _inputs(rows, Hq, Hk, D, dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    caches = [[torch.full((pages, 8, Hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2)] for _ in range(2)]
    a = vs.rope_cache(q, k, v, _freq(rot), position, slot, *caches[0], interleaved=interleaved, scale=0.75)
    b = vs.norm_rope_cache(q, k, v, _freq(rot), position, slot, *caches[1], interleaved=interleaved, scale=0.75)
    assert torch.equal(a, b) and torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])


@pytest.mark.parametrize("rows", [30, 1300])
@pytest.mark.parametrize("which", ["q", "k"])
def test_a_norm_of_one_kind_alone(which, rows):
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, 40, 8, 64, BF)
    q, k, v = qkv[:, :40], qkv[:, 40:48], qkv[:, 48:]
    caches = [[torch.zeros(pages, 8, 8, 64, dtype=BF, device="cuda") for _ in range(2)] for _ in range(3)]
    both = vs.norm_rope_cache(q, k, v, _freq(64), position, slot, *caches[0], q_weight=qw, k_weight=kw)
    none = vs.norm_rope_cache(q, k, v, _freq(64), position, slot, *caches[1])
    one = vs.norm_rope_cache(q, k, v, _freq(64), position, slot, *caches[2], **{f"{which}_weight": qw if which == "q" else kw})
    assert torch.equal(one, both if which == "q" else none)
    assert torch.equal(caches[2][0], caches[1 if which == "q" else 0][0])


@pytest.mark.parametrize("rows,Hq,Hk,D", [(1500, 40, 8, 128), (4500, 8, 1, 64)])
def test_the_batch_does_not_change_a_row(rows, Hq, Hk, D):
    """Rows alone, in a few and in a long batch, and of heads that lie apart, come out with the same bits."""
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, Hq, Hk, D, BF)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    freq = _freq(D)

    def call(n, q=q):
        kc, vc = vs.packed_cache(pages, 8, Hk, D), vs.packed_cache(pages, 8, Hk, D)
        out = vs.norm_rope_cache(q[:n], k[:n], v[:n], freq, position[:n].contiguous(), slot[:n].contiguous(), kc, vc, q_weight=qw, k_weight=kw)
        return out, *vs.cache_read_packed(kc, vc, slot[:n].contiguous())

    long = call(rows)
    for n in (1, 7, 400):
        assert all(torch.equal(a, b[:n]) for a, b in zip(call(n), long))
    apart = torch.zeros(rows, 2 * Hq, D, dtype=BF, device="cuda")[:, ::2]
    apart.copy_(q)
    assert all(torch.equal(a, b) for a, b in zip(call(rows, apart), long))


PACKED = [(1, 32, 8, 128, 128, 16), (1, 1, 1, 32, 2, 1), (7, 4, 2, 96, 32, 8), (33, 6, 3, 64, 22, 5), (2, 8, 8, 512, 512, 16),
          (311, 40, 8, 128, 64, 64), (700, 4, 1, 64, 32, 16), (9, 5, 5, 32, 0, 3), (64, 7, 1, 160, 24, 24), (40, 3, 2, 256, 256, 32),
          (700, 40, 8, 128, 128, 64), (2100, 32, 4, 128, 64, 16), (1500, 70, 5, 64, 64, 16), (1111, 9, 3, 256, 192, 16)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot,P", PACKED)
def test_packed_keys_and_values_match_64_bits(rows, Hq, Hk, D, rot, P, interleaved, dt):
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, Hq, Hk, D, dt, P=P)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    kc, vc = _filled_cache(pages, P, Hk, D), _filled_cache(pages, P, Hk, D)
    before = [packed_ref.decode(c).flatten(0, 1) for c in (kc, vc)]
    freq = _freq(rot)
    kwargs = dict(q_weight=qw, k_weight=kw, eps=1e-3, interleaved=interleaved, scale=1.25)
    got = vs.norm_rope_cache(q, k, v, freq, position, slot, kc, vc, **kwargs)
    _check(got, *_turned(_normed(q, qw, 1e-3), position, freq, 1.25, interleaved), _near(D))
    at = slot.long()
    # values: the definition's very codes (bf16 values have 8 bits, and no quotient by 7 or by a scale of 4 comes within an
    # fp32 rounding of a border without lying on it; 24-bit values may: see below)
    stored = [packed_ref.decode(c).flatten(0, 1) for c in (kc, vc)]
    code, n = packed_ref.encode(v)
    if dt == BF:
        assert torch.equal(stored[1][at], (n * packed_ref.scales(code)[..., None]).flatten(-2))
    # within half a step (of a scale that may be the next one where amax / 7 lies on a border) and fp32's error
    y, size = _turned(_normed(k, kw, 1e-3), position, freq, 1.25, interleaved)
    for x, near, have, c in ((y.cuda(), (_near(D) * size).cuda(), stored[0][at], kc), (v.double(), 2.0 ** -23 * v.double().abs(), stored[1][at], vc)):
        step = packed_ref.scales(c[1].transpose(1, 2).flatten(0, 1)[at]).repeat_interleave(32, -1)  # [rows, Hk, D]
        assert torch.all((x - have).abs() <= step / 2 + near + 2.0 ** -22 * x.abs())
        group = x.unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1) / 7
        wide = near.unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1) / 7
        # the scale is amax / 7 within half a unit of its fourth bit
        assert torch.all((step - group).abs() <= step / 16 + wide + 2.0 ** -22 * group + 2.0 ** -20)
    # other slots as they were
    rest = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    rest[at] = False
    for a, b in zip(stored, before):
        assert torch.equal(a[rest], b[rest])
    for out_dt in (F32, BF):
        rk, rv = vs.cache_read_packed(kc, vc, slot, dtype=out_dt)
        assert torch.equal(rk.double(), stored[0][at]) and torch.equal(rv.double(), stored[1][at])


def test_codes_of_special_values():
    """Zeros, ties, the scales' ends, infinities and NaN."""
    D, P = 64, 4
    v = torch.zeros(8, 1, D, device="cuda")
    v[1, 0, :15] = torch.arange(-7, 8, device="cuda") + 0.0  # scale 1: whole numbers
    v[2, 0, :6] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -6.5], device="cuda")  # halves go to even numbers
    v[3, 0, 0] = 1e9  # saturates
    v[4, 0, :3] = torch.tensor([2.0 ** -21, 2.0 ** -20, 1.6 * 2.0 ** -20], device="cuda")  # the smallest scale
    v[5, 0, :3] = torch.tensor([math.inf, -math.inf, 5.0], device="cuda")
    v[6, 0, :2] = torch.tensor([math.nan, 7.0], device="cuda")
    v[7, 0, 32:34] = torch.tensor([3.5, 7 * 17 / 16], device="cuda")  # 17 / 16 lies between 1 and 9 / 8: up
    kc, vc = vs.packed_cache(2, P, 1, D), vs.packed_cache(2, P, 1, D)
    slot = torch.arange(8, dtype=torch.int32, device="cuda")
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    vs.norm_rope_cache(v, torch.zeros_like(v), v, _freq(0), pos, slot, kc, vc)
    _, got = vs.cache_read_packed(kc, vc, slot, dtype=F32)
    got = got[:, 0].cpu()
    assert torch.all(got[0] == 0)
    assert torch.equal(got[1, :15], torch.arange(-7.0, 8.0)) and torch.all(got[1, 15:] == 0)
    assert got[2, :6].tolist() == [7.0, 0.0, 2.0, 2.0, 0.0, -6.0]
    assert got[3, 0] == 7 * 3840.0 and got[3, 1] == 0
    assert got[4, :3].tolist() == [0.0, 2.0 ** -20, 2.0 ** -19]
    assert got[5, :3].tolist() == [7 * 3840.0, -7 * 3840.0, 0.0]
    assert got[6, :2].tolist() == [0.0, 7.0]
    assert got[7, 32:34].tolist() == [3 * 1.125, 7 * 1.125]
    assert vc[1][1, 0, 3, 1] == 161 and packed_ref.scales(torch.tensor(161)).item() == 1.125


@pytest.mark.parametrize("packed", [False, True])
def test_left_out_rows_bad_slots_and_far_positions(packed):
    qkv, position, slot, pages, (qw, kw) = _inputs(6, 2, 1, 64, F32, far=1000)
    position[1], position[2], slot[3], slot[4] = -1, 1 << 24, -1, pages * 8
    freq = _freq(64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((6, 2, 64), 5.0, device="cuda")
    make = (lambda: _filled_cache(pages, 8, 1, 64)) if packed else (lambda: torch.full((pages, 8, 1, 64), 7.0, device="cuda"))
    kc, vc = make(), make()
    values = (lambda c: packed_ref.decode(c).flatten(0, 1)) if packed else (lambda c: c.flatten(0, 1).double())
    empty = values(make())
    vs.norm_rope_cache(qkv[:, :2], qkv[:, 2:3], qkv[:, 3:], freq, position, slot, kc, vc, q_weight=qw, k_weight=kw, q_out=q_out, status=status)
    assert status.item() == vs.STATUS_BAD_PAGE | vs.STATUS_BAD_POSITION
    assert torch.all(q_out[1] == 5)
    position[2] = (1 << 24) - 1
    want, size = _turned(_normed(qkv[:, :2], qw, 1e-6), position, freq, 1.0, False)
    live = [0, 2, 3, 4, 5]
    _check(q_out[live], want[live], size[live], _near(64))
    written = sorted(int(slot[i]) for i in (0, 2, 5))
    for c in (kc, vc):
        changed = (values(c) != empty).any(-1).any(-1).nonzero()[:, 0].tolist()
        assert changed == written
    if packed:
        status.zero_()
        out = [torch.full((6, 1, 64), 9.0, device="cuda") for _ in range(2)]
        vs.cache_read_packed(kc, vc, slot, out=tuple(out), status=status)
        assert status.item() == vs.STATUS_BAD_PAGE
        assert torch.all(out[0][3:5] == 0) and torch.all(out[1][3:5] == 0) and torch.equal(out[1][[0, 2, 5]].double(), values(vc)[slot[[0, 2, 5]].long()])


@pytest.mark.parametrize("rows", [20, 1300])
@pytest.mark.parametrize("packed", [False, True])
def test_stream_and_graph(packed, rows):
    qkv, position, slot, pages, (qw, kw) = _inputs(rows, 40, 4, 128, BF)
    freq = _freq(128)
    kc, vc = (vs.packed_cache(pages, 8, 4, 128) if packed else torch.zeros(pages, 8, 4, 128, dtype=BF, device="cuda") for _ in range(2))
    data = kc[0] if packed else kc
    call = lambda **kwargs: vs.norm_rope_cache(qkv[:, :40], qkv[:, 40:44], qkv[:, 44:], freq, position, slot, kc, vc, q_weight=qw,  # noqa: E731
                                               k_weight=kw, **kwargs)
    want, keys = call(), data.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
        if packed:
            k, v = vs.cache_read_packed(kc, vc, slot)
    data.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(data, keys)
    if packed:
        assert torch.equal(v.double(), packed_ref.decode(vc).flatten(0, 1)[slot.long()])


def test_refusals():
    qkv, position, slot, pages, (qw, kw) = _inputs(4, 2, 1, 64, F32)
    freq = _freq(64)
    q, k, v = qkv[:, :2], qkv[:, 2:3], qkv[:, 3:]
    kc, vc = (torch.zeros(pages, 8, 1, 64, device="cuda") for _ in range(2))
    pk, pv = vs.packed_cache(pages, 8, 1, 64), vs.packed_cache(pages, 8, 1, 64)
    ok = (q, k, v, freq, position, slot)
    for caches, kwargs, err in (((kc, vc), dict(q_weight=qw.bfloat16()), TypeError), ((kc, vc), dict(q_weight=qw[:63]), ValueError),
                                ((kc, vc), dict(k_weight=kw.cpu()), TypeError), ((kc, pv), {}, ValueError), ((pk, vc), {}, ValueError),
                                ((pk, (pv[0][:1], pv[1][:1])), {}, ValueError), ((pk, (pv[0], pv[1][..., :1])), {}, ValueError),
                                (((pk[0].float(), pk[1]), pv), {}, TypeError), ((pk, (pv[0].transpose(1, 2), pv[1])), {}, ValueError),
                                ((None, vc), {}, TypeError), ((list(pk), pv), {}, TypeError), ((kc.bfloat16(), vc), {}, TypeError), ((kc, vc), dict(eps=-1.0), vs.SpecError),
                                ((kc, vc), dict(eps=math.nan), vs.SpecError), ((kc[:1], vc), {}, ValueError)):
        with pytest.raises(err):
            vs.norm_rope_cache(*ok, *caches, **kwargs)
    for args, err in (((pk, pv, slot.long()), TypeError), ((pk, (pv[0][:1], pv[1][:1]), slot), ValueError), ((kc, vc, slot), (TypeError, ValueError))):
        with pytest.raises(err):
            vs.cache_read_packed(*args)
    with pytest.raises(TypeError):
        vs.cache_read_packed(pk, pv, slot, dtype=torch.float16)
    with pytest.raises(ValueError):
        vs.packed_cache(1, 8, 1, 48)
    assert vs.cache_read_packed(pk, pv, slot[:0])[0].shape == (0, 1, 64)


def test_scales_on_both_sides_of_their_borders():
    """A group whose largest magnitude is 7 h, h half way between two scales, takes the larger one; the next smaller number
    the smaller one."""
    D, P = 32, 5
    code = torch.arange(1, 255, dtype=torch.float64)
    scale = lambda c: torch.exp2((c // 8) - 20) * (1 + c % 8 / 8)  # noqa: E731
    border = (7 * (scale(code - 1) + scale(code)) / 2).float()
    v = torch.zeros(2 * len(code), 1, D)
    v[:len(code), 0, 3] = border
    v[len(code):, 0, 3] = torch.nextafter(border, torch.zeros(()))
    v[::2] *= -1
    pages = -(-len(v) // P)
    kc, vc = vs.packed_cache(pages, P, 1, D), vs.packed_cache(pages, P, 1, D)
    slot = torch.arange(len(v), dtype=torch.int32, device="cuda")
    vs.norm_rope_cache(v.cuda(), torch.zeros_like(v).cuda(), v.cuda(), _freq(0), torch.zeros_like(slot), slot, kc, vc)
    got = vc[1].flatten().cpu().long()[:len(v)]
    assert torch.equal(got, torch.cat([code, code - 1]).long())
