"""Rotary positions and the cache write on the GPU against complex products in 64 bits."""
import pytest
import torch

import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu


def _turned(x, position, freq, scale, interleaved):
    """The formula in 64 bits, and the sizes |x| + |y| of each pair (laid out like the result)."""
    x, n = x.double().cpu(), freq.numel()
    z = torch.polar(torch.full((len(position), n), scale, dtype=torch.float64),
                    position.double().cpu()[:, None] * freq.cpu())[:, None]
    y, size = x.clone(), torch.zeros_like(x)
    at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    t = torch.complex(x[..., at[0]], x[..., at[1]]) * z
    y[..., at[0]], y[..., at[1]] = t.real, t.imag
    for a in at:
        size[..., a] = x[..., at[0]].abs() + x[..., at[1]].abs()
    return y, size * scale


def _check(got, want, size):
    """An angle within 4e-7 rad (its remainder and the sine to an ulp or two each) and three fp32 roundings of
    products no larger than the pair, then one rounding to the stored type."""
    err = (got.double().cpu() - want).abs()
    tol = 1e-6 * size
    if got.dtype == torch.bfloat16:
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + tol)
    assert torch.all(err <= tol), float((err - tol).max())


def _inputs(rows, Hq, Hk, D, dt, seed=0, far=1 << 24, pages=None, P=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(rows, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
    position = torch.randint(0, far, (rows,), generator=g, device="cuda", dtype=torch.int32)
    if rows > 1:
        position[0], position[-1] = 0, far - 1
    pages = -(-rows // P) + 2
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:rows].to(torch.int32)
    caches = [torch.full((pages, P, Hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    return qkv, position, slot, caches


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot", [
    (1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (5, 3, 1, 80, 80), (7, 4, 2, 96, 32), (33, 6, 3, 50, 22), (2, 8, 8, 512, 512),
    (311, 40, 8, 128, 64), (700, 4, 1, 64, 64), (1300, 2, 2, 24, 16), (9, 5, 5, 33, 0), (305, 100, 4, 128, 128), (64, 7, 1, 136, 24)])
def test_turned_rows_and_cache_match_64_bits(rows, Hq, Hk, D, rot, interleaved, dt):
    qkv, position, slot, (kc, vc) = _inputs(rows, Hq, Hk, D, dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    freq, _ = vs.rope_frequencies(rot) if rot else (torch.zeros(0, dtype=torch.float64, device="cuda"), 1)
    got = vs.rope_cache(q, k, v, freq, position, slot, kc, vc, interleaved=interleaved, scale=1.25)
    _check(got, *_turned(q, position, freq, 1.25, interleaved))
    want, size = _turned(k, position, freq, 1.25, interleaved)
    at = slot.long()
    _check(kc.flatten(0, 1)[at], want, size)
    assert torch.equal(vc.flatten(0, 1)[at], v)
    rest = torch.ones(kc.shape[0] * kc.shape[1], dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(kc.flatten(0, 1)[rest] == 7) and torch.all(vc.flatten(0, 1)[rest] == 7)
    # the queries in place, from rows that lie apart and off 16 bytes
    wide = torch.zeros(rows, Hq + 1, D + 1, dtype=dt, device="cuda")
    view = wide[:, 1:, 1:]
    view.copy_(q)
    vs.rope_cache(view, None, None, freq, position, None, None, None, interleaved=interleaved, scale=1.25, q_out=view)
    assert torch.equal(view, got) and torch.all(wide[:, 0] == 0) and torch.all(wide[:, :, 0] == 0)


def test_left_out_rows_bad_slots_and_far_positions():
    qkv, position, slot, (kc, vc) = _inputs(6, 2, 1, 64, torch.float32, far=1000)
    position[1], position[2], slot[3], slot[4] = -1, 1 << 24, -1, kc.shape[0] * kc.shape[1]
    freq, _ = vs.rope_frequencies(64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((6, 2, 64), 5.0, device="cuda")
    vs.rope_cache(qkv[:, :2], qkv[:, 2:3], qkv[:, 3:], freq, position, slot, kc, vc, q_out=q_out, status=status)
    assert status.item() == vs.STATUS_BAD_PAGE | vs.STATUS_BAD_POSITION
    assert torch.all(q_out[1] == 5)
    position[2] = (1 << 24) - 1
    want, size = _turned(qkv[:, :2], position, freq, 1.0, False)
    live = [0, 2, 3, 4, 5]
    _check(q_out[live], want[live], size[live])
    written = [int(slot[i]) for i in (0, 2, 5)]
    assert torch.equal(vc.flatten(0, 1)[written], qkv[[0, 2, 5], 3:])
    assert int((kc.flatten(0, 1) != 7).any(-1).any(-1).sum()) == 3


def test_stream_and_graph():
    qkv, position, slot, (kc, vc) = _inputs(20, 4, 2, 64, torch.bfloat16)
    freq, _ = vs.rope_frequencies(64)
    call = lambda **kw: vs.rope_cache(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], freq, position, slot, kc, vc, **kw)  # noqa: E731
    want, keys = call(), kc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(kc.flatten(0, 1)[slot.long()], keys.flatten(0, 1)[slot.long()])


def test_refusals():
    qkv, position, slot, (kc, vc) = _inputs(4, 2, 1, 64, torch.float32)
    freq, _ = vs.rope_frequencies(64)
    q, k, v = qkv[:, :2], qkv[:, 2:3], qkv[:, 3:]
    for args in ((q, k, v, freq.float(), position, slot, kc, vc), (q, k.bfloat16(), v, freq, position, slot, kc, vc),
                 (q.half(), k.half(), v.half(), freq, position, slot, kc, vc), (q.cpu(), k, v, freq, position, slot, kc, vc),
                 (q, k, v, freq, position.long(), slot, kc, vc)):
        with pytest.raises(TypeError):
            vs.rope_cache(*args)
    for args in ((q, k, v[:3], freq, position, slot, kc, vc), (q, k, v, freq, position, slot, kc, vc[:1]),
                 (q, k, v, freq, position[:3], slot, kc, vc), (q.transpose(1, 2), k, v, freq, position, slot, kc, vc)):
        with pytest.raises(ValueError):
            vs.rope_cache(*args)
    with pytest.raises(vs.SpecError):
        vs.rope_cache(q, k, v, torch.cat([freq, freq]), position, slot, kc, vc)  # 128 elements of 64


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,D,rot", [
    (609, 64, 8, 128, 128), (2601, 16, 2, 128, 64), (4301, 8, 1, 160, 96), (6001, 7, 1, 128, 128), (2500, 5, 1, 512, 512),
    (60001, 2, 1, 48, 16), (99991, 1, 0, 64, 64), (32003, 0, 3, 64, 64), (20001, 3, 1, 64, 0), (1300, 20, 8, 256, 32),
    (700, 100, 4, 256, 128)])
def test_many_rows_with_heads_side_by_side(rows, Hq, Hk, D, rot, interleaved, dt):
    """The formula, the same bits as calls of a few rows each, and rows that go nowhere."""
    qkv, position, slot, (kc, vc) = _inputs(rows, Hq, Hk, D, dt, far=1 << 20)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    freq, _ = vs.rope_frequencies(rot) if rot else (torch.zeros(0, dtype=torch.float64, device="cuda"), 1)
    n_slots = kc.shape[0] * kc.shape[1]
    position[5], position[rows - 2], slot[7], slot[9], position[11] = -1, -1, -1, n_slots, 1 << 24
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    few, many, part = [torch.full((rows, Hq, D), 5.0, dtype=dt, device="cuda") for _ in range(3)]
    kw = dict(interleaved=interleaved, scale=1.25, status=status)
    kf, vf = kc.clone(), vc.clone()

    def call(rows, out, kc, vc):
        if Hk == 0:
            return vs.rope_cache(q[rows], None, None, freq, position[rows], None, None, None, q_out=out[rows], **kw)
        return vs.rope_cache(q[rows], k[rows], v[rows], freq, position[rows], slot[rows], kc, vc, q_out=out[rows], **kw)

    call(slice(0, rows), many, kc, vc)
    assert status.item() == vs.STATUS_BAD_POSITION | (vs.STATUS_BAD_PAGE if Hk else 0)
    step = min(500, 10000000 // ((Hq + 2 * Hk) * D * 4))  # too few for the kernel of long batches
    for a in range(0, rows, step):
        call(slice(a, a + step), few, kf, vf)
    assert torch.equal(many, few) and torch.equal(kc, kf) and torch.equal(vc, vf)
    assert Hq == 0 or (torch.all(many[5] == 5) and torch.all(many[rows - 2] == 5))
    live = torch.ones(rows, dtype=torch.bool)
    live[[5, rows - 2, 11]] = False
    if Hq:
        want, size = _turned(q[live], position[live], freq, 1.25, interleaved)
        _check(many[live], want, size)
    if Hk:
        live[[7, 9]] = False
        at = slot[live].long()
        want, size = _turned(k[live], position[live], freq, 1.25, interleaved)
        _check(kc.flatten(0, 1)[at], want, size)
        assert torch.equal(vc.flatten(0, 1)[at], v[live])
        rest = torch.ones(n_slots, dtype=torch.bool, device="cuda")
        rest[at] = False
        rest[slot[11].long()] = False
        assert torch.all(kc.flatten(0, 1)[rest] == 7) and torch.all(vc.flatten(0, 1)[rest] == 7)
    if Hq:  # the queries in place
        part.copy_(q)
        vs.rope_cache(part, None, None, freq, position, None, None, None, q_out=part, interleaved=interleaved, scale=1.25)
        live[:] = position.cpu() >= 0
        assert torch.equal(part[live], many[live]) and torch.equal(part[~live], q[~live])
