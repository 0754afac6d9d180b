"""The example's rounds when requests run out of pages: a refused request emits nothing and stays as it is."""
import importlib.util
import os
import types

import pytest
import torch

import verify_sampling_gb300 as vs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32 = torch.int32


def _example():
    spec = importlib.util.spec_from_file_location("target_step", os.path.join(ROOT, "examples", "target_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain_calls(R, gamma, V, gen):
    """The calls of a round on the CPU: random drafts and verdicts, and the page bookkeeping as a loop over requests."""

    def draft_sample(inp, seed, status=None):
        return {"x": torch.randint(0, V, (R, gamma), generator=gen, dtype=I32), "q_tok": None, "lse_q": None, "a": None}

    def schedule(*_, status=None):
        ell = torch.randint(0, gamma + 1, (R,), generator=gen, dtype=I32)
        return {"ell": ell, "row_off": torch.cat([torch.zeros(1, dtype=I32), (1 + ell).cumsum(0).to(I32)])}

    def cache_reserve(c, off, rows, pos_base=None, status=None):
        P, (R_, width) = c["page_size"], c["block_table"].shape
        request = torch.full((rows,), -1, dtype=I32)
        slot, position, new_len = request.clone(), request.clone(), c["kv_len"].clone()
        head, tail = c["ring_pos"].tolist()
        for r in range(R_):
            a, b, kv = int(off[r]), int(off[r + 1]), int(c["kv_len"][r])
            have, want = -(-kv // P), -(-(kv + b - a) // P)
            if want > width or (want > have and head + want - have > tail):
                status |= vs.STATUS_NO_PAGES
                continue
            for i in range(have, want):
                c["block_table"][r, i] = c["ring"][head % len(c["ring"])]
                head += 1
            new_len[r] = kv + b - a
            request[a:b] = r
            at = torch.arange(kv, kv + b - a)
            position[a:b] = (at + pos_base[r]).to(I32)
            slot[a:b] = c["block_table"][r][at // P] * P + (at % P).to(I32)
        return {"request": request, "slot": slot, "position": position, "new_len": new_len, "ring_pos": torch.tensor([head, tail])}

    def cache_commit(c, res, keep, status=None):
        P, kv = c["page_size"], c["kv_len"].clone()
        head, tail = res["ring_pos"].tolist()
        for r in range(len(kv)):
            kv[r] = 0 if keep[r] < 0 else min(int(kv[r] + keep[r]), int(res["new_len"][r]))
            for i in range(-(-int(kv[r]) // P), -(-int(res["new_len"][r]) // P)):
                c["ring"][tail % len(c["ring"])] = c["block_table"][r, i]
                tail += 1
        return {"kv_len": kv, "ring_pos": torch.tensor([head, tail])}

    def prefix_attention(q, *_, **__):
        return q

    def adjust_logits(z, *_, **__):
        return z

    def verify(mode, z, off, ell, x, seed, **__):
        n = (torch.rand(R, generator=gen) * (1 + ell)).to(I32) + 1  # 1 .. 1 + ell emitted tokens
        out = torch.randint(0, V, (R, gamma + 1), generator=gen, dtype=I32)
        return {"n_out": n, "out_tok": torch.where(torch.arange(gamma + 1) < n[:, None], out, -1)}

    return types.SimpleNamespace(draft_sample=draft_sample, schedule=schedule, cache_reserve=cache_reserve, cache_commit=cache_commit,
                                 prefix_attention=prefix_attention, adjust_logits=adjust_logits, verify=verify, VERIFY_SAMPLE=0)


def _check_rounds(s, rounds, step):
    """Lengths, tokens and cache of a run that goes on after requests are full."""
    full = torch.zeros(s.R, dtype=torch.bool)
    for t in range(rounds):
        tokens, length, kv, x0 = s.tokens.clone(), s.length.clone(), s.cache["kv_len"].clone(), s.x0.clone()
        got = step(t)
        refused = (got["reserved"]["new_len"] == kv).cpu()
        full |= refused
        n, out = got["verify"]["n_out"], got["verify"]["out_tok"]
        assert torch.equal(s.cache["kv_len"], s.length - 1)
        for r in range(s.R):
            a, b, k = int(length[r]), int(s.length[r]), int(n[r])
            assert torch.equal(s.tokens[r, :a], tokens[r, :a])
            assert b - a == (0 if refused[r] else k)
            if refused[r]:
                assert s.x0[r] == x0[r]
            else:
                assert torch.equal(s.tokens[r, a:b], out[r, :k]) and s.x0[r] == out[r, k - 1]
    return full


@pytest.mark.parametrize("pages", [None, 5])
def test_full_requests_emit_nothing(monkeypatch, pages):
    m = _example()
    R, gamma, V, P, own = 3, 2, 50, 4, 3
    gen = torch.Generator().manual_seed(3)
    monkeypatch.setattr(m, "vs", _plain_calls(R, gamma, V, gen))
    s = m.TargetStep.__new__(m.TargetStep)
    z = lambda *n: torch.zeros(*n, dtype=I32)  # noqa: E731
    s.R, s.gamma, s.V, s.P, s.draft_in, s.wl = R, gamma, V, P, types.SimpleNamespace(), types.SimpleNamespace(K=0)
    s.sps = s.b_lo = s.b_step = s.group_off = s.prefix_len = s.prefix_table = s.mask = s.mask_row = s.k_cache = s.v_cache = None
    s.penalty, s.pos_base, s.status = {}, z(R), z(1)
    s.w_out = s.w_head = torch.zeros(8, 8)
    s._project = lambda tokens, position, slot: (torch.zeros(len(tokens), 8), torch.zeros(len(tokens), 2, 4))
    s.tokens, s.prompt_len, s.length, s.x0 = z(R, own * P + 2), z(R) + 1, z(R) + 1, z(R)
    n_pages = R * own
    s.cache = {"kv_len": z(R), "block_table": z(R, own), "ring": torch.arange(n_pages, dtype=I32), "page_size": P,
               "ring_pos": torch.tensor([0, pages or n_pages])}
    full = _check_rounds(s, 40, s.round)
    assert torch.all(full) and s.status.item() == vs.STATUS_NO_PAGES
    assert torch.all(s.length <= own * P + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [None, 7])
def test_full_requests_emit_nothing_on_the_gpu(pages):
    """Past the capacity: the rounds of a small cache agree with those of a large one until a request is full."""
    m = _example()
    kw = dict(R=4, gamma=3, prompt=5, page_size=8)
    s = m.TargetStep(room=24, **kw)
    if pages is not None:  # pages that no request holds, besides the prompts'
        s.cache["ring_pos"][1] = s.cache["ring_pos"][0] + pages
    full = _check_rounds(s, 40, s.round)
    assert torch.all(full) and s.status.item() == vs.STATUS_NO_PAGES
    assert int(s.length.max()) <= 25
    wide = m.TargetStep(room=400, **kw)
    alike = torch.ones(4, dtype=torch.bool)
    small = m.TargetStep(room=24, **kw)
    for t in range(12):
        a, b = small.round(t), wide.round(t)
        alike &= (a["reserved"]["request"][a["sched"]["row_off"][:-1].long()] >= 0).cpu()
        assert torch.equal(a["sched"]["ell"], b["sched"]["ell"]) or not torch.all(alike)
        if not torch.all(alike):
            break
        assert torch.equal(small.length, wide.length) and torch.equal(small.x0, wide.x0)
    assert wide.status.item() == 0
