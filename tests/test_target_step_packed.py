"""Rounds of the example with head norms and a cache in 4 bits: every operator together, against a dense forward pass in 64
bits over what the cache then stands for."""
import importlib.util
import os

import pytest
import torch

import packed_ref
import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def _example():
    spec = importlib.util.spec_from_file_location("target_step", os.path.join(ROOT, "examples", "target_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _heads(s, tokens, at):
    """Normed and turned queries and keys, and values, in 64 bits from the bf16 projections."""
    h = s.embed[tokens.long()]
    qkv = (h @ s.w_qkv).view(len(h), s.Hq + 2 * s.Hk, s.D).double()
    z = torch.polar(torch.full((len(at), s.freq.numel()), s.rope_scale, dtype=torch.float64, device="cuda"), at.double()[:, None] * s.freq)[:, None]
    n, out = s.freq.numel(), []
    for x, w in ((qkv[:, :s.Hq], s.q_weight), (qkv[:, s.Hq:s.Hq + s.Hk], s.k_weight)):
        x = x * w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        t = torch.complex(x[..., :n], x[..., n:]) * z
        out.append(torch.cat([t.real, t.imag], -1))
    return h, *out, qkv[:, s.Hq + s.Hk:]


def test_rounds_agree_with_a_dense_pass_over_the_cache():
    s = _example().TargetStep(packed=True)
    for t in range(8):
        before = (s.tokens.clone(), s.length.clone())
        got = s.round(t)
        off, ell, kv = got["sched"]["row_off"].tolist(), got["sched"]["ell"].tolist(), got["reserved"]["new_len"].tolist()
        stored = [packed_ref.decode(c).flatten(0, 1) for c in (s.k_cache, s.v_cache)]
        prefix = torch.arange(len(s.prefix_tokens), device="cuda")
        slots = got["reserved"]["slot"].long()
        for r in range(s.R):
            n = int(before[1][r])
            own = torch.cat([before[0][r, :n], got["draft"]["x"][r, :ell[r]]])
            assert len(own) == kv[r]
            every = torch.cat([s.prefix_tokens, own])
            at = torch.arange(len(every), device="cuda")
            h, q, k, v = _heads(s, every, at)
            # the slots of the request's keys: its pages as they were during the round, whose new rows' slots are known
            table = s.cache["block_table"][r].long()
            place = torch.arange(kv[r], device="cuda")
            slot = torch.cat([prefix, table[place // s.P] * s.P + place % s.P])
            new = kv[r] - (off[r + 1] - off[r])
            assert torch.equal(slot[len(prefix) + new:], slots[off[r]:off[r + 1]])
            kept = slot  # (pages given back after the verification keep what they hold until the next round)
            # every key and value is stored within half a step of its scale (and bf16 projections, the same ones, are exact)
            for x, c, have in ((k, s.k_cache, stored[0][kept]), (v, s.v_cache, stored[1][kept])):
                step = packed_ref.scales(c[1].transpose(1, 2).flatten(0, 1)[kept]).repeat_interleave(32, -1)
                # rows computed in another batch may differ by a bf16 step of the projection: the scale's 1 / 16 and a little
                assert torch.all((x - have).abs() <= step / 2 + 2 * torch.finfo(BF).eps * x.abs().amax(-1, keepdim=True))
            rows = slice(len(prefix) + new, None)
            z = torch.einsum("nhgd,lhd->hgnl", q[rows].to(BF).double().view(-1, s.Hk, s.Hq // s.Hk, s.D), stored[0][kept]) * s.D ** -0.5
            z = z.masked_fill(at[None, :] > at[rows][:, None], -torch.inf)
            o = torch.einsum("hgnl,lhd->nhgd", torch.softmax(z, -1), stored[1][kept]).reshape(z.shape[2], -1).to(BF)
            want = ((h[rows] + o @ s.w_out) @ s.w_head).float()
            raw = got["raw"][off[r]:off[r + 1]]
            # two bf16 results of sums of 512 products with a difference of a bf16 step in some terms: a few steps of the largest
            assert torch.all((raw - want).abs() <= 8 * torch.finfo(BF).eps * want.abs().max())
        assert torch.equal(s.cache["kv_len"], s.length - 1)
    assert s.status.item() == 0
    made = s.tokens[0, int(s.prompt_len[0]):int(s.length[0])]
    assert len(made) >= 8 and torch.all((made >= 0) & (made < s.V))


def test_a_graph_replays_the_packed_operators_of_a_round():
    s = _example().TargetStep(R=3, gamma=2, packed=True)
    off = torch.tensor([0, 3, 4, 6], dtype=torch.int32, device="cuda")
    fed = torch.zeros(9, dtype=torch.int32, device="cuda")
    keep = torch.tensor([2, 1, 2], dtype=torch.int32, device="cuda")

    def body():
        r = vs.cache_reserve(s.cache, off, 9, pos_base=s.pos_base)
        h, q = s._project(fed, r["position"], r["slot"])
        o = s._attend(q, off, r["new_len"])
        return o, vs.cache_commit(s.cache, r, keep)

    fed.copy_(torch.arange(9, device="cuda") * 7)
    body()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, c = body()
    for t in range(3):
        fed.copy_((torch.arange(9, device="cuda") * 31 + 5 * t) % s.V)
        want, wc = body()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[:6], want[:6]) and torch.equal(c["kv_len"], wc["kv_len"])
