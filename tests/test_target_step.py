"""The operators run together: rounds of the example against a dense forward pass from the tokens alone."""
import importlib.util
import os

import pytest
import torch

import verify_sampling_gb300 as vs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("target_step", os.path.join(ROOT, "examples", "target_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _turned(x, at, freq, scale):
    z = torch.polar(torch.full((len(at), freq.numel()), scale, dtype=torch.float64, device="cuda"),
                    at.double()[:, None] * freq)[:, None]
    n = freq.numel()
    t = torch.complex(x[..., :n], x[..., n:]) * z
    return torch.cat([t.real, t.imag], -1)


def _dense(s, tokens):
    """Raw logits after each of ``tokens`` (a request's own, behind the prefix), in 64 bits from bf16 weights and
    with the values that the step stores in bf16 (projections, turned keys and queries) rounded alike."""
    BF = torch.bfloat16
    every = torch.cat([s.prefix_tokens, tokens])
    h = s.embed[every.long()]
    qkv = (h @ s.w_qkv).view(len(h), s.Hq + 2 * s.Hk, s.D).double()
    at = torch.arange(len(every), device="cuda")
    q, k = (_turned(t, at, s.freq, s.rope_scale).to(BF).double() for t in (qkv[:, :s.Hq], qkv[:, s.Hq:s.Hq + s.Hk]))
    v = qkv[:, s.Hq + s.Hk:]
    z = torch.einsum("nhgd,lhd->hgnl", q.view(len(q), s.Hk, -1, s.D), k) * s.D ** -0.5
    z = z.masked_fill(at[None, :] > at[:, None], -torch.inf)
    o = torch.einsum("hgnl,lhd->nhgd", torch.softmax(z, -1), v).reshape(len(q), -1).to(BF)
    return ((h + o @ s.w_out) @ s.w_head).float()[len(s.prefix_tokens):]


def test_rounds_agree_with_a_dense_forward_pass():
    m = _example()
    s = m.TargetStep()
    free0 = int(s.cache["ring"].numel() - s.prefix_pages)
    for t in range(12):
        before = (s.tokens.clone(), s.length.clone())
        got = s.round(t)
        off, ell = got["sched"]["row_off"].tolist(), got["sched"]["ell"].tolist()
        for r in range(s.R):
            n = int(before[1][r])
            own = torch.cat([before[0][r, :n], got["draft"]["x"][r, :ell[r]]])
            want = _dense(s, own)[n - 1:]  # rows of the last emitted token and the draft
            raw = got["raw"][off[r]:off[r + 1]]
            # two bf16 results of sums of 512 products with a difference of a bf16 step in some terms: a few steps of the largest
            assert torch.all((raw - want).abs() <= 8 * torch.finfo(torch.bfloat16).eps * want.abs().max())
        # the kept tokens' lengths: all but the last emitted one are in the cache
        assert torch.equal(s.cache["kv_len"], s.length - 1)
        head, tail = s.cache["ring_pos"].tolist()
        held = sum(-(-k // s.P) for k in s.cache["kv_len"].tolist())
        assert tail - head == free0 - held
        masked = (s.mask[0][torch.arange(s.V, device="cuda") // 32] >> (torch.arange(s.V, device="cuda") % 32).to(torch.int32)) & 1 == 0
        assert torch.all(torch.isneginf(got["logits"][:off[-1], masked]))
    assert s.status.item() == 0
    made = s.tokens[0, int(s.prompt_len[0]):int(s.length[0])]
    assert len(made) >= 12 and torch.all((made >= 0) & (made < s.V))


def test_same_seeds_make_the_same_tokens():
    m = _example()
    a, b = m.TargetStep(), m.TargetStep()
    for t in range(5):
        a.round(t)
        b.round(t)
    assert torch.equal(a.tokens, b.tokens) and torch.equal(a.length, b.length)


def test_a_graph_replays_the_operators_of_a_round():
    """cache_reserve, rope_cache, prefix_attention, adjust_logits and cache_commit captured once, replayed on new tokens."""
    m = _example()
    s = m.TargetStep(R=3, gamma=2)
    off = torch.tensor([0, 3, 4, 6], dtype=torch.int32, device="cuda")
    fed = torch.zeros(9, dtype=torch.int32, device="cuda")
    keep = torch.tensor([2, 1, 2], dtype=torch.int32, device="cuda")

    def body():
        r = vs.cache_reserve(s.cache, off, 9, pos_base=s.pos_base)
        h, q = s._project(fed, r["position"], r["slot"])
        o = vs.prefix_attention(q, s.k_cache, s.v_cache, off, r["new_len"], s.cache["block_table"], group_off=s.group_off,
                                prefix_len=s.prefix_len, prefix_table=s.prefix_table)
        z = ((h + o.flatten(1) @ s.w_out) @ s.w_head).float()
        z = vs.adjust_logits(z, s.tokens, s.prompt_len, s.length, row_off=off, **s.penalty)
        return z, vs.cache_commit(s.cache, r, keep)

    fed.copy_(torch.arange(9, device="cuda") * 7)
    body()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z, c = body()
    for t in range(3):
        fed.copy_((torch.arange(9, device="cuda") * 31 + 5 * t) % s.V)
        want, wc = body()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(z[:6], want[:6]) and torch.equal(c["kv_len"], wc["kv_len"])
