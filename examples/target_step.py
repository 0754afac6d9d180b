"""Rounds of speculative decoding around a small target model with a paged cache.

    python examples/target_step.py [rounds]

Each round, without a host synchronisation: draft, schedule, cache slots for the
scheduled rows (cache_reserve), rotary positions and the cache write (rope_cache),
attention over a system prompt that all requests share and each request's own pages
(prefix_attention), penalties and a grammar mask on the packed logits
(adjust_logits), verification, and the kept lengths and freed pages (cache_commit).
The target is one attention layer between random embeddings and a random output
matrix: it stands in for a real one, whose other layers change nothing here.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
import verify_sampling_gb300 as vs  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


class TargetStep:
    """R requests behind one shared prefix; ``tokens`` are each request's own tokens so far (``length`` of them,
    ``prompt_len`` of those the prompt).  All but a request's last token are in the cache, which has pages for
    ``room`` tokens a request: one whose next rows do not fit is refused by cache_reserve and stays as it is."""

    def __init__(self, R=6, gamma=4, V=1000, Hq=8, Hk=2, D=64, page_size=16, prefix=75, prompt=9, room=400, seed=0):
        dev, g = "cuda", torch.Generator("cuda").manual_seed(seed)
        self.R, self.gamma, self.V, self.Hq, self.Hk, self.D, self.P = R, gamma, V, Hq, Hk, D, page_size
        wl = synth.WORKLOADS["tiny"].scaled(R=R, gamma=gamma, V=V)
        inp = {k: (t.to(dev) if isinstance(t, torch.Tensor) else t) for k, t in synth.make_inputs(wl, "cpu").items()}
        self.draft_in, self.wl = synth.draft_inputs(inp), wl
        self.sps, self.b_lo, self.b_step = inp["sps"], inp["b_lo"], inp["b_step"]

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=dev) / shape[-2] ** 0.5).to(BF16)

        hidden = Hq * D
        self.embed = torch.randn(V, hidden, generator=g, device=dev).to(BF16)
        self.w_qkv, self.w_out, self.w_head = weight(hidden, (Hq + 2 * Hk) * D), weight(hidden, hidden), weight(hidden, V)
        self.freq, self.rope_scale = vs.rope_frequencies(D, 10000.0, scaling="ramp", factor=4.0, trained=64)

        # the cache: the prefix's pages are set aside, the others are in the ring
        own = -(-room // page_size)
        self.prefix_pages = -(-prefix // page_size)
        n_pages = self.prefix_pages + R * own
        self.k_cache = torch.zeros(n_pages, page_size, Hk, D, dtype=BF16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.cache = vs.cache_tables(R, n_pages, page_size, own, dev)
        self.cache["ring_pos"][0] = self.prefix_pages
        self.prefix_tokens = torch.randint(0, V, (prefix,), generator=g, device=dev, dtype=I32)
        self.prefix_table = torch.arange(self.prefix_pages, dtype=I32, device=dev)[None]
        self.prefix_len = torch.tensor([prefix], dtype=I32, device=dev)
        self.group_off = torch.tensor([0, R], dtype=I32, device=dev)
        self.pos_base = torch.full((R,), prefix, dtype=I32, device=dev)

        # a full cache's tokens and the last emitted one; the last column takes what a round does not emit
        self.tokens = torch.zeros(R, own * page_size + 2, dtype=I32, device=dev)
        self.tokens[:, :prompt] = torch.randint(0, V, (R, prompt), generator=g, device=dev, dtype=I32)
        self.prompt_len = torch.full((R,), prompt, dtype=I32, device=dev)
        self.length = self.prompt_len.clone()
        self.x0 = self.tokens[:, prompt - 1].contiguous()
        self.penalty = dict(repetition=torch.full((R,), 1.1, device=dev), frequency=torch.full((R,), 0.3, device=dev),
                            presence=torch.full((R,), 0.2, device=dev))
        allowed = torch.randint(-(1 << 31), 1 << 31, (1, -(-V // 32)), generator=g, device=dev).to(I32)
        self.mask = allowed | 1  # every 32nd token is always allowed
        self.mask_row = torch.zeros(R * (gamma + 1), dtype=I32, device=dev)
        self.status = torch.zeros(1, dtype=I32, device=dev)

        # the prefix's keys and values, then the prompts' (all but their last tokens)
        at = torch.arange(prefix, dtype=I32, device=dev)
        self._project(self.prefix_tokens, at, at)
        n = prompt - 1
        off = torch.arange(R + 1, dtype=I32, device=dev) * n
        r = vs.cache_reserve(self.cache, off, R * n, pos_base=self.pos_base, status=self.status)
        self._project(self.tokens[:, :n].reshape(-1), r["position"], r["slot"])
        self.cache.update(vs.cache_commit(self.cache, r, torch.full((R,), n, dtype=I32, device=dev), status=self.status))

    def _project(self, tokens, position, slot):
        """Embeddings of the rows and their turned queries (zeros where a row has no position); keys and values
        go to the cache."""
        h = self.embed[tokens.long()]
        qkv = (h @ self.w_qkv).view(len(h), self.Hq + 2 * self.Hk, self.D)
        q = vs.rope_cache(qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hk], qkv[:, self.Hq + self.Hk:], self.freq, position,
                          slot, self.k_cache, self.v_cache, scale=self.rope_scale, status=self.status,
                          q_out=torch.zeros(len(h), self.Hq, self.D, dtype=BF16, device=h.device))
        return h, q

    def round(self, seed: int) -> dict:
        R, G1 = self.R, self.gamma + 1
        rows = R * G1
        self.draft_in.x0 = self.x0
        d = vs.draft_sample(self.draft_in, seed, status=self.status)
        s = vs.schedule(d["a"], self.sps, self.b_lo, self.b_step, self.wl.K, status=self.status)
        r = vs.cache_reserve(self.cache, s["row_off"], rows, pos_base=self.pos_base, status=self.status)
        # the rows' tokens: the last emitted one, then the draft
        req = r["request"].clamp(min=0).long()
        j = torch.arange(rows, device=req.device) - s["row_off"].long()[req]
        fed = torch.cat([self.x0[:, None], d["x"]], 1)[req, j.clamp(0, self.gamma)]
        h, q = self._project(fed, r["position"], r["slot"])
        o = vs.prefix_attention(q, self.k_cache, self.v_cache, s["row_off"], r["new_len"], self.cache["block_table"],
                                group_off=self.group_off, prefix_len=self.prefix_len, prefix_table=self.prefix_table, status=self.status)
        raw = ((h + o.flatten(1) @ self.w_out) @ self.w_head).float()
        logits = vs.adjust_logits(raw, self.tokens, self.prompt_len, self.length, row_off=s["row_off"], x=d["x"], mask=self.mask,
                                  mask_row=self.mask_row, status=self.status, **self.penalty)
        v = vs.verify(vs.VERIFY_SAMPLE, logits, s["row_off"], s["ell"], d["x"], seed, q_tok=d["q_tok"], lse_q=d["lse_q"],
                      draft=self.draft_in, status=self.status)
        # a refused request (its new rows, one at least, are not in the cache) emits nothing
        n_out = torch.where(r["new_len"] > self.cache["kv_len"], v["n_out"], 0)
        self.cache.update(vs.cache_commit(self.cache, r, n_out, status=self.status))
        # emitted tokens join the history
        i = torch.arange(G1, device=req.device)[None, :]
        to = torch.where(i < n_out[:, None], self.length[:, None] + i, self.tokens.shape[1] - 1).long()
        self.tokens.scatter_(1, to, v["out_tok"].clamp(min=0))
        self.length = self.length + n_out
        last = v["out_tok"].gather(1, (n_out[:, None] - 1).clamp(min=0).long())[:, 0]
        self.x0 = torch.where(n_out > 0, last, self.x0)
        return {"fed": fed, "reserved": r, "sched": s, "draft": d, "raw": raw, "logits": logits, "verify": v}


def main() -> None:
    rounds = int(sys.argv[1]) if len(sys.argv) > 1 else 20
    step = TargetStep()
    for t in range(rounds):
        step.round(t)
    torch.cuda.synchronize()
    made = (step.length - step.prompt_len).tolist()
    free = int((step.cache["ring_pos"][1] - step.cache["ring_pos"][0]).item())
    print(f"{rounds} rounds, tokens made per request {made}, free pages {free}, status {step.status.item():#x}")


if __name__ == "__main__":
    main()
