"""Cases, plain forms and exact values of the operators around a verification round of the target model.

One round of speculative decoding asks the target model for 1 + l_r rows of logits for each request r. Four operators
stand between the schedule and the verifier:

  tables     the rows' positions, requests and cache slots from the requests' lengths, with pages taken from a ring of free
             ones, and after the verification the kept lengths and the pages given back
  rope       rotary positions on queries and keys, the keys and values written to their slots of the paged cache
  attention  the rows' attention over a prefix that many requests share and over each request's own pages
  logits     penalties for repeated tokens, biases and grammar masks on the packed rows of logits

`run` computes each in elementary torch operations, or through the public calls of verify_sampling_gb300 where `own` is true.
Lengths are a fixed collection for a case, dealt to the requests in an order that the seed gives, so that every seed
means the same work.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one request of a chat decoded alone: launch latency
        {"name": "tables one", "op": "tables", "R": 1, "new": 1, "kv": 700, "page": 16, "pad": False},
        # a round of the 512-request workload: up to 1 + 11 rows a request, outputs of a fixed capacity for graphs
        {"name": "tables round", "op": "tables", "R": 512, "new": 12, "kv": 8192, "page": 16, "pad": True},
        # prompts taken in: thousands of new tokens a request
        {"name": "tables prompts", "op": "tables", "R": 250, "new": 4000, "kv": 2000, "page": 64, "pad": False},
        # one token in 32 bits
        {"name": "rope one", "op": "rope", "dtype": "f32", "rows": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "interleaved": False,
         "far": 5000, "scaled": False, "page": 16},
        # a round's rows from one packed projection
        {"name": "rope round", "op": "rope", "dtype": "bf16", "rows": 2560, "Hq": 64, "Hk": 8, "D": 128, "rot": 128, "interleaved": False,
         "far": 32768, "scaled": False, "page": 64},
        # long prompts at far positions, pairs side by side, half of the head, scaled
        {"name": "rope prompts", "op": "rope", "dtype": "bf16", "rows": 40001, "Hq": 32, "Hk": 4, "D": 128, "rot": 64, "interleaved": True,
         "far": 1000000, "scaled": True, "page": 32},
        # one long conversation: few rows, a long axis
        {"name": "attention one", "op": "attention", "dtype": "bf16", "R": 1, "new": 1, "own": 20001, "groups": 0, "prefix": 0,
         "Hq": 32, "Hk": 8, "D": 128, "page": 16},
        # a small model in 32 bits, heads of an odd size
        {"name": "attention f32", "op": "attention", "dtype": "f32", "R": 9, "new": 5, "own": 333, "groups": 2, "prefix": 500,
         "Hq": 12, "Hk": 4, "D": 80, "page": 16},
        # a round of 256 requests behind one long system prompt
        {"name": "attention round", "op": "attention", "dtype": "bf16", "R": 256, "new": 12, "own": 2048, "groups": 1, "prefix": 16384,
         "Hq": 64, "Hk": 8, "D": 128, "page": 64},
        # one row of one request
        {"name": "logits one", "op": "logits", "dtype": "f32", "R": 1, "new": 1, "V": 129280, "hist": 700, "bias": 8, "masks": 1},
        # an odd vocabulary in 16 bits
        {"name": "logits odd", "op": "logits", "dtype": "bf16", "R": 96, "new": 9, "V": 50257, "hist": 2000, "bias": 300, "masks": 40},
        # a round of the 512-request workload
        {"name": "logits round", "op": "logits", "dtype": "f32", "R": 512, "new": 9, "V": 129280, "hist": 4000, "bias": 100, "masks": 600},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "attention", "attention", "logits"])
    if op == "tables":
        return {"op": op, "R": _log(rng, 1, 700), "new": _log(rng, 1, 1400), "kv": _log(rng, 1, 9000),
                "page": rng.choice([1, 8, 16, 24, 32, 64, 128, 256]), "pad": rng.random() < 0.5}
    if op == "rope":
        hk = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([48, 64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        hq = hk * rng.randint(1, 8)
        return {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16"]), "rows": _log(rng, 1, 40000 * 128 // ((hq + 2 * hk) * d // 20 + 128)),
                "Hq": hq, "Hk": hk, "D": d, "rot": rot, "interleaved": rng.random() < 0.5, "far": _log(rng, 10, 8000000),
                "scaled": rng.random() < 0.5, "page": rng.choice([1, 16, 24, 64])}
    if op == "attention":
        f32 = rng.random() < 0.25
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4, 5, 8])
        d = rng.choice([16, 40, 80, 128, 256]) if f32 else rng.choice([64, 128, 128])
        r = _log(rng, 1, 40 if f32 else 200)
        n = _log(rng, 1, 6 if f32 else 14)
        g = rng.choice([0, 1, 1, min(r, 3)])
        return {"op": op, "dtype": "f32" if f32 else "bf16", "R": r, "new": n, "own": _log(rng, n, 700 if f32 else 4000 if r < 64 else 1500),
                "groups": g, "prefix": _log(rng, 1, 1500 if f32 else 12000) if g else 0, "Hq": hq, "Hk": hk, "D": d,
                "page": rng.choice([8, 16, 24, 64]) if f32 else rng.choice([16, 32, 64, 128, 256])}
    return {"op": op, "dtype": rng.choice(["f32", "bf16"]), "R": _log(rng, 1, 400), "new": _log(rng, 1, 9),
            "V": rng.choice([_log(rng, 1000, 150000), 32000, 50257, 129280, 151936]), "hist": _log(rng, 1, 9000),
            "bias": rng.choice([0, 1, 50, 300]), "masks": rng.choice([0, 1, 30, 300])}


def _spread(n, lo, hi, salt):
    """n whole numbers of [lo, hi], the same ones for the same arguments."""
    return np.random.RandomState(salt + 7 * n + hi).randint(lo, hi + 1, n)


def _lengths(case):
    """New tokens and own cached tokens (the new ones among them) of each request, in no order yet."""
    R, new = case["R"], case["new"]
    n = _spread(R, 1, new, 1)
    if case["op"] == "logits":
        return n, _spread(R, 1, case["hist"], 2)
    if case["op"] == "attention":
        kv = np.maximum(_spread(R, 1, case["own"], 3), n) if R > 1 else np.array([case["own"]])
        return np.minimum(n, kv), kv
    return (n, _spread(R, 0, case["kv"], 4)) if R > 1 else (np.array([new]), np.array([case["kv"]]))


def _groups(case):
    """First request of each group and each prefix's length."""
    G, R = case["groups"], case["R"]
    off = np.linspace(0, R, G + 1).round().astype(np.int64)
    lens = np.maximum(1, case["prefix"] - np.arange(G) * (case["prefix"] // 5))
    return off, lens


# ------------------------------------------------------------------ inputs --
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed * 1000003 + 17)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _row_off(n):
    return _i32(np.concatenate([[0], np.cumsum(n)]))


def _deal(pages, width, perm):
    """Page tables [len(pages), width] that deal out the pages of `perm` in turn; -1 past the end."""
    col = np.arange(width)[None, :]
    start = np.cumsum(pages) - pages
    at = np.where(col < pages[:, None], start[:, None] + col, 0)
    return _i32(np.where(col < pages[:, None], perm[at], -1))


def prepare(case, seed):
    return {"tables": _tables_state, "rope": _rope_state, "attention": _attention_state, "logits": _logits_state}[case["op"]](dict(case), seed)


def _tables_state(case, seed):
    r = np.random.RandomState(seed % (1 << 31))
    n, kv = _lengths(case)
    order = r.permutation(case["R"])
    n, kv, P = n[order], kv[order], case["page"]
    have, want = -(-kv // P), -(-(kv + n) // P)
    n_pages = int(want.sum()) + 11
    perm = r.permutation(n_pages)
    width = int(want.max()) + 2
    free, head = perm[have.sum():], 5
    ring = np.full(n_pages, -1)
    ring[(head + np.arange(len(free))) % n_pages] = free
    keep = np.minimum(n, 1 + r.randint(0, case["new"], case["R"]))
    keep = np.where(r.rand(case["R"]) < 0.02, -1, keep)  # some requests end
    rows = case["R"] * case["new"] if case["pad"] else int(n.sum())
    return {"op": "tables", "P": P, "rows": rows, "row_off": _row_off(n), "keep": _i32(keep), "base": _i32(r.randint(0, 2000, case["R"])),
            "cache": {"kv_len": _i32(kv), "block_table": _deal(have, width, perm), "ring": _i32(ring),
                      "ring_pos": torch.tensor([head, head + len(free)], dtype=torch.int64, device="cuda"), "page_size": P}}


def _frequencies(case):
    rot = case["rot"]
    f = 1.0 / 10000.0 ** (np.arange(0, rot, 2, dtype=np.float64) / rot)
    return f / 8.0 if case["scaled"] else f


def _rope_state(case, seed):
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    rows, hq, hk, d = case["rows"], case["Hq"], case["Hk"], case["D"]
    dt = DTYPES[case["dtype"]]
    qkv = torch.randn(rows, hq + 2 * hk, d, generator=g, device="cuda").to(dt)  # one projection's output
    pages = -(-rows // case["page"]) + 3
    slot = torch.randperm(pages * case["page"], generator=g, device="cuda")[:rows].to(torch.int32)
    cache = [torch.zeros(pages, case["page"], hk, d, dtype=dt, device="cuda") for _ in range(2)]
    return {"op": "rope", "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:], "position": _i32(r.randint(0, case["far"], rows)),
            "slot": slot, "freq": torch.from_numpy(_frequencies(case)).cuda(), "scale": 1.1 if case["scaled"] else 1.0,
            "interleaved": case["interleaved"], "k_cache": cache[0], "v_cache": cache[1]}


def _attention_state(case, seed):
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    n, kv = _lengths(case)
    order = r.permutation(case["R"])
    n, kv, P, G = n[order], kv[order], case["page"], case["groups"]
    dt, hq, hk, d = DTYPES[case["dtype"]], case["Hq"], case["Hk"], case["D"]
    pages = -(-kv // P)
    goff, plen = _groups(case) if G else (np.zeros(1), np.zeros(0, np.int64))
    ppages = -(-plen // P)
    n_pages = int(pages.sum() + ppages.sum()) + 3
    perm = r.permutation(n_pages)
    rows = int(n.sum())
    k = torch.empty(n_pages, P, hk, d, dtype=dt, device="cuda")
    v = torch.empty_like(k)
    for t in (k, v):  # a tensor's normal numbers in parts, so that 32 bits of it are never whole on the card
        for part in t.view(-1).split(1 << 28):
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return {"op": "attention", "rows": rows, "nmax": int(n.max()), "kvmax": int(kv.max()), "pmax": int(plen.max()) if G else 0,
            "gmax": max(int(n[int(goff[i]):int(goff[i + 1])].sum()) for i in range(G)) if G else 0,
            "q": (2.0 * torch.randn(rows, hq, d, generator=g, device="cuda")).to(dt), "k_cache": k, "v_cache": v, "row_off": _row_off(n), "kv_len": _i32(kv),
            "block_table": _deal(pages, int(pages.max()), perm), "scale": 1.0 / math.sqrt(d),
            "group_off": _i32(goff) if G else None, "prefix_len": _i32(plen) if G else None,
            "prefix_table": _deal(ppages, int(ppages.max()), perm[pages.sum():]) if G else None}


def _logits_state(case, seed):
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    n, hist = _lengths(case)
    order = r.permutation(case["R"])
    n, hist, R, V, nb = n[order], hist[order], case["R"], case["V"], min(case["bias"], case["V"])
    rows = int(n.sum())
    z = torch.empty(rows, V, dtype=DTYPES[case["dtype"]], device="cuda")
    for part in z.split(max(1, (1 << 28) // V)):
        part.copy_(4.0 * torch.randn(part.shape, generator=g, device="cuda"))
    # tokens of a text: few of them often
    tok = np.minimum(V - 1, (np.exp(r.rand(R, int(hist.max())) * math.log(V)) - 1).astype(np.int64)) * 7919 % V
    x = np.minimum(V - 1, (np.exp(r.rand(R, case["new"]) * math.log(V)) - 1).astype(np.int64)) * 7919 % V
    s = {"op": "logits", "rows": rows, "logits": z, "row_off": _row_off(n), "tokens": _i32(tok), "prompt_len": _i32(np.minimum(hist, r.randint(0, hist.max() + 1, R))),
         "length": _i32(hist), "x": _i32(x), "repetition": torch.from_numpy(r.uniform(1.0, 1.4, R).astype(np.float32)).cuda(),
         "frequency": torch.from_numpy(r.uniform(-0.2, 0.8, R).astype(np.float32)).cuda(),
         "presence": torch.from_numpy(r.uniform(-0.2, 0.8, R).astype(np.float32)).cuda(), "bias": None, "mask": None, "mask_row": None}
    if nb:
        step = max(1, V // nb)  # each request's biased tokens are different ones
        bt = (np.arange(nb)[None, :] * step + r.randint(0, step, (R, nb))) % V
        s["bias"] = (_i32(np.arange(R + 1) * nb), _i32(bt.reshape(-1)), torch.randn(R * nb, generator=g, device="cuda"))
    if case["masks"]:
        s["mask"] = torch.randint(-(1 << 31), 1 << 31, (case["masks"], -(-V // 32)), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        s["mask_row"] = _i32(np.where(np.arange(rows) % 3 == 2, -1, r.randint(0, case["masks"], rows)))
    return s


# --------------------------------------------------------------- the calls --
def run(s):
    if own:
        import verify_sampling_gb300 as vs
        return {"tables": _tables_own, "rope": _rope_own, "attention": _attention_own, "logits": _logits_own}[s["op"]](vs, s)
    return {"tables": _tables_plain, "rope": _rope_plain, "attention": _attention_plain, "logits": _logits_plain}[s["op"]](s)


def _tables_own(vs, s):
    # The commit writes to a second ring that the program keeps: returned pages may take the places of those that the
    # reserve took, and a round that is run again from its start has to find these.
    c = s["cache"]
    if "after" not in s:
        s["after"] = {**c, "ring": c["ring"].clone()}
    p = vs.cache_reserve(c, s["row_off"], s["rows"], pos_base=s["base"])
    d = vs.cache_commit(s["after"], p, s["keep"])
    return {"new_len": p["new_len"], "position": p["position"], "request": p["request"], "slot": p["slot"], "block_table": c["block_table"],
            "ring": s["after"]["ring"], "ring_pos": d["ring_pos"], "kv_len": d["kv_len"]}


def _rope_own(vs, s):
    q = vs.rope_cache(s["q"], s["k"], s["v"], s["freq"], s["position"], s["slot"], s["k_cache"], s["v_cache"], interleaved=s["interleaved"],
                      scale=s["scale"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attention_own(vs, s):
    out, lse = vs.prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["row_off"], s["kv_len"], s["block_table"], scale=s["scale"],
                                   group_off=s["group_off"], prefix_len=s["prefix_len"], prefix_table=s["prefix_table"], want_lse=True)
    return {"out": out, "lse": lse}


def _logits_own(vs, s):
    return vs.adjust_logits(s["logits"], s["tokens"], s["prompt_len"], s["length"], row_off=s["row_off"], x=s["x"], repetition=s["repetition"],
                            frequency=s["frequency"], presence=s["presence"], bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"])


# ------------------------------------------------------------- plain forms --
def _request_of(row_off, rows):
    """Request and place of each row; the request is R past the last row."""
    b = torch.arange(rows, device=row_off.device)
    r = torch.searchsorted(row_off[1:].long(), b, right=True)
    return r, b - row_off.long()[r.clamp(max=row_off.numel() - 1)]


def _tables_plain(s):
    c, P, rows = s["cache"], s["P"], s["rows"]
    kv, off, table, ring, pos = c["kv_len"].long(), s["row_off"].long(), c["block_table"].long(), c["ring"].long(), c["ring_pos"]
    n = off[1:] - off[:-1]
    have, want = (kv + P - 1) // P, (kv + n + P - 1) // P
    need = want - have
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    place = pos[0] + first[:, None] + (col - have[:, None])
    table = torch.where((col >= have[:, None]) & (col < want[:, None]), ring[place % ring.numel()], table)
    new_len = kv + n
    r, j = _request_of(s["row_off"], rows)
    real = r < n.numel()
    r = r.clamp(max=n.numel() - 1)
    at = torch.where(real, kv[r] + j, 0)
    slot = torch.where(real, table[r, at // P] * P + at % P, -1)
    position = torch.where(real, s["base"].long()[r] + at, -1)
    # after the verification: the kept tokens, the pages past them go back
    keep = s["keep"].long()
    kept = torch.where(keep < 0, 0, torch.minimum(kv + keep, new_len))
    stay = (kept + P - 1) // P
    back = want - stay
    to = pos[1] + (torch.cumsum(back, 0) - back)[:, None] + (col - stay[:, None])
    goes = (col >= stay[:, None]) & (col < want[:, None])
    at = torch.where(goes, to % ring.numel(), ring.numel())
    ring = torch.cat([ring, ring[:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:-1]
    moved = torch.stack([pos[0] + need.sum(), pos[1] + back.sum()])
    as32 = [t.to(torch.int32) for t in (new_len, position, torch.where(real, r, -1), slot, table, ring, kept)]
    return dict(zip(("new_len", "position", "request", "slot", "block_table", "ring", "kv_len"), as32), ring_pos=moved)


def _turned(x, cos, sin, rot, interleaved):
    x = x.float()
    t, rest = x[..., :rot], x[..., rot:]
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., :rot // 2], t[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    t = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([t, rest], -1)


def _rope_plain(s):
    rot = 2 * s["freq"].numel()
    angle = s["position"].double()[:, None] * s["freq"][None, :]  # 64 bits: far positions
    cos, sin = ((f(angle) * s["scale"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    q = _turned(s["q"], cos, sin, rot, s["interleaved"]).to(s["q"].dtype)
    k = _turned(s["k"], cos, sin, rot, s["interleaved"]).to(s["q"].dtype)
    slot = s["slot"].long()
    s["k_cache"].flatten(0, 1).index_copy_(0, slot, k)
    s["v_cache"].flatten(0, 1).index_copy_(0, slot, s["v"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _softmax_parts(q, k, v, scale, keep):
    """Maximum, sum and weighted values of q [N, M, Hq, D] against k, v [N, L, Hk, D] where keep [N, M, L]."""
    N, M, hq, d = q.shape
    hk = k.shape[2]
    q = q.reshape(N, M, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(N, hk, -1, d)  # a key's head with all its queries' heads
    z = (q @ k.permute(0, 2, 3, 1)).view(N, hk, hq // hk, M, -1) * scale
    z.masked_fill_(~keep[:, None, None], -torch.inf)
    m = z.amax(-1).clamp(min=-1e30)
    z.sub_(m[..., None]).exp_()
    o = (z.view(N, hk, -1, z.shape[-1]) @ v.permute(0, 2, 1, 3)).view(N, hk, hq // hk, M, d)
    return [t.permute(0, 3, 1, 2, *range(4, t.dim())).reshape(N, M, hq, *t.shape[4:]) for t in (m, z.sum(-1), o)]


def _gathered(cache, table, L):
    """[N, L, Hk, D] in 32 bits from pages; what a table does not name is nothing."""
    pages = cache[table.clamp(min=0).long()].flatten(1, 2)[:, :L].float()
    return pages


def _attention_plain(s):
    q, rows, R = s["q"].float(), s["rows"], s["kv_len"].numel()
    r, j = _request_of(s["row_off"], rows)
    n = (s["row_off"][1:] - s["row_off"][:-1]).long()
    kv = s["kv_len"].long()
    M, L = s["nmax"], s["kvmax"]
    padded = q.new_zeros(R, M, *q.shape[1:])
    padded[r, j] = q
    last = (kv - n)[:, None] + torch.arange(M, device=q.device)[None, :]
    keep = torch.arange(L, device=q.device)[None, None, :] <= last[..., None]
    m, l, o = [t[r, j] for t in _softmax_parts(padded, _gathered(s["k_cache"], s["block_table"], L), _gathered(s["v_cache"], s["block_table"], L), s["scale"], keep)]
    if s["prefix_len"] is not None:
        G, M, L = s["prefix_len"].numel(), s["gmax"], s["pmax"]
        g = torch.searchsorted(s["group_off"][1:].contiguous(), r.to(torch.int32), right=True)
        i = torch.arange(rows, device=q.device) - s["row_off"].long()[s["group_off"].long()[g]]
        padded = q.new_zeros(G, M, *q.shape[1:])
        padded[g, i] = q
        keep = (torch.arange(L, device=q.device)[None, :] < s["prefix_len"].long()[:, None])[:, None, :].expand(G, M, L)
        m2, l2, o2 = [t[g, i] for t in _softmax_parts(padded, _gathered(s["k_cache"], s["prefix_table"], L), _gathered(s["v_cache"], s["prefix_table"], L), s["scale"], keep)]
        top = torch.maximum(m, m2)
        a, b = torch.exp(m - top), torch.exp(m2 - top)
        m, l, o = top, l * a + l2 * b, o * a[..., None] + o2 * b[..., None]
    return {"out": (o / l[..., None]).to(s["q"].dtype), "lse": m + torch.log(l)}


def _logits_plain(s):
    z, rows = s["logits"].float(), s["rows"]
    R, V = s["length"].numel(), z.shape[1]
    r, j = _request_of(s["row_off"], rows)
    tok = s["tokens"].long()
    at = torch.arange(tok.shape[1], device=z.device)[None, :]
    prompt, length = s["prompt_len"].long()[:, None], s["length"].long()[:, None]
    said = torch.zeros(R, V, device=z.device).scatter_add_(1, tok, ((at >= prompt) & (at < length)).float())
    asked = torch.zeros(R, V, device=z.device).scatter_add_(1, tok, ((at < prompt) & (at < length)).float())
    x = s["x"].long()[r]
    count = said[r].scatter_add_(1, x, (torch.arange(x.shape[1], device=z.device)[None, :] < j[:, None]).float())
    seen = (count > 0) | (asked[r] > 0)
    rep, freq, pres = (s[k][r][:, None] for k in ("repetition", "frequency", "presence"))
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - freq * count - pres * (count > 0)
    if s["bias"] is not None:
        off, bt, bv = s["bias"]
        bias = torch.zeros(R, V, device=z.device).scatter_(1, bt.view(R, -1).long(), bv.view(R, -1))
        z = z + bias[r]
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=z.device, dtype=torch.int32)) & 1
        allowed = bits.flatten(1)[:, :V].bool()
        row = s["mask_row"].long()
        z = z.masked_fill((row >= 0)[:, None] & ~allowed[row.clamp(min=0)], -torch.inf)
    return z.to(s["logits"].dtype)


# ------------------------------------------------------------ in 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(s)
    if case["op"] == "attention":
        return _attention_exact(s)
    if case["op"] == "logits":
        return _logits_exact(s)
    return None  # whole numbers only


def _rope_exact(s):
    half = s["freq"].numel()
    angle = torch.outer(s["position"].double(), s["freq"].double())
    turn = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, None]

    def turned(x):
        y = x.double()
        t = y[..., :2 * half]
        z = torch.complex(t[..., 0::2].contiguous(), t[..., 1::2].contiguous()) if s["interleaved"] else torch.complex(t[..., :half].contiguous(), t[..., half:].contiguous())
        z = z * turn
        if s["interleaved"]:
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        else:
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    out = {"q": turned(s["q"].clone())}
    for name, x in (("k_cache", turned(s["k"].clone())), ("v_cache", s["v"].double())):
        c = s[name].double()
        c.view(-1, *c.shape[2:])[s["slot"].long()] = x
        out[name] = c
    return out


def _attention_exact(s):
    hq, d = s["q"].shape[1:]
    off, kv = s["row_off"].tolist(), s["kv_len"].tolist()
    goff = s["group_off"].tolist() if s["group_off"] is not None else []
    k_all, v_all = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    hk, P = k_all.shape[1], s["k_cache"].shape[1]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["rows"], hq, dtype=torch.float64, device="cuda")

    def slots(table, n):
        at = torch.arange(n, device="cuda")
        return table.long()[at // P] * P + at % P

    for r in range(len(kv)):
        n = off[r + 1] - off[r]
        at, shared = slots(s["block_table"][r], kv[r]), 0
        for g in range(len(goff) - 1):
            if goff[g] <= r < goff[g + 1]:
                shared = int(s["prefix_len"][g])
                at = torch.cat([slots(s["prefix_table"][g], shared), at])
        k, v = k_all[at].double(), v_all[at].double()
        q = s["q"][off[r]:off[r + 1]].double().view(n, hk, hq // hk, d)
        z = torch.einsum("nhgd,lhd->hgnl", q, k) * s["scale"]
        last = shared + kv[r] - n + torch.arange(n, device="cuda")
        z = z.masked_fill(torch.arange(len(at), device="cuda")[None, :] > last[:, None], -torch.inf)
        out[off[r]:off[r + 1]] = torch.einsum("hgnl,lhd->nhgd", torch.softmax(z, -1), v).reshape(n, hq, d)
        lse[off[r]:off[r + 1]] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(n, hq)
    return {"out": out, "lse": lse}


def _logits_exact(s):
    out = s["logits"].double()
    off, length, prompt = s["row_off"].tolist(), s["length"].tolist(), s["prompt_len"].tolist()
    V = out.shape[1]
    masks = s["mask_row"].tolist() if s["mask_row"] is not None else None
    bit = torch.arange(V, device="cuda")
    for r in range(len(length)):
        asked = torch.bincount(s["tokens"][r, :min(prompt[r], length[r])].long(), minlength=V) > 0
        said = torch.bincount(s["tokens"][r, min(prompt[r], length[r]):length[r]].long(), minlength=V).double()
        rep, freq, pres = (s[k][r].double() for k in ("repetition", "frequency", "presence"))
        for b in range(off[r], off[r + 1]):
            z = out[b]
            seen = asked | (said > 0)
            z[seen] = torch.where(z[seen] > 0, z[seen] / rep, z[seen] * rep)
            z -= freq * said + pres * (said > 0)
            if s["bias"] is not None:
                lo, hi = (int(t) for t in s["bias"][0][r:r + 2])
                z[s["bias"][1][lo:hi].long()] += s["bias"][2][lo:hi].double()
            if masks is not None and masks[b] >= 0:
                z[(s["mask"][masks[b]][bit // 32] >> (bit % 32).to(torch.int32)) & 1 == 0] = -torch.inf
            said[s["x"][r, b - off[r]].long()] += 1
    return out


# --------------------------------------------------------------- the work --
def work(case):
    if case["op"] == "rope":
        es, n = DTYPES[case["dtype"]].itemsize, case["rows"]
        heads, turned = case["Hq"] + 2 * case["Hk"], case["Hq"] + case["Hk"]
        return {"bytes": 2 * n * heads * case["D"] * es + 8 * n + 4 * case["rot"], "flops": n * turned * case["rot"] * 3}
    n, other = _lengths(case)
    rows, R = int(n.sum()), case["R"]
    if case["op"] == "tables":
        P = case["page"]
        out = R * case["new"] if case["pad"] else rows
        taken = int((-(-(other + n) // P) - -(-other // P)).sum())
        # lengths and offsets in, three values a row out, each page taken read and written, two lengths out; about half of the pages go back
        return {"bytes": 4 * (4 * R + 3 * out + 2 * taken + 2 * R + taken), "flops": 4 * out}
    if case["op"] == "attention":
        es, d, hk, hq = DTYPES[case["dtype"]].itemsize, case["D"], case["Hk"], case["Hq"]
        keys = int((n * other - n * (n - 1) // 2).sum())
        shared = 0
        if case["groups"]:
            goff, plen = _groups(case)
            shared = int(plen.sum())
            per = (plen * np.diff(goff)).sum() / R  # each request as likely in each group
            keys += int(rows * per)
        return {"bytes": 2 * rows * hq * d * es + 4 * rows * hq + 2 * (int(other.sum()) + shared) * hk * d * es, "flops": 4 * keys * hq * d}
    V, es = case["V"], DTYPES[case["dtype"]].itemsize
    masked = min(case["masks"], rows) if case["masks"] else 0
    return {"bytes": 2 * rows * V * es + masked * (V // 8) + 4 * int(other.sum()) + 8 * R * case["bias"], "flops": 2 * rows * V}
