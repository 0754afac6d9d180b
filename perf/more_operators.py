"""Cases, plain forms and exact values of head norms with rotary positions, and of a paged cache held in 4 bits.

  norm     each head's queries and keys divided by their root mean square, turned by their positions, keys and values
           written to their slots of the paged cache
  append   the same (with or without the norms) into a cache held in 4 bits, and the written slots read back as values
  attend   attention of packed rows over such a cache: a prefix that many requests share, and each request's own pages

The cache in 4 bits: a head's elements in groups of 32, a group's element j in nibble j of its 16 bytes (the low one of a byte
first) and a byte b for its scale s = 2^((b >> 3) - 20) (1 + (b & 7) / 8); an element is s (nibble - 8). Data lie as
[pages, key heads, groups, tokens of a page, 16], scales as [pages, key heads, tokens of a page, groups].

`run` computes each in elementary torch operations, or through the public calls of verify_sampling_gb300 where `own` is true.
Lengths are a fixed collection for a case, dealt to the requests in an order that the seed gives, so that every seed
means the same work.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GROUP = 32
EPS = 1e-6


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one token in 32 bits: launch latency
        {"name": "norm one", "op": "norm", "dtype": "f32", "rows": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "interleaved": False,
         "far": 5000, "scaled": False, "page": 16},
        # the rows of a round of several hundred requests, parts of one projection
        {"name": "norm round", "op": "norm", "dtype": "bf16", "rows": 2560, "Hq": 64, "Hk": 8, "D": 128, "rot": 128, "interleaved": False,
         "far": 32768, "scaled": False, "page": 64},
        # long prompts at far positions, pairs side by side, half of the head, scaled
        {"name": "norm prompts", "op": "norm", "dtype": "bf16", "rows": 40001, "Hq": 32, "Hk": 4, "D": 128, "rot": 64, "interleaved": True,
         "far": 1000000, "scaled": True, "page": 32},
        # one token of a chat decoded alone
        {"name": "append one", "op": "append", "dtype": "bf16", "rows": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "interleaved": False,
         "far": 5000, "scaled": False, "page": 16, "norm": True},
        # a round's rows
        {"name": "append round", "op": "append", "dtype": "bf16", "rows": 2560, "Hq": 64, "Hk": 8, "D": 128, "rot": 128, "interleaved": False,
         "far": 32768, "scaled": False, "page": 64, "norm": True},
        # long prompts of a model without norms, small heads, a part of them turned
        {"name": "append prompts", "op": "append", "dtype": "bf16", "rows": 30011, "Hq": 16, "Hk": 8, "D": 64, "rot": 32, "interleaved": False,
         "far": 100000, "scaled": True, "page": 16, "norm": False},
        # one long conversation: one row, a long axis
        {"name": "attend one", "op": "attend", "dtype": "bf16", "R": 1, "new": 1, "own": 20001, "groups": 0, "prefix": 0,
         "Hq": 32, "Hk": 8, "D": 128, "page": 16},
        # a small model in 32 bits, heads of an odd number of groups
        {"name": "attend f32", "op": "attend", "dtype": "f32", "R": 9, "new": 5, "own": 333, "groups": 2, "prefix": 500,
         "Hq": 12, "Hk": 4, "D": 96, "page": 16},
        # small heads, a few rows a request, an odd number of requests
        {"name": "attend small", "op": "attend", "dtype": "bf16", "R": 101, "new": 4, "own": 3000, "groups": 0, "prefix": 0,
         "Hq": 24, "Hk": 8, "D": 64, "page": 32},
        # 256 requests decoded token by token
        {"name": "attend decode", "op": "attend", "dtype": "bf16", "R": 256, "new": 1, "own": 8192, "groups": 0, "prefix": 0,
         "Hq": 64, "Hk": 8, "D": 128, "page": 64},
        # a round of 256 requests behind one long system prompt
        {"name": "attend round", "op": "attend", "dtype": "bf16", "R": 256, "new": 12, "own": 2048, "groups": 1, "prefix": 16384,
         "Hq": 64, "Hk": 8, "D": 128, "page": 64},
        # a few prompts taken in behind what is in the cache
        {"name": "attend prompts", "op": "attend", "dtype": "bf16", "R": 4, "new": 3000, "own": 6000, "groups": 0, "prefix": 0,
         "Hq": 32, "Hk": 8, "D": 128, "page": 16},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend"])
    if op != "attend":
        hk = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 64, 96, 128, 128, 192, 256]) if op == "append" else rng.choice([48, 64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        hq = hk * rng.randint(1, 8)
        case = {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16"]), "rows": _log(rng, 1, 40000 * 128 // ((hq + 2 * hk) * d // 20 + 128)),
                "Hq": hq, "Hk": hk, "D": d, "rot": rot, "interleaved": rng.random() < 0.5, "far": _log(rng, 10, 8000000),
                "scaled": rng.random() < 0.5, "page": rng.choice([1, 16, 24, 64])}
        return {**case, "norm": rng.random() < 0.7} if op == "append" else case
    f32 = rng.random() < 0.25
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 8])
    d = rng.choice([32, 64, 96, 128, 256]) if f32 else rng.choice([64, 128, 128])
    r = _log(rng, 1, 40 if f32 else 250)
    n = _log(rng, 1, 6) if f32 else _log(rng, 1, 14) if r > 8 else _log(rng, 1, 1000)
    g = rng.choice([0, 0, 1, min(r, 3)])
    return {"op": op, "dtype": "f32" if f32 else "bf16", "R": r, "new": n,
            "own": max(n, _log(rng, n, 700 if f32 else 6000 if r < 64 else 3000)),
            "groups": g, "prefix": _log(rng, 1, 1500 if f32 else 12000) if g else 0, "Hq": hq, "Hk": hk, "D": d,
            "page": rng.choice([8, 16, 24, 64]) if f32 else rng.choice([16, 32, 64, 128, 256])}


def _spread(n, lo, hi, salt):
    """n whole numbers of [lo, hi], the same ones for the same arguments."""
    return np.random.RandomState(salt + 7 * n + hi).randint(lo, hi + 1, n)


def _lengths(case):
    """New tokens and own cached tokens (the new ones among them) of each request, in no order yet."""
    R, new = case["R"], case["new"]
    n = _spread(R, 1, new, 1) if R > 1 else np.array([new])
    kv = np.maximum(_spread(R, 1, case["own"], 3), n) if R > 1 else np.array([case["own"]])
    return np.minimum(n, kv), kv


def _groups(case):
    """First request of each group and each prefix's length."""
    G, R = case["groups"], case["R"]
    off = np.linspace(0, R, G + 1).round().astype(np.int64)
    lens = np.maximum(1, case["prefix"] - np.arange(G) * (case["prefix"] // 5))
    return off, lens


# -------------------------------------------------------------- in 4 bits ---
def _scale(code):
    """Scales of code bytes (whole numbers), exactly."""
    c = code.to(torch.int32)
    return ((c << 20) + (107 << 23)).view(torch.float32)


def _coded(x):
    """Scale bytes [..., groups] and nibbles [..., groups, 32] of values x [..., D], in 32 bits."""
    x = x.unflatten(-1, (-1, GROUP))
    t = (x.abs().amax(-1) / 7.0).contiguous()
    code = (((t.view(torch.int32) + (1 << 19)) >> 20) - 107 * 8).clamp(0, 255)  # to four significant bits, halves up
    n = torch.round(x / _scale(code)[..., None]).clamp(-7, 7)
    return code.to(torch.uint8), (n + 8).to(torch.uint8)


def _values(code, nibble):
    """What scale bytes [..., groups] and nibbles [..., groups, 32] stand for: [..., D]."""
    return ((nibble.float() - 8.0) * _scale(code)[..., None]).flatten(-2)


def _nibbles(data):
    """Nibbles [..., 32] of bytes [..., 16]."""
    return torch.stack([data & 15, data >> 4], -1).flatten(-2)


# ------------------------------------------------------------------ inputs --
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed * 1000003 + 17)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _deal(pages, width, perm):
    """Page tables [len(pages), width] that deal out the pages of `perm` in turn; -1 past the end."""
    col = np.arange(width)[None, :]
    start = np.cumsum(pages) - pages
    at = np.where(col < pages[:, None], start[:, None] + col, 0)
    return _i32(np.where(col < pages[:, None], perm[at], -1))


def prepare(case, seed):
    return _attend_state(dict(case), seed) if case["op"] == "attend" else _rows_state(dict(case), seed)


def _rows_state(case, seed):
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    rows, hq, hk, d, P = case["rows"], case["Hq"], case["Hk"], case["D"], case["page"]
    dt = DTYPES[case["dtype"]]
    qkv = torch.randn(rows, hq + 2 * hk, d, generator=g, device="cuda")  # one projection's output
    if case["op"] == "append":
        # Keys of a flat spread: 32 and 64 bits may put a key next to the border of two stored values on either side, and
        # a step of the stored values is then no more than about a third of what keys usually are.
        qkv[:, hq:hq + hk] = 3.0 * torch.rand(rows, hk, d, generator=g, device="cuda") - 1.5
    qkv = qkv.to(dt)
    pages = -(-rows // P) + 3
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:rows].to(torch.int32)
    freq = 1.0 / 10000.0 ** (np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
    s = {"op": case["op"], "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:], "position": _i32(r.randint(0, case["far"], rows)),
         "slot": slot, "freq": torch.from_numpy(freq / 8.0 if case["scaled"] else freq).cuda(), "scale": 1.1 if case["scaled"] else 1.0,
         "interleaved": case["interleaved"], "q_weight": None, "k_weight": None}
    if case.get("norm", True):
        s["q_weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["k_weight"] = 0.95 + 0.1 * torch.rand(d, generator=g, device="cuda")
    if case["op"] == "norm":
        s["k_cache"], s["v_cache"] = (torch.zeros(pages, P, hk, d, dtype=dt, device="cuda") for _ in range(2))
    else:
        s["k_cache"], s["v_cache"] = ((torch.zeros(pages, hk, d // GROUP, P, 16, dtype=torch.uint8, device="cuda"),
                                       torch.zeros(pages, hk, P, d // GROUP, dtype=torch.uint8, device="cuda")) for _ in range(2))
    return s


def _attend_state(case, seed):
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
    caches = []
    for _ in range(2):
        data = torch.empty(n_pages, hk, d // GROUP, P, 16, dtype=torch.uint8, device="cuda")
        scale = torch.empty(n_pages, hk, P, d // GROUP, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (hk * P * d))
        for a in range(0, n_pages, step):  # normal numbers in parts, so that 32 bits of a cache are never whole on the card
            b = min(n_pages, a + step)
            code, nib = _coded(torch.randn(b - a, hk, P, d, generator=g, device="cuda"))
            scale[a:b] = code
            data[a:b] = (nib[..., 0::2] | (nib[..., 1::2] << 4)).transpose(2, 3)
        caches.append((data, scale))
    return {"op": "attend", "rows": rows, "nmax": int(n.max()), "kvmax": int(kv.max()), "pmax": int(plen.max()) if G else 0,
            "gmax": max(int(n[int(goff[i]):int(goff[i + 1])].sum()) for i in range(G)) if G else 0,
            "q": (2.0 * torch.randn(rows, hq, d, generator=g, device="cuda")).to(dt), "k_cache": caches[0], "v_cache": caches[1],
            "row_off": _i32(np.concatenate([[0], np.cumsum(n)])), "kv_len": _i32(kv),
            "block_table": _deal(pages, int(pages.max()), perm), "scale": 1.0 / math.sqrt(d),
            "group_off": _i32(goff) if G else None, "prefix_len": _i32(plen) if G else None,
            "prefix_table": _deal(ppages, int(ppages.max()), perm[pages.sum():]) if G else None}


# --------------------------------------------------------------- the calls --
def run(s):
    if own:
        import verify_sampling_gb300 as vs
        return _attend_own(vs, s) if s["op"] == "attend" else _rows_own(vs, s)
    return _attend_plain(s) if s["op"] == "attend" else _rows_plain(s)


def _rows_own(vs, s):
    q = vs.norm_rope_cache(s["q"], s["k"], s["v"], s["freq"], s["position"], s["slot"], s["k_cache"], s["v_cache"],
                           q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"], scale=s["scale"])
    if s["op"] == "norm":
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    k, v = vs.cache_read_packed(s["k_cache"], s["v_cache"], s["slot"])
    return {"q": q, "k": k, "v": v}


def _attend_own(vs, s):
    out, lse = vs.prefix_attention_packed(s["q"], s["k_cache"], s["v_cache"], s["row_off"], s["kv_len"], s["block_table"], scale=s["scale"],
                                        group_off=s["group_off"], prefix_len=s["prefix_len"], prefix_table=s["prefix_table"], want_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------- plain forms --
def _normed(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)


def _turned(x, cos, sin, rot, interleaved):
    t, rest = x[..., :rot], x[..., rot:]
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., :rot // 2], t[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    t = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([t, rest], -1)


def _rows_plain(s):
    rot = 2 * s["freq"].numel()
    angle = s["position"].double()[:, None] * s["freq"][None, :]  # 64 bits: far positions
    cos, sin = ((f(angle) * s["scale"])[:, None, :] for f in (torch.cos, torch.sin))
    q = _turned(_normed(s["q"].float(), s["q_weight"]), cos.float(), sin.float(), rot, s["interleaved"]).to(s["q"].dtype)
    slot = s["slot"].long()
    if s["op"] == "norm":
        k = _turned(_normed(s["k"].float(), s["k_weight"]), cos.float(), sin.float(), rot, s["interleaved"])
        s["k_cache"].flatten(0, 1).index_copy_(0, slot, k.to(s["q"].dtype))
        s["v_cache"].flatten(0, 1).index_copy_(0, slot, s["v"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    # 64 bits up to the coding: values next to the border of two stored ones
    k = _turned(_normed(s["k"].double(), s["k_weight"]), cos, sin, rot, s["interleaved"]).float()
    out, P = {"q": q}, s["k_cache"][1].shape[2]
    for name, cache, x in (("k", s["k_cache"], k), ("v", s["v_cache"], s["v"].float())):
        code, nib = _coded(x)
        cache[1][slot // P, :, slot % P] = code
        cache[0][slot // P, :, :, slot % P] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        out[name] = _values(code, nib).to(torch.bfloat16)  # exact: seven significant bits at most
    return out


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
    """Values [N, L, Hk, D] in 32 bits from pages; what a table does not name is nothing."""
    page = table.clamp(min=0).long()
    x = _values(cache[1][page], _nibbles(cache[0][page].transpose(3, 4)))  # [N, pages, Hk, P, D]
    return x.transpose(2, 3).flatten(1, 2)[:, :L]


def _request_of(row_off, rows):
    """Request and place of each row."""
    b = torch.arange(rows, device=row_off.device)
    r = torch.searchsorted(row_off[1:].long(), b, right=True)
    return r, b - row_off.long()[r]


def _attend_plain(s):
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


# ------------------------------------------------------------ in 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    return _attend_exact(s) if case["op"] == "attend" else _rows_exact(s)


def _rows_exact(s):
    half = s["freq"].numel()
    angle = torch.outer(s["position"].double(), s["freq"].double())
    turn = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, None]

    def turned(x, weight):
        y = x.double().clone()
        if weight is not None:
            y *= weight.double() / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / y.shape[-1] + EPS)
        t = y[..., :2 * half]
        z = torch.complex(t[..., 0::2].contiguous(), t[..., 1::2].contiguous()) if s["interleaved"] else torch.complex(t[..., :half].contiguous(), t[..., half:].contiguous())
        z = z * turn
        if s["interleaved"]:
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        else:
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    out = {"q": turned(s["q"], s["q_weight"])}
    if s["op"] == "norm":
        for name, x in (("k_cache", turned(s["k"], s["k_weight"])), ("v_cache", s["v"].double())):
            c = s[name].double()
            c.view(-1, *c.shape[2:])[s["slot"].long()] = x
            out[name] = c
        return out
    out["k"] = None  # a key next to a border is right on either side of it
    x = s["v"].double().unflatten(-1, (-1, GROUP))
    most = x.abs().amax(-1, keepdim=True) / 7.0
    e = torch.floor(torch.log2(most.clamp(min=2.0 ** -60)))
    e = e + (torch.exp2(e + 1) <= most).double() - (torch.exp2(e) > most).double()  # a logarithm next to a whole number
    step = torch.floor(most * torch.exp2(3 - e) + 0.5) * torch.exp2(e - 3)
    step = step.clamp(2.0 ** -20, 1.875 * 2.0 ** 11)
    out["v"] = (torch.round(x / step).clamp(-7, 7) * step).flatten(-2)
    return out


def _attend_exact(s):
    hq, d = s["q"].shape[1:]
    off, kv = s["row_off"].tolist(), s["kv_len"].tolist()
    goff = s["group_off"].tolist() if s["group_off"] is not None else []
    hk, P = s["k_cache"][1].shape[1:3]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["rows"], hq, dtype=torch.float64, device="cuda")
    bit = torch.arange(2, device="cuda") * 4

    def keys(cache, table, n):
        """[n, Hk, D] of a page table."""
        at = torch.arange(n, device="cuda")
        page, place = table.long()[at // P], at % P
        nib = ((cache[0][page, :, :, place][..., None].long() >> bit) & 15).flatten(3)
        code = cache[1][page, :, place].long()
        step = torch.exp2((code // 8 - 20).double()) * (1 + (code % 8).double() / 8)
        return ((nib - 8).double() * step[..., None]).flatten(2)

    shared = {}
    for r in range(len(kv)):
        n = off[r + 1] - off[r]
        k, v = (keys(s[c], s["block_table"][r], kv[r]) for c in ("k_cache", "v_cache"))
        before = 0
        for g in range(len(goff) - 1):
            if goff[g] <= r < goff[g + 1]:
                before = int(s["prefix_len"][g])
                if g not in shared:
                    shared = {g: [keys(s[c], s["prefix_table"][g], before) for c in ("k_cache", "v_cache")]}
                k, v = torch.cat([shared[g][0], k]), torch.cat([shared[g][1], v])
        q = s["q"][off[r]:off[r + 1]].double().view(n, hk, hq // hk, d)
        z = torch.einsum("nhgd,lhd->hgnl", q, k) * s["scale"]
        last = before + kv[r] - n + torch.arange(n, device="cuda")
        z = z.masked_fill(torch.arange(len(k), device="cuda")[None, :] > last[:, None], -torch.inf)
        out[off[r]:off[r + 1]] = torch.einsum("hgnl,lhd->nhgd", torch.softmax(z, -1), v).reshape(n, hq, d)
        lse[off[r]:off[r + 1]] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(n, hq)
    return {"out": out, "lse": lse}


# --------------------------------------------------------------- the work --
def work(case):
    es, d, hk, hq = DTYPES[case["dtype"]].itemsize, case["D"], case["Hk"], case["Hq"]
    packed = d // 2 + d // GROUP  # bytes of a head in 4 bits
    if case["op"] != "attend":
        n, heads, turned = case["rows"], hq + 2 * hk, hq + hk
        flops = n * turned * (3 * case["rot"] + (4 * d if case.get("norm", True) else 0))
        if case["op"] == "norm":
            return {"bytes": 2 * n * heads * d * es + 8 * n + 4 * case["rot"] + 8 * d, "flops": flops}
        # the inputs, the turned queries, the packed heads written and read back, their values
        return {"bytes": n * (heads + hq) * d * es + 2 * n * hk * (2 * packed + 2 * d) + 12 * n + 4 * case["rot"] + 8 * d, "flops": flops + 4 * n * hk * d}
    n, kv = _lengths(case)
    rows, R = int(n.sum()), case["R"]
    keys = int((n * kv - n * (n - 1) // 2).sum())
    shared = 0
    if case["groups"]:
        goff, plen = _groups(case)
        shared = int(plen.sum())
        per = (plen * np.diff(goff)).sum() / R  # each request as likely in each group
        keys += int(rows * per)
    return {"bytes": 2 * rows * hq * d * es + 4 * rows * hq + 2 * (int(kv.sum()) + shared) * hk * packed, "flops": 4 * keys * hq * d}
