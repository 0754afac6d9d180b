"""A paged cache in 4 bits in plain numpy and torch, written from its definition: what nibbles and scale bytes stand for,
and the nearest code of values in 64 bits."""
import numpy as np
import torch

GROUP = 32


def scales(code):
    """2^((b >> 3) - 20) (1 + (b & 7) / 8) of scale bytes, in 64 bits."""
    b = code.long()
    return torch.exp2((b // 8 - 20).double()) * (1 + (b % 8).double() / 8)


def decode(cache):
    """Values [pages, page_size, Hk, D] in 64 bits of a (data, scales) pair."""
    data, scale = cache
    nib = torch.stack([data & 15, data >> 4], -1).flatten(-2).double() - 8  # [pages, Hk, groups, P, 32]
    x = nib * scales(scale).transpose(2, 3)[..., None]
    return x.permute(0, 3, 1, 2, 4).flatten(3)


def encode(x):
    """Scale bytes [..., groups] and whole numbers -7 .. 7 [..., groups, 32] of values [..., D] of 64 bits."""
    x = x.double().unflatten(-1, (-1, GROUP))
    t = x.abs().amax(-1) / 7
    m, e = np.frexp(t.cpu().numpy())  # t = m 2^e, 1/2 <= m < 1
    eighths = np.floor(m * 16 + 0.5).astype(np.int64)  # 8 .. 16
    e = e.astype(np.int64) - 1
    b = np.where(t.cpu().numpy() == 0, 0, np.clip((e + 20) * 8 + eighths - 8, 0, 255))
    code = torch.from_numpy(b).to(x.device)
    n = torch.round(x / scales(code)[..., None]).clamp(-7, 7)
    return code, n


def pack(code, n):
    """A (data, scales) pair of codes [pages, P, Hk, groups] and numbers [pages, P, Hk, groups, 32]."""
    u = (n + 8).to(torch.uint8)
    data = (u[..., 0::2] | (u[..., 1::2] << 4)).permute(0, 2, 3, 1, 4).contiguous()
    return data, code.to(torch.uint8).permute(0, 2, 1, 3).contiguous()
