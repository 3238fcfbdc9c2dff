"""The operators around a linear layer in binary64, for the tests: dropout's
words, activations and slopes, layer norm and its gradients, and the values
of block-scaled operands.  Written from the formulas in include/qfp4.h."""
import numpy as np
import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def philox(c, k):
    """Philox4x32-10 of counters c (4 arrays) under key k (2 ints)."""
    c = [np.asarray(v, np.uint64) for v in c]
    m = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    for r in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        k0 = np.uint64((k[0] + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64((k[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        c = [(p1 >> s) ^ c[1] ^ k0, p1 & m, (p0 >> s) ^ c[3] ^ k1, p0 & m]
    return c


def keep(shape, p, seed, step=0):
    """The elements that dropout keeps, as a numpy bool array."""
    n = int(np.prod(shape))
    q = np.arange(-(-n // 4), dtype=np.uint64)
    c = [q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, step & 0xFFFFFFFF),
         np.full_like(q, (step >> 32) + (1 << 31))]
    w = np.stack(philox(c, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)), -1).reshape(-1)[:n]
    return (w >= np.uint64(int(p * 2.0 ** 32))).reshape(shape)


def drop(v, p, seed, step=0):
    if p == 0:
        return v
    k = torch.from_numpy(keep(tuple(v.shape), p, seed, step)).to(v.device)
    return torch.where(k, v / (1.0 - p), torch.zeros_like(v))


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / 2 ** 0.5)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, name):
    """d act / dz by formula (relu: 0 at 0)."""
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    if name == "gelu_tanh":
        c = (2 / np.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        f = 1 / (1 + torch.exp(-z))
        return f * (1 + z * (1 - f))
    return torch.ones_like(z)


def layernorm(x, gamma, beta, eps):
    mean = x.mean(-1)
    xc = x - mean[:, None]
    rstd = 1 / torch.sqrt((xc * xc).mean(-1) + eps)
    y = xc * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_grads(dy, x, gamma, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


_GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def values(t, fmt):
    """What an operand's codes and scales stand for, in binary64; fmt 0 MXFP4, 1 NVFP4, 2 MXFP8."""
    codes, scales = t["codes"], t["scales"]
    if fmt == 2:
        v = codes.view(torch.float8_e4m3fn).double()
    else:
        v = _GRID.to(codes.device)[torch.stack([codes & 15, codes >> 4], -1).long()].flatten(1)
    s = scales.view(torch.float8_e4m3fn).double() if fmt == 1 else torch.exp2(scales.double() - 127)
    v = v * s.repeat_interleave(16 if fmt == 1 else 32, 1)
    return v * t["tscale"].double() if fmt == 1 else v


def random_operand(rows, K, fmt, seed, device="cuda", spread=3):
    """An operand of random codes under random scales of 2^-spread .. 2^spread."""
    g = torch.Generator().manual_seed(seed)
    if fmt == 2:
        v = (torch.randn((rows, K), generator=g) * 8).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes = v.view(torch.uint8)
    else:
        codes = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    if fmt == 1:
        scales = torch.randint(8 * (7 - spread), 8 * (7 + spread), (rows, K // 16), generator=g, dtype=torch.uint8)
    else:
        scales = torch.randint(127 - spread, 128 + spread, (rows, K // 32), generator=g, dtype=torch.uint8)
    out = {"codes": codes.to(device), "scales": scales.to(device)}
    if fmt == 1:
        out["tscale"] = torch.tensor([0.0371], device=device)
    return out


def keep_range(start, count, p, seed, step=0):
    """keep() of elements start .. start + count - 1 (start a multiple of 4)."""
    q = np.arange(start // 4, (start + count + 3) // 4, dtype=np.uint64)
    c = [q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, step & 0xFFFFFFFF),
         np.full_like(q, (step >> 32) + (1 << 31))]
    w = np.stack(philox(c, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)), -1).reshape(-1)[:count]
    return w >= np.uint64(int(p * 2.0 ** 32))
