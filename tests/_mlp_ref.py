"""Plain float64 forms of the MLP operators, for the tests: layer norm, dropout's
mask, the activations and their derivatives."""
import math

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def rounding(dtype, ref):
    """How far one rounding to dtype moves numbers near ref: half a step, which below
    the smallest normal number is half of the smallest subnormal one."""
    info = torch.finfo(dtype)
    return torch.clamp(ref.abs() * (info.eps / 2), min=info.tiny * info.eps / 2)


def philox(counter, key):
    """Philox 4x32-10 of one block: four counter words, two key words -> four words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(count, p, seed, offset):
    """Truth values of the elements that dropout keeps (numpy, vectorised)."""
    u = np.uint64
    with np.errstate(over="ignore"):
        i = np.arange(-(-count // 8), dtype=u) + u(offset % 2 ** 64)
    c = [i & u(0xFFFFFFFF), i >> u(32), np.zeros_like(i), np.zeros_like(i)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & u(0xFFFFFFFF), (a >> u(32)) ^ c[3] ^ u(k[1]),
             a & u(0xFFFFFFFF)]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.empty((i.size, 8), dtype=np.uint32)
    for w in range(4):
        bits[:, 2 * w], bits[:, 2 * w + 1] = c[w] & u(0xFFFF), c[w] >> u(16)
    return bits.reshape(-1)[:count] >= threshold(p)


def threshold(p):
    return math.floor(65536 * p + 0.5)


def gate(z, act):
    """(v, dv/dz) where the activation is z sigmoid(v)."""
    if act == "silu":
        return z, torch.ones_like(z)
    a = math.sqrt(8 / math.pi)
    return a * (z + 0.044715 * z ** 3), a * (1 + 3 * 0.044715 * z ** 2)


def activation(z, act):
    return z if act == "none" else z * torch.sigmoid(gate(z, act)[0])


def slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    v, dv = gate(z, act)
    s = torch.sigmoid(v)
    return s + z * dv * s * torch.sigmoid(-v)


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) of float64 rows x."""
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = gamma * (x - mean) * rstd
    return y if beta is None else y + beta, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, gamma, dres):
    xh = (x - mean) * rstd
    t = gamma * dy
    dx = rstd * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    lead = tuple(range(dy.ndim - 1))
    return dx if dres is None else dx + dres, (dy * xh).sum(lead), dy.sum(lead)
