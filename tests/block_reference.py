"""The gated feed-forward block's operators in 64 bits, written from their formulas
(include/quest.h), with no library code. Tensors stay on the device they are given on."""
import math

import torch


def hadamard(n, device):
    """Sylvester matrix, normalised: H_ij = (-1)^popcount(i & j) / sqrt(n)."""
    rows = [[-1.0 if bin(i & j).count("1") % 2 else 1.0 for j in range(n)] for i in range(n)]
    return torch.tensor(rows, dtype=torch.float64, device=device) / math.sqrt(n)


def transform(x, had):
    if not had:
        return x
    return (x.reshape(-1, had) @ hadamard(had, x.device)).reshape(x.shape)


def gate(a, act):
    """act(a) and its derivative."""
    if act == "silu":
        z, dz = a, torch.ones_like(a)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (a + 0.044715 * a ** 3), c * (1 + 0.134145 * a ** 2)
    s = torch.sigmoid(z)
    return a * s, s + a * s * torch.sigmoid(-z) * dz


def restore(codes, scales):
    """What an 8-bit checkpoint half stands for: codes [M, F], scales [M, ceil(F / 128)]."""
    col = torch.arange(codes.shape[1], device=codes.device) // 128
    return (codes.double() + 0.5) * scales.double()[:, col]


def halves(ckpt):
    F, g = ckpt["codes"].shape[1] // 2, ckpt["scales"].shape[1] // 2
    return (restore(ckpt["codes"][:, :F], ckpt["scales"][:, :g]),
            restore(ckpt["codes"][:, F:], ckpt["scales"][:, g:]))


def block_back(gh, a, b, act):
    v, dv = gate(a, act)
    return torch.cat([gh * b * dv, gh * v], 1)


def unpack4(packed, rows):
    p = packed.view(torch.uint8).reshape(rows, -1).long()
    return torch.stack([p % 16, p // 16], -1).reshape(rows, -1)


def midrise4(packed, rows):
    c = unpack4(packed, rows)
    return torch.where(c < 8, c, c - 16).double() + 0.5


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e2m1(packed, rows):
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=packed.device)
    return t[unpack4(packed, rows)]


def scaled(v, scales):
    """v [rows, K] times its steps [rows, groups] (or [rows])."""
    s = scales.double().reshape(v.shape[0], -1)
    return (v.reshape(v.shape[0], s.shape[1], -1) * s[..., None]).reshape(v.shape)


def bf16_input(values, scales):
    """bf16(value * step), the product in fp32: the operand a layer multiplied."""
    s = scales.reshape(values.shape[0], -1)
    v = values.float().reshape(values.shape[0], s.shape[1], -1) * s[..., None]
    return v.reshape(values.shape).to(torch.bfloat16).double()


def mask_values(mask, rows, cols):
    m = mask.view(torch.uint8).reshape(-1)[: rows * cols // 8].reshape(rows, cols // 8).long()
    bit = torch.arange(8, device=mask.device)
    return ((m[..., None] >> bit) & 1).reshape(rows, cols).double()


def weight_grad(gy, xh, mask, had=128):
    g = gy.double().t() @ xh
    if mask is not None:
        g = g * mask_values(mask, g.shape[0], g.shape[1])
    return transform(g, had)
