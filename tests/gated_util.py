"""Plain 64-bit definitions of the gated block and the bounds its tests use, in
torch float64 on the CPU; nothing here calls the library."""
import torch

from llm_util import U, act, act_slope, rounding

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def operands(M, F, K, seed, ft, lo=-127):
    g = torch.Generator().manual_seed(seed)

    def codes(rows):
        return torch.randint(lo, 128, (rows, K), generator=g, dtype=torch.int64).to(torch.int8)
    qx, qg, qu = codes(M), codes(F), codes(F)
    sx = (0.5 + torch.rand(M, generator=g)) / 64
    sg, su = ((0.5 + torch.rand(F, generator=g)) / (74 * max(1, K) ** 0.5) for _ in range(2))
    bg, bu = (torch.randn(F, generator=g).to(ft) for _ in range(2))
    return qx, sx, qg, sg, qu, su, bg, bu


def project(qx, sx, qw, sw, bias):
    """A projection and the bound of its binary32 evaluation: four roundings."""
    acc = qx.double() @ qw.double().t() if qx.shape[1] else torch.zeros(qx.shape[0], qw.shape[0], dtype=torch.float64)
    t = acc.abs() * sx.double()[:, None] * sw.double() + (0 if bias is None else bias.double().abs())
    z = acc * sx.double()[:, None] * sw.double() + (0 if bias is None else bias.double())
    return z, 4 * U * t


def gate(g, tg, u, tu, name):
    """act(g) u of values that are off by tg and tu.  An activation's slope is
    below 1.2, and its own evaluation is within 16 roundings plus the error of its
    exponent's argument where the result still matters: 24 U |g| in all."""
    a = act(g, name)
    ta = 1.2 * tg + (0 if name in ("none", "relu") else 24 * U * g.abs())
    y = a * u
    return y, ta * u.abs() + a.abs() * tu + ta * tu + 2 * U * y.abs()


def gate_backward(dy, z, name, ft):
    """dz, its bound, and the bound of dz before its rounding.  A slope is within
    32 U (1 + |g|) (its two terms may cancel), an activation within 24 U |g|."""
    F = z.shape[1] // 2
    d, g, u = dy.double(), z[:, :F].double(), z[:, F:].double()
    s, a = act_slope(g, name), act(g, name)
    dz = torch.cat([d * u * s, d * a], 1)
    tol = torch.cat([(d * u).abs() * 32 * U * (1 + g.abs()), d.abs() * 24 * U * g.abs()], 1) + 3 * U * dz.abs()
    return dz, tol + rounding(dz, ft), tol
