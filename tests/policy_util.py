"""Plain 64-bit definitions of a token's log-probability and the clipped policy
loss, their gradients by formula, and the bounds their tests use; torch float64 on
the CPU, nothing here calls the library."""
import math

import torch

from llm_util import U, rounding, sum_depth


def logp(logits, token, temperature):
    """(log-probabilities of every column, of the token or 0, rows that count)."""
    lq = torch.log_softmax(logits.double() / temperature, 1)
    dead = ~(logits > -math.inf).any(1) & ~torch.isnan(logits).any(1)
    lq = lq.masked_fill(dead[:, None], -math.inf)       # nothing can be drawn from a row of nothing but -inf
    here = (token >= 0) & (token < logits.shape[1])
    at = torch.where(here, token, torch.zeros_like(token)).long()
    l = lq.gather(1, at[:, None])[:, 0].masked_fill(~here, 0)
    return lq, l, here, at, dead


def logp_tol(logits, token, temperature):
    """l = s (z_y - m) - ln S.  S's sum goes through D additions, an exponential is
    off by a few U times its argument, which matters by its share of S (the mean of
    |log q| is at most ln V, and s's own rounding has the same effect), and the two
    terms are rounded."""
    V = logits.shape[1]
    z = logits.double()
    lq, l, here, at, dead = logp(logits, token, temperature)
    m = z.amax(1)
    reach = ((z.gather(1, at[:, None])[:, 0] - m) / temperature).abs()
    reach = torch.where(torch.isfinite(reach), reach, torch.zeros_like(reach))
    D = 64 + 2 * sum_depth(V)
    return U * (D + 16 * (1 + reach + math.log(V) + l.abs().nan_to_num(0.0, 0.0, 0.0)))


def loss(l, adv, old, ref, lo, hi, beta):
    """The loss of log-probabilities l, from the definition (float64, differentiable)."""
    a = adv.double()
    rho = (l - (l.detach() if old is None else old.double())).exp()
    out = -torch.minimum(rho * a, rho.clamp(1 - lo, 1 + hi) * a)
    if ref is not None and beta > 0:
        d = ref.double() - l
        out = out + beta * (torch.expm1(d) - d)
    return out


def slope(l, adv, old, ref, lo, hi, beta):
    """The formula of dloss/dl."""
    a = adv.double()
    rho = torch.ones_like(l) if old is None else (l - old.double()).exp()
    free, held = rho * a, rho.clamp(1 - lo, 1 + hi) * a
    g = torch.where(free <= held, -free, torch.zeros_like(free))
    if ref is not None and beta > 0:
        g = g - beta * torch.expm1(ref.double() - l)
    return g


def tolerances(l, tl, adv, old, ref, beta):
    """(bound of the loss, bound of its slope): exp(x) is off by its argument's error
    and a few roundings, and expm1 likewise, relative to itself."""
    a = adv.double().abs()
    apart = torch.zeros_like(l) if old is None else (l - old.double()).abs()
    rho = torch.ones_like(l) if old is None else (l - old.double()).exp()
    # the clipped ratio is 1 - lo or 1 + hi in binary32
    t = a * (rho * (tl * (old is not None) + U * (4 + 4 * apart)) + 3 * U)
    t_loss, t_slope = t, t
    if ref is not None and beta > 0:
        d = ref.double() - l
        e, x = d.exp(), torch.expm1(d).abs()
        td = tl + 2 * U * (d.abs() + l.abs())
        t_loss = t_loss + beta * (x * td + 8 * U * (x + d.abs()))
        t_slope = t_slope + beta * (e * td + 8 * U * x)
    return t_loss + 1e-30, t_slope + 1e-30


def gradient(logits, token, temperature, g_l, t_l, ft):
    """dlogits = g_l s (1[j = y] - q_j) and its bound, where g_l (already times the
    row's dloss) is off by t_l."""
    lq, l, here, at, dead = logp(logits, token, temperature)
    s = 1.0 / temperature
    q = lq.exp()
    one = torch.zeros_like(q).scatter_(1, at[:, None], 1.0)
    k, tk = (v.masked_fill(~here | dead, 0)[:, None] * s for v in (g_l, t_l))
    D = 64 + 2 * sum_depth(logits.shape[1])
    tq = q * (D + 8 * lq.abs().nan_to_num(0.0, 0.0, 0.0).clamp_max(1e4)) * U
    grad = k * (one - q)
    tol = tk * (one - q).abs() + k.abs() * (tq + 3 * U * (one + q)) + 2.0 ** -126
    return grad, tol + rounding(grad, ft)
