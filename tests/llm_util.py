"""Plain 64-bit definitions of the operators around a quantized layer (layer
norm, the epilogue of the W8A8 product, distillation from top logits) and the
error bounds their tests use.  Written from the formulas, in torch float64 on
the CPU; nothing here calls the library."""
import math

import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24                                        # half an ulp of binary32, relative
HALF_ULP = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}   # the types' smallest steps


def rounding(v, ft):
    """Bound of rounding the values v to type ft (subnormals included)."""
    return v.abs() * HALF_ULP[ft] + TINY[ft]


def assert_within(got, want, tol, what):
    """|got - want| <= tol element by element; infinities and NaNs in place."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(same[odd].all()), "%s: infinities or NaNs differ" % what
    err = (got - want).abs()
    bad = ~odd & ~(err <= tol)
    if bool(bad.any()):
        at = torch.nonzero(bad)[0].tolist()
        raise AssertionError("%s: %d of %d outside; first at %s: got %r want %r tol %r" % (
            what, int(bad.sum()), bad.numel(), at, float(got[tuple(at)]), float(want[tuple(at)]),
            float(tol[tuple(at)] if isinstance(tol, torch.Tensor) else tol)))


# ---------------------------------------------------------------- layer norm
def sum_depth(n):
    """Most additions one term of a row's sum goes through: 16 in a thread or n
    / 1024 in the kernel of long rows, 6 across a wave, 16 across waves."""
    return 16 + math.ceil(n / 1024) + 6 + 16


def layer_norm(x, w, b, eps):
    x = x.double()
    mu = x.mean(-1, keepdim=True)
    var = ((x - mu) ** 2).mean(-1, keepdim=True)
    r = (var + eps) ** -0.5
    h = (x - mu) * r
    y = h * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mu, r, h


def layer_norm_tol(x, w, b, eps, ft):
    """mu is off by D u mean|x| (D the sum's depth) and carries into the
    variance, r by half the variance's relative error (D u of its own sum, and
    the mean's error squared or against the spread), then one rounding for
    each of x - mu, times r, times w plus b."""
    y, mu, r, h = layer_norm(x, w, b, eps)
    D = sum_depth(x.shape[-1]) + 4
    dmu = D * U * x.double().abs().mean(-1, keepdim=True)
    rel = (D + 8) * U + (dmu * r) ** 2
    ww = torch.ones_like(y) if w is None else w.double().abs().expand_as(y)
    bb = 0 if b is None else b.double().abs()
    tol = ww * (h.abs() * (rel + 4 * U) + dmu * r * (1 + rel)) + 2 * U * (bb + y.abs())
    return tol + rounding(y, ft), dmu + U * mu.abs(), r * (rel + 2 * U)


def layer_norm_backward(dy, x, w, mean, rstd):
    x, dy = x.double(), dy.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    g = dy if w is None else dy * w.double()
    dx = rstd * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0), g, h


def layer_norm_backward_tol(dy, x, w, mean, rstd, ft, wt):
    dx, dw, db, g, h = layer_norm_backward(dy, x, w, mean, rstd)
    D = sum_depth(x.shape[-1]) + 8
    r = rstd.double()[:, None]
    m1, m2 = g.abs().mean(-1, keepdim=True), (g * h).abs().mean(-1, keepdim=True)
    tdx = r * (6 * U * g.abs() + D * U * m1 + (D + 6) * U * h.abs() * m2) + rounding(dx, ft)
    # rows in a thread (256 groups of at least one team), then teams, groups and lanes
    R = x.shape[0] / 64 + 64
    return (tdx, (R + 4) * U * (dy.double() * h).abs().sum(0) + rounding(dw, wt),
            (R + 4) * U * dy.double().abs().sum(0) + rounding(db, wt))


# ----------------------------------------------------------------- epilogue
def act(z, name):
    f = torch.nn.functional
    if name == "relu":
        return f.relu(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z ** 2)
    return torch.ones_like(z)


def epilogue(acc, sx, sw, bias, name, residual):
    z = acc.double() * sx.double()[:, None] * sw.double()[None, :]
    if bias is not None:
        z = z + bias.double()
    y = act(z, name)
    return z, (y if residual is None else y + residual.double())


def epilogue_tol(acc, sx, sw, bias, name, residual, ft):
    """z takes at most four roundings; an activation's slope is below 1.2, and
    its own evaluation is within 16 roundings plus the error of its exponent's
    argument, |a| u, where the result still matters (z times a slope that has
    decayed by exp(-|a|): |a| exp(-|a|) < 1)."""
    z, y = epilogue(acc, sx, sw, bias, name, residual)
    t = acc.double().abs() * sx.double()[:, None] * sw.double()[None, :] + (0 if bias is None else bias.double().abs())
    tz = 4 * U * t
    ty = 1.2 * tz + (0 if name in ("none", "relu") else 24 * U * z.abs())
    if residual is not None:
        ty = ty + U * (y.abs() + residual.double().abs())
    return tz + rounding(z, ft), ty + rounding(y, ft)


# -------------------------------------------------------------- distillation
def distill(logits, idx, val, temperature, teacher_lse):
    """Loss of every row, from the definition (float64, differentiable)."""
    s = 1.0 / temperature
    V = logits.shape[1]
    here = (idx >= 0) & (idx < V)
    at = torch.where(here, idx, torch.zeros_like(idx)).long()
    t = (val.double() * s).masked_fill(~here, -math.inf)
    none = ~here.any(1) if teacher_lse is not None else ~(t > -math.inf).any(1)
    logq = torch.log_softmax(logits * s, 1)
    logp = t - (teacher_lse.double()[:, None] if teacher_lse is not None
                else torch.logsumexp(t, 1, keepdim=True).masked_fill(none[:, None], 0))
    p = logp.exp()
    terms = p * (logp - logq.gather(1, at))
    loss = torch.where(p > 0, terms, torch.zeros_like(p)).sum(1)
    if teacher_lse is not None:
        pr = (1 - p.sum(1)).clamp_min(0)
        taken = torch.zeros(logits.shape, dtype=torch.int32)
        taken.scatter_add_(1, at, here.int())
        log_rest = torch.logsumexp(logq.masked_fill(taken > 0, -math.inf), 1)
        loss = loss + torch.where(pr > 0, pr * (pr.log() - log_rest), torch.zeros_like(pr))
    # nothing can be drawn from a row of nothing but -inf: whatever the teacher expects there is lost
    loss = torch.where((logits > -math.inf).any(1) | torch.isnan(logits).any(1), loss, torch.full_like(loss, math.inf))
    return torch.where(none, torch.zeros_like(loss), loss), p.masked_fill(none[:, None], 0), none


def distill_grad(logits, idx, val, temperature, teacher_lse, dloss):
    """The formula of the gradient, and a bound for a binary32 evaluation:
    every exponential is off by a few u times its argument (|log q|, |log p|),
    the sums by their depth, p_r = 1 - sum p by its own sum's rounding."""
    s = 1.0 / temperature
    z = logits.double()
    loss, p, none = distill(z, idx, val, temperature, teacher_lse)
    V = z.shape[1]
    here = (idx >= 0) & (idx < V)
    at = torch.where(here, idx, torch.zeros_like(idx)).long()
    pj = torch.zeros_like(z).scatter_add_(1, at, p.masked_fill(~here, 0))
    taken = torch.zeros_like(z).scatter_add_(1, at, here.double()) > 0
    q = torch.softmax(z * s, 1)
    lq = torch.log_softmax(z * s, 1)
    D = 64 + 2 * sum_depth(V)
    scale = (s * (torch.ones(z.shape[0]) if dloss is None else dloss).double())[:, None]
    lp = torch.where(pj > 0, pj.log().abs(), torch.zeros_like(pj))
    eq = q * (D + 8 * lq.abs().clamp_max(1e4)) * U
    if teacher_lse is None:
        grad = q - pj
        tol = eq + pj * (D + 8 * lp) * U
    else:
        # s t and teacher_lse are subtracted in binary32: an error of their size in the exponent
        big = (val.double().abs() * s).masked_fill(~(p > 0), 0).amax(1) + teacher_lse.double().abs()
        dp = (D + 8 * big)[:, None] * U
        pr = (1 - p.sum(1)).clamp_min(0)[:, None]
        qr = q.masked_fill(taken, 0).sum(1, keepdim=True)
        Z = p.sum(1, keepdim=True) + pr
        ratio = torch.where((pr > 0) & (qr > 0), pr / qr, torch.zeros_like(pr))
        grad = torch.where(taken, q * Z - pj, q * (Z - ratio))
        tol = (eq + dp * q) * (Z + ratio) + pj * (dp + 8 * U * lp) + torch.where(taken | (qr == 0), 0 * q, q * dp / qr)
    gone = none | ~(z > -math.inf).any(1)
    grad = grad.masked_fill(gone[:, None], 0)
    tol = tol.masked_fill(gone[:, None], 0)
    return grad * scale, tol * scale.abs() + 2.0 ** -126, loss


def distill_loss_tol(logits, idx, val, temperature, teacher_lse):
    s = 1.0 / temperature
    z = logits.double()
    loss, p, none = distill(z, idx, val, temperature, teacher_lse)
    V = z.shape[1]
    here = (idx >= 0) & (idx < V)
    at = torch.where(here, idx, torch.zeros_like(idx)).long()
    lq = torch.log_softmax(z * s, 1).gather(1, at).abs()
    lq = torch.where(p > 0, lq, torch.zeros_like(lq))
    lp = torch.where(p > 0, p.log().abs(), torch.zeros_like(p))
    D = 64 + 2 * sum_depth(V)
    own = (p * (D + 8 * (lq + lp)) * (1 + lq + lp)).masked_fill(~(p > 0), 0).sum(1)
    if teacher_lse is None:
        return own * U + U
    big = (val.double().abs() * s).masked_fill(~(p > 0), 0).amax(1) + teacher_lse.double().abs()
    # p's error times its term, the rest's and its logarithm's
    q = torch.softmax(z * s, 1)
    taken = torch.zeros_like(z).scatter_add_(1, at, here.double()) > 0
    qr = q.masked_fill(taken, 0).sum(1)
    pr = (1 - p.sum(1)).clamp_min(0)
    lr = torch.where((pr > 0) & (qr > 0), (pr / qr).log().abs(), torch.zeros_like(pr))
    dp = D + 8 * big
    return (own + dp * ((p * (1 + lq + lp)).masked_fill(~(p > 0), 0).sum(1) + 1 + lr) + pr * D * (1 + lr)) * U + U
