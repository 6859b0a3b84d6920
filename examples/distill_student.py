"""Quantization-aware distillation of a small W8A8 student from a teacher's
stored top logits, on the library's calls end to end:

    x -> layer norm + s8 codes -> W8A8 product, bias, gelu -> s8 codes
      -> W8A8 product, bias, + x -> layer norm + s8 codes -> W8A8 product -> logits
    loss and its gradient at the logits in one call, then back through the
    epilogues and the norms; the quantizers are passed straight through, and
    the weights' gradients are plain matrix products.

    python examples/distill_student.py [--steps 60]

The teacher is a random two-layer network, of which only each position's top
logits and their log-sum-exp are kept, as a stored distillation set would."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import tensor_quantization_amd as tq  # noqa: E402


def deq(q, scale):
    """s8 codes [rows, cols] as the values they stand for."""
    return tq.tq_dequant_per_token(q, q.shape, scale)


class Student:
    """Binary32 master parameters; the products run on s8 codes of them, one
    scale per output channel."""

    def __init__(self, width, hidden, vocab, gen):
        def w(n, k):
            return torch.randn((n, k), generator=gen, device="cuda") / k ** 0.5
        ones, zeros = (lambda n: torch.ones(n, device="cuda")), (lambda n: torch.zeros(n, device="cuda"))
        self.params = {"g1": ones(width), "c1": zeros(width), "w1": w(hidden, width), "b1": zeros(hidden),
                       "w2": w(width, hidden), "b2": zeros(width), "g2": ones(width), "c2": zeros(width),
                       "head": w(vocab, width)}

    def step(self, x, idx, val, lse, temperature):
        """One forward and backward pass: (mean loss, logits, gradients)."""
        p, t = self.params, x.shape[0]
        qw = {n: tq.tq_quant_per_token(p[n])[:2] for n in ("w1", "w2", "head")}

        q0, s0, m0, r0 = tq.tq_layer_norm_quant_per_token(x, p["g1"], p["c1"], stats=True)
        a, z = tq.tq_w8a8_linear_epilogue(q0, s0, *qw["w1"], bias=p["b1"], act="gelu", out_dtype=x.dtype, preact=True)
        q1, s1, _ = tq.tq_quant_per_token(a)
        y = tq.tq_w8a8_linear_epilogue(q1, s1, *qw["w2"], bias=p["b2"], residual=x, out_dtype=x.dtype)
        q2, s2, m2, r2 = tq.tq_layer_norm_quant_per_token(y, p["g2"], p["c2"], stats=True)
        logits = tq.tq_w8a8_linear_epilogue(q2, s2, *qw["head"], out_dtype=x.dtype)

        mean = torch.full((t,), 1.0 / t, device=x.device)
        loss, dlogits = tq.tq_topk_distill_grad(logits, idx, val, dloss=mean, temperature=temperature, teacher_lse=lse)

        g = {"head": dlogits.float().t() @ deq(q2, s2)}
        dn2 = (dlogits.float() @ deq(*qw["head"])).to(x.dtype)
        dy, g["g2"], g["c2"] = tq.tq_layer_norm_backward(dn2, y, p["g2"], m2, r2)
        _, g["b2"] = tq.tq_linear_epilogue_backward(dy, y)
        g["w2"] = dy.float().t() @ deq(q1, s1)
        da = (dy.float() @ deq(*qw["w2"])).to(x.dtype)
        dz, g["b1"] = tq.tq_linear_epilogue_backward(da, z, "gelu")
        g["w1"] = dz.float().t() @ deq(q0, s0)
        dn1 = (dz.float() @ deq(*qw["w1"])).to(x.dtype)
        _, g["g1"], g["c1"] = tq.tq_layer_norm_backward(dn1, x, p["g1"], m0, r0)
        return loss.mean(), logits, g


def stored_teacher(x, vocab, top, temperature, gen):
    """A random teacher's top logits [tokens, top], their columns and the
    log-sum-exp of all its logits / temperature."""
    a = torch.randn((x.shape[1], 2 * x.shape[1]), generator=gen, device="cuda") / x.shape[1] ** 0.5
    b = torch.randn((2 * x.shape[1], vocab), generator=gen, device="cuda") * (8 / x.shape[1]) ** 0.5
    logits = torch.tanh(x.float() @ a) @ b
    val, idx = logits.topk(top, dim=1)
    return idx, val, torch.logsumexp(logits / temperature, 1)


def train(steps=60, tokens=1024, width=256, hidden=640, vocab=4000, top=32, temperature=1.5, lr=3e-3, seed=0,
          log=print):
    """Trains on one batch; returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, width), generator=gen, device="cuda").to(torch.bfloat16)
    idx, val, lse = stored_teacher(x, vocab, top, temperature, gen)
    student = Student(width, hidden, vocab, gen)
    opt = torch.optim.Adam(student.params.values(), lr=lr)
    losses = []
    for i in range(steps):
        loss, _, grads = student.step(x, idx, val, lse, temperature)
        for name, p in student.params.items():
            p.grad = grads[name].to(p.dtype)
        opt.step()
        losses.append(loss)
        if i % 10 == 0 or i == steps - 1:
            log("step %3d  loss %.4f" % (i, loss.item()))
    return [v.item() for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)
