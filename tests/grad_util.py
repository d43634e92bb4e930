"""64-bit gradients of masked attention, and how far the kernels may be from them.

The kernel rounds P and dS to bf16 in front of their tensor products and the gradients at the end,
each by at most U = eps / 2 = 2^-8 of the value; P itself carries the error of its exponential and of
the fp32 exponent (below 2^-12 of the value for exponents up to a few hundred), and every product of
a length-d row is summed in fp32 (below ACC of the sum of the absolute terms).  The bounds add these
up, element by element, over the sums the gradients are made of.
"""
import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
P_REL = 2.0 ** -12
ACC = 2.0 ** -15      # up to 128 fp32 additions at 2^-23 each, with room for the two final ones
SUM = 2.0 ** -14      # fp32 sums over the keys or queries, relative to the sum of the absolute terms


def reference(q, k, v, do, allowed, scale=None, d_lse=None, o=None, lse=None, own_o=False):
    """One head in 64 bits on natural-order rows.  allowed: [N, N] bool, queries by keys.  o and lse:
    the forward call's, where given; else the exact ones.  own_o: the kernel's delta comes from its own
    O before its rounding, whose error is that of P (U + P_REL of every term).  Returns o, lse,
    (dq, dk, dv) and their bounds."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    scale = 1 / math.sqrt(q.shape[1]) if scale is None else scale
    s = (q @ k.T * scale).masked_fill(~allowed, -math.inf)
    true_lse = torch.logsumexp(s, dim=1)
    sees = allowed.any(1)
    p_true = torch.where(sees[:, None], torch.exp(s - torch.where(sees, true_lse, 0.0)[:, None]), 0.0)
    true_o = p_true @ v
    o = true_o if o is None else o.double()
    lse = true_lse if lse is None else lse.double()
    p = torch.where((lse != -math.inf)[:, None], torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    delta = (do * o).sum(1)
    if d_lse is not None:
        delta = delta - d_lse.double()
    ds = p * (do @ v.T - delta[:, None])
    grads = (scale * ds @ k, scale * ds.T @ q, p.T @ do)
    e = ACC * ((do.abs() @ v.abs().T) + (do.abs() * o.abs()).sum(1)[:, None] +
               (d_lse.double().abs()[:, None] if d_lse is not None else 0.0))
    if own_o:
        e = e + (U + P_REL + SUM) * (do.abs() * (p @ v.abs())).sum(1)[:, None]
    w = (U + P_REL + SUM) * ds.abs() + 1.01 * p * e
    # dq's own sum of the errors, times the row's mean key, is taken off again: at worst it adds up
    bounds = (scale * (w @ k.abs() + 1.01 * w.sum(1, keepdim=True) * (p @ k.abs())) + U * grads[0].abs(), scale * w.T @ q.abs() + U * grads[1].abs(),
              (U + P_REL + SUM) * p.T @ do.abs() + U * grads[2].abs())
    # bf16 stores nothing finer than its smallest subnormal step
    return true_o, true_lse, grads, tuple(1.02 * b + 2.0 ** -133 for b in bounds)


def assert_grads(got, want, bounds, what="", names=("dq", "dk", "dv")):
    for name, g, w, b in zip(names, got, want, bounds):
        g = g.double()
        assert torch.isfinite(g).all(), f"{what}: {name} is not finite"
        over = (g - w).abs() - b
        at = int(over.argmax())
        assert over.max() <= 0, (f"{what}: {name}[{at // g.shape[1]}, {at % g.shape[1]}] = {g.flatten()[at]:.6g}, "
                                 f"want {w.flatten()[at]:.6g} within {b.flatten()[at]:.3g}")


def allowed_blocks(keep, slots, block, kslots=None):
    """[N, N] token mask from a block mask [nb, nb] over layouts: slots[t] is token t's slot."""
    keep = torch.as_tensor(keep)
    qb = torch.as_tensor(slots) // block
    kb = qb if kslots is None else torch.as_tensor(kslots) // block
    return keep[qb][:, kb]
