"""The operators of a layer around the decode step, from their definitions in 64 bits (test infrastructure), and the
tolerances they are held to.

Tolerances, from the arithmetic and the number formats:

* bf16 results are rounded once, to nearest: off by at most half a step, 2^-8 relative, on top of the error of the
  fp32 value behind them.
* The scan's fp32 values: operands are pairs of 22 significant bits and the product of their low halves is dropped, so
  a product is within 3 2^-22 of exact; a chunk runs at most six products in sequence (pairs of tokens, triangular
  solve, rows, residual, state, output), each over up to 128 terms whose rounded sums add up to 2^-22 of the sum of
  the terms' magnitudes.  That is 6 * 4 2^-22 of sums of magnitudes, which for the random signs here exceed the
  results' largest value by less than a factor of 4 (half the square root of the 128 terms, as the largest of many
  results is 2 or more standard deviations): 96 2^-22 = 2.3e-5 of the largest value.  The recurrence contracts
  (decays at most 1, |k| at most 1, beta in [0, 1]), so errors of earlier chunks do not grow.  SCAN_REL = 2.5e-5.
* An element far below its tile's largest is held within 2^-39 of that largest (the pair's low half ends there), not
  within 2^-22 of itself.  Decays make such elements: where everything at the start has been forgotten, results fall to
  any size while their operands' tiles do not, and are off by up to 2^-39 of the products that forgot them.  With at most
  8 such products in a chunk: FLOOR = 2^-36 of the largest input (values, states, gradients), absolute.
* dg is a difference of sums, of rows and columns of its 16-token sub-block (random signs: a factor of 4) and of whole
  sub-blocks: DG_REL = 4 SCAN_REL of the largest value, and of the terms |q dq| + |k dk|, whose difference may vanish
  (for a single token from a zero state it does, exactly).  Over a whole tensor the errors are random: a product's is
  1.6 2^-24 in the mean (two operand pairs rounded, a dropped product, four additions), and dg adds up some 40 of them,
  sqrt(40) 1.6 2^-24 = 6e-7 of terms of its own size: DG_NORM, normwise, is twice that.
* The norm and rotation: sums of D <= 256 squares in fp32, a reciprocal square root (2 ulp), cos and sin (2 ulp) and a
  handful of products: below 32 ulp = 2^-19 of the head's largest value.  QK_REL = 2^-19; the weights' gradients, sums
  of fp32 products in fp32 and fp64, within 2^-19 of the sum of the terms' magnitudes.
"""
from __future__ import annotations

import torch

BF16_HALF_STEP = 2.0 ** -8
SCAN_REL = 2.5e-5
DG_REL = 4 * SCAN_REL
DG_NORM = 1.2e-6
FLOOR = 2.0 ** -36
QK_REL = 2.0 ** -19


def check(got, ref, rel, what, half_step=0.0, floor=0.0):
    """|got - ref| <= half_step |ref| + rel max|ref| + floor, element by element."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    got, ref = got.double(), ref.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    if ref.numel() == 0:
        return
    # the rounding is of the computed value, itself within rel max|ref| of ref
    bound = half_step * ref.abs() + (1 + half_step) * (rel * ref.abs().max() + floor)
    over = (got - ref).abs() - bound
    assert float(over.max()) <= 0, (f"{what}: {int((over > 0).sum())} of {ref.numel()} elements off, worst by "
                                    f"{float(over.max()):.3e}, largest reference {float(ref.abs().max()):.3e}")


def scan(q, k, v, g, beta, state, cu, scale):
    """The recurrence token by token: out [rows, HV, V] (zeros outside the sequences) and the final states; fp64,
    differentiable.  Sequences run side by side; a token past the end of one leaves its state (k = beta = g = 0)."""
    cu = [int(x) for x in cu]
    N, rows = len(cu) - 1, q.shape[0]
    longest = max([b - a for a, b in zip(cu, cu[1:])], default=0)
    idx = torch.full((longest, N), rows, dtype=torch.long, device=q.device)
    for n in range(N):
        idx[:cu[n + 1] - cu[n], n] = torch.arange(cu[n], cu[n + 1], device=q.device)
    q, k, v, g, beta = (torch.cat([x, x.new_zeros(1, *x.shape[1:])])[idx] for x in (q, k, v, g, beta))
    S, outs = state, []
    for t in range(longest):
        S = torch.exp(g[t])[..., None] * S
        r = v[t] - (k[t][..., None] * S).sum(-2)
        S = S + (beta[t][..., None] * k[t])[..., None] * r[..., None, :]
        outs.append(scale * (q[t][..., None] * S).sum(-2))
    out = v.new_zeros(rows + 1, *v.shape[2:])
    if outs:
        out = out.index_put((idx.reshape(-1),), torch.stack(outs).flatten(0, 1))
    return out[:-1], S


def scan_gradients(q, k, v, g, beta, state, cu, scale, d_out, d_final):
    """(out, final, dq, dk, dv, dg, dbeta, dstate) in fp64."""
    leaves = [x.detach().double().requires_grad_() for x in (q, k, v, g, beta, state)]
    out, final = scan(*leaves, cu, scale)
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device=q.device)
    for a, b in zip(cu, cu[1:]):
        inside[int(a):int(b)] = True
    loss = (out * d_out.double() * inside[:, None, None]).sum() + (final * d_final.double()).sum()
    grads = torch.autograd.grad(loss, leaves, allow_unused=True)
    return (out.detach(), final.detach(), *(torch.zeros_like(x) if d is None else d for d, x in zip(grads, leaves)))


def qk(x, norm, eps, weight, positions, inv_freq, interleaved, rope_scale):
    """The norm and rotation of [rows, heads, D] in fp64, differentiable; the rotation as a complex product."""
    y = x
    if norm == "l2":
        y = y / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)
    elif norm == "rms":
        y = y / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight
    if inv_freq is None or inv_freq.numel() == 0:
        return y
    r = 2 * inv_freq.numel()
    angle = positions.double().reshape(-1)[:, None, None] * inv_freq
    turn = torch.polar(torch.full_like(angle, rope_scale), angle)
    if interleaved:
        z = turn * torch.view_as_complex(y[..., :r].unflatten(-1, (-1, 2)).contiguous())
        return torch.cat([torch.view_as_real(z).flatten(-2), y[..., r:]], -1)
    z = turn * torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous())
    return torch.cat([z.real, z.imag, y[..., r:]], -1)
