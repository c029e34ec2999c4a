"""Plain 64-bit definitions of the population operators and, beside each result, the sum of the
magnitudes that a rounding of a term can act on (the tolerances are a factor of it).

All functions take CPU tensors of any float type and compute in double, one sequence, row or model
at a time, from the formulas of include/cdrge.h.
"""
from __future__ import annotations

import torch

F = torch.float64


def scan(xbc, dt, conv_weight, conv_bias, decay, skip, dt_bias, heads, head_dim, groups, state, bounds, z=None,
         ring=None, state_in=None, positions=None):
    """Sequences bounds[i] = (first, end) of the rows of xbc; ring[i] [W, channels] and state_in[i] [heads, head_dim,
    state] are sequence i's carried state. Returns y, its magnitudes, and per sequence (state, its magnitudes, ring)."""
    W, d = conv_weight.shape[1], heads * head_dim
    cw, cb = conv_weight.to(F), (torch.zeros(conv_weight.shape[0]) if conv_bias is None else conv_bias).to(F)
    y, mag, carried = torch.zeros(xbc.shape[0], d, dtype=F), torch.zeros(xbc.shape[0], d, dtype=F), []
    for i, (first, end) in enumerate(bounds):
        pos = 0 if positions is None else max(int(positions[i]), 0)
        S = torch.zeros(heads, head_dim, state, dtype=F)
        past = torch.zeros(W, xbc.shape[1], dtype=F)
        if ring is not None:
            past = ring[i].to(F).clone()
        if pos > 0:
            S = state_in[i].to(F).clone()
        Sm = S.abs()
        for t in range(first, end):
            q = pos + t - first
            past[q % W] = xbc[t].to(F)
            u, um = cb.clone(), cb.abs()
            for j in range(W):
                at = q - (W - 1) + j
                if at >= 0:
                    u = u + cw[:, j] * past[at % W]
                    um = um + (cw[:, j] * past[at % W]).abs()
            u = u * torch.sigmoid(u)
            um = u.abs() + um / 16  # a sum's rounding acts on its terms, not on what is left of them
            step = torch.nn.functional.softplus(dt[t].to(F) + (0 if dt_bias is None else dt_bias.to(F)), threshold=1e9)
            fade = torch.exp(step * decay.to(F))[:, None, None]

            def split(v):
                x = v[:d].view(heads, head_dim)
                B = v[d:d + groups * state].view(groups, state).repeat_interleave(heads // groups, 0)
                C = v[d + groups * state:].view(groups, state).repeat_interleave(heads // groups, 0)
                return x, B, C

            (x, B, C), (xm, Bm, Cm) = split(u), split(um)
            S = fade * S + (step[:, None] * x)[:, :, None] * B[:, None, :]
            Sm = fade * Sm + (step[:, None] * xm)[:, :, None] * Bm[:, None, :]
            out, om = (S * C[:, None, :]).sum(2), (Sm * Cm[:, None, :]).sum(2)
            if skip is not None:
                out, om = out + skip.to(F)[:, None] * x, om + skip.to(F)[:, None].abs() * xm
            gate = 1.0 if z is None else (z[t].to(F) * torch.sigmoid(z[t].to(F)))
            y[t] = out.reshape(-1) * gate
            mag[t] = om.reshape(-1) * (1.0 if z is None else gate.abs())
        carried.append((S, Sm, past))
    return y, mag, carried


# Bounds of each element by the magnitudes of its terms, which hold for any inputs and are wide: what a matrix product of
# operands in bf16 (both off by 2^-8: (1 + 2^-8)^2 - 1), and one of operands in two bf16 halves (2^-16 each and 2^-16 for
# the low halves' product, twice in a row in y), may be off by; sums, exponentials and the convolution add less than 2^-17.
# The kernels round operands to 22 bits in two half precision halves. That they do is held by the 2-norm of the errors,
# in test_gpu_operator_precision.py: a sum of random terms is far below its magnitudes.
SCAN_Y = {"bf16": 2 ** -7 + 2 ** -14, "f32": 8 * 2 ** -16}
SCAN_STATE = 4 * 2 ** -16
HALF_STEP = {"bf16": 2 ** -8, "f32": 2 ** -24}


def adapters(x, weight, bias, down, up, ranks, row_adapter, row_scale):
    """y and the tolerance's parts: the magnitudes of the shared and of the low-rank product."""
    y = x.to(F) @ weight.to(F).t()
    shared = x.to(F).abs() @ weight.to(F).abs().t()
    if bias is not None:
        y, shared = y + bias.to(F), shared + bias.to(F).abs()
    low = torch.zeros_like(y)
    for r in range(x.shape[0]):
        a = -1 if row_adapter is None else int(row_adapter[r])
        if a < 0:
            continue
        n = down.shape[1] if ranks is None else min(max(int(ranks[a]), 0), down.shape[1])
        s = 1.0 if row_scale is None else float(row_scale[r])
        D, U = down[a, :n].to(F), up[a, :, :n].to(F)
        y[r] += s * (U @ (D @ x[r].to(F)))
        low[r] = abs(s) * (U.abs() @ (D.abs() @ x[r].to(F).abs()))
    return y, shared, low


def adapters_tol(y, shared, low, dtype, K, R):
    # float32 sums of K and of R terms; in bf16 the low-rank value enters its product as two halves (2^-16)
    return HALF_STEP[dtype] * y.abs() + (K + 64) * 2 ** -24 * shared + ((K + R + 64) * 2 ** -24 + 2 ** -15) * low


def distill(logits, ids, teacher, tau, models, row_grad=None):
    """row losses, means by model, gradient, and the tolerance factor of each row (times 2^-24)."""
    n, V = logits.shape
    z = logits.to(F) / tau
    row, grad, width = torch.zeros(n, dtype=F), torch.zeros(n, V, dtype=F), torch.zeros(n, dtype=F)
    scored = torch.zeros(n, dtype=torch.bool)
    for r in range(n):
        have = [j for j in range(ids.shape[1]) if ids[r, j] >= 0 and teacher[r, j] != -float("inf")]
        if not have:
            continue
        scored[r] = True
        t, at = teacher[r, have].to(F) / tau, ids[r, have].long()
        logp = torch.log_softmax(t, 0)
        p = torch.exp(logp)
        logq = torch.log_softmax(z[r], 0)
        terms = torch.where(p > 0, p * (logp - logq[at]), torch.zeros_like(p))
        row[r] = tau * tau * terms.sum()
        g = torch.exp(logq)
        g.index_add_(0, at, -p)
        grad[r] = g * tau * (1.0 if row_grad is None else float(row_grad[r]))
        finite = z[r][torch.isfinite(z[r])]
        width[r] = V / 64 + 64 + 32 * (1 + float(finite.max() - finite.min()) + float(t.max() - t.min()))
    each = row.view(models, -1).sum(1) / scored.view(models, -1).sum(1)
    return row, each, grad, width
