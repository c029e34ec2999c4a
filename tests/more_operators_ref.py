"""Plain 64-bit definitions of the delta rule, the token scores and the 4-bit format, and what a rounding may act on.

All functions take CPU tensors of any float type and compute in double from the formulas of include/cdrge.h.
"""
from __future__ import annotations

import math

import torch

F = torch.float64
HALF_STEP = {"bf16": 2 ** -8, "f32": 2 ** -24}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def delta(q, k, v, dt, beta, decay, dt_bias, heads, groups, key_dim, value_dim, bounds, q_scale, eps=1e-6, state_in=None,
          positions=None):
    """Sequences bounds[i] = (first, end) of the rows; state_in[i] [heads, value_dim, key_dim]. Returns y, for each element
    of y what an error of one part acts on, and per sequence (state, the same for it).

    A token's map S -> a S (1 - b k' k'^T) does not lengthen (|k'| <= 1, 0 < b < 1, a <= 1), so an error of one part of
    what a token forms, |a S| + |b v|, stays at most that and adds to the others': E_t = a E_{t-1} + |a S| + |b v|, by
    head, in the Frobenius norm. y_t = S_t q' then has |q'| E_t."""
    n, rep = q.shape[0], heads // groups

    def unit(x):
        x = x.to(F).view(n, groups, key_dim)
        return (x / torch.sqrt((x * x).sum(2, keepdim=True) + eps)).repeat_interleave(rep, 1)

    qn, kn, vv = unit(q) * q_scale, unit(k), v.to(F).view(n, heads, value_dim)
    step = torch.nn.functional.softplus(dt.to(F) + (0 if dt_bias is None else dt_bias.to(F)), threshold=1e9)
    a, b = torch.exp(step * decay.to(F)), torch.sigmoid(beta.to(F))
    y, part, carried = torch.zeros(n, heads, value_dim, dtype=F), torch.zeros(n, heads, dtype=F), []
    for i, (first, end) in enumerate(bounds):
        S = torch.zeros(heads, value_dim, key_dim, dtype=F)
        if positions is not None and int(positions[i]) > 0:
            S = state_in[i].to(F).clone()
        E = torch.zeros(heads, dtype=F)
        for t in range(first, end):
            S = S * a[t][:, None, None]
            E = a[t] * E + S.flatten(1).norm(dim=1) + b[t] * vv[t].norm(dim=1)
            S = S + ((vv[t] - (S * kn[t][:, None, :]).sum(2)) * b[t][:, None])[:, :, None] * kn[t][:, None, :]
            y[t] = (S * qn[t][:, None, :]).sum(2)
            part[t] = qn[t].norm(dim=1) * (E + S.flatten(1).norm(dim=1))
        carried.append((S, E))
    return y.view(n, -1), part.repeat_interleave(value_dim, 1), carried


# What a token's parts may be off by. Sums of key_dim and of up to 64 terms, in float32 and of operands of 24 bits: a term's
# product and every addition it passes is off by 2^-24, with the gates' few roundings (32 of them, of exponentials whose
# arguments are off by a rounding each).
def delta_eps(key_dim):
    return (2 * key_dim + 4 * 64 + 32) * 2 ** -24


# In bf16 y's operands may be of 16 bits: the state's and the corrected values' (half a step of 2^-16 each way and the
# product of the two rests), over the state and up to 64 corrections.
def delta_tol(y, part, dtype, key_dim):
    return HALF_STEP[dtype] * y.abs() + (delta_eps(key_dim) + (2 ** -14 if dtype == "bf16" else 0)) * part


def scores(logits, tokens, tau):
    """logprob, entropy, gradients of both [rows, vocab], all in double."""
    z = logits.to(F) / tau
    logp = torch.log_softmax(z, 1)
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    entropy = -plogp.sum(1)
    pad = tokens < 0
    at = tokens.clamp(0, logits.shape[1] - 1).long()[:, None]
    lp = torch.gather(logp, 1, at)[:, 0]
    d_lp = (torch.zeros_like(p).scatter_(1, at, 1.0) - p) / tau
    d_h = -(plogp + p * entropy[:, None]) / tau
    return torch.where(pad, torch.zeros_like(lp), lp), entropy, d_lp.masked_fill(pad[:, None], 0.0), d_h


def top(logits, k):
    """The k largest logits' ids, equal ones from the lowest id on; -1 past the last that is not minus infinity."""
    out = torch.full((logits.shape[0], k), -1, dtype=torch.int32)
    for r in range(logits.shape[0]):
        row = [(-float(x) + 0.0, i) for i, x in enumerate(logits[r].double().tolist()) if x != -math.inf]
        ids = [i for _, i in sorted(row)[:k]]
        out[r, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return out


GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mx_quantize(x):
    """codes [rows, 16 blocks] and scales [rows, blocks]: each value's nearest of the grid, the even code of two."""
    rows, K = x.shape
    v = torch.nn.functional.pad(x.to(F), (0, -K % 32)).view(rows, -1, 32)
    bad = ~torch.isfinite(v).all(2)
    v = torch.where(bad[:, :, None], torch.zeros_like(v), v)
    most = v.abs().amax(2)
    e = torch.where(most > 0, (torch.frexp(most)[1] - 3).clamp(min=-127), torch.full_like(most, -127).int()).int()
    apart = (torch.tensor(GRID, dtype=F) - torch.ldexp(v.abs(), -e[:, :, None])[..., None]).abs()
    nearest = apart == apart.amin(3, keepdim=True)
    code = torch.where(nearest, torch.arange(8) % 2, torch.full((8,), 2)).argmin(3)
    code = torch.where(v < 0, code + 8, code).to(torch.uint8)
    code = torch.where(bad[:, :, None], torch.zeros_like(code), code).view(rows, -1, 2)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), scales


def mx_values(codes, scales, K):
    rows, blocks = scales.shape
    code = torch.stack([codes & 15, codes >> 4], 2).view(rows, blocks, 32).long()
    size = torch.tensor(GRID, dtype=F)[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    v = torch.ldexp(size, scales.to(torch.int32)[:, :, None] - 127)
    v = torch.where((scales == 255)[:, :, None], torch.full_like(v, math.nan), v)
    return v.view(rows, blocks * 32)[:, :K]
