"""The attention's plain 64-bit form with the tolerance of each row from the errors of each
token's own score, for rows whose tokens are of very unequal size: a key of no weight does
not loosen it.

Base-2 scores.  Token t's score is off by at most d_t = 2^-19 B_t, B_t the sum of |q_d k_td|
in the score's units (tile_ref).  With p the exact weights and m the heaviest token, the
weights stand to that one's as p_t 2^e_t, |e_t| <= d_t + d_m (0 for m itself), so each is off
by r_t = p_t (2^(d_t + d_m) - 1) at most, their sum by R = sum r_t, and an output
sum p_t v_t by (sum r_t |v_t| + R |out|) / (1 - R).  The weights' and sums' own roundings add
2^-18 of sum p_t |v_t| (16-bit weights of bf16 outputs 2^-11 more).  Where R is a half or
more the scores' errors decide between tokens: such a row says nothing."""
import math

import torch

import tile_ref as ref


def attend(q, k, v, lims, sm=ref.SM, bf16=False):
    """(out [m, 128], tolerance [m, 128], decided [m]) of query rows q [m, 128], row i over the tokens t < lims[i] (one at
    least)."""
    qd, unit = ref.q_values(q), sm * ref.LOG2E
    seen = torch.arange(k.shape[0], device=k.device)[None] < lims[:, None]
    s = torch.where(seen, qd @ k.T * unit, -math.inf)
    s = s - s.amax(1, keepdim=True)
    d = torch.where(seen, qd.abs() @ k.abs().T * abs(unit), 0.0) * 2.0 ** -19
    top = s.argmax(1, keepdim=True)
    off = (d + d.gather(1, top)).scatter(1, top, 0.0)
    p = torch.exp2(s)
    total = p.sum(1, keepdim=True)
    r = (torch.exp2(s + off) - p) / total
    p = p / total
    R = r.sum(1, keepdim=True)
    out, size = p @ v, p @ v.abs()
    decided = (R < 0.5)[:, 0]
    tol = (r @ v.abs() + R * out.abs()) / (1 - R) + (2.0 ** -18 + (2.0 ** -11 if bf16 else 0.0)) * size.amax(1, keepdim=True)
    return out, torch.where(decided[:, None], tol, math.inf), decided


def check(got, want, tol, what=""):
    ref.check(got.reshape(-1, 128), want, tol, what)


def sharp(want, tol, decided, share):
    """Whether the tolerance tells this output from others: `share` of the rows at least are decided, and of those a row of
    zeros is out of bounds, by eight times and more."""
    if decided.double().mean().item() < share:
        return False
    return bool((8 * tol[decided].amax(1) <= want[decided].abs().amax(1)).double().mean() >= share)
