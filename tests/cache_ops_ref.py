"""Plain references of the operators around the int8 cache: their fp32 rounding
rules (1/127 and 1/qm as factors, where the append and the plain decode divide)
and the softmax in 64 bits, by the oracle, over the codes."""
import numpy as np

import oracle
from kvq8_harness import SM_SCALE

ONE, C127 = np.float32(1), np.float32(127)


def row_codes(v):
    """K/V rows: scale = max * fl(1/127), code = round_half_even(fl(v / scale)),
    non-finite rows as zeros."""
    v = np.asarray(v, np.float32)
    v = np.where(np.isfinite(v).all(-1, keepdims=True), v, np.float32(0))
    s = np.abs(v).max(-1) * (ONE / C127)
    with np.errstate(all="ignore"):
        c = np.where(s[..., None] == 0, np.float32(0), np.rint(v / s[..., None]))
    return np.clip(c, -127, 127).astype(np.int8), s


def q_codes(q):
    """Query rows in blocks of 32: code = round_half_even(fl(x * fl(fl(1/qm) * 127)))."""
    x = np.asarray(q, np.float32).reshape(*q.shape[:-1], -1, 32)
    x = np.where(np.isfinite(x).all(-1, keepdims=True), x, np.float32(0))
    m = np.abs(x).max(-1)
    m = np.where(m < np.float32(1e-6), ONE, m)
    c = np.clip(np.rint(x * ((ONE / m) * C127)[..., None]), -128, 127).astype(np.int8)
    return c.reshape(q.shape), m * (ONE / C127)


def unit_rows(k, v, step=False):
    """Codes and scales of a unit's cached rows; step: the last row was appended by a decode step."""
    rows = []
    for x in (k, v):
        c, s = oracle.kv_quantize_rows(x)
        if step:
            c[-1], s[-1] = row_codes(x[-1])
        rows += [c, s]
    return rows


def decode(q, kq, ks, vq, vs, sm_scale=SM_SCALE):
    """Output rows [G][128] over the given cached rows."""
    qi, qsc = q_codes(q)
    return oracle.decode_quantized_unit(qi, qsc, kq, ks, vq, vs, sm_scale)


def weights(q, kq, ks, sm_scale=SM_SCALE):
    """Softmax weights summed over the group's heads [L], and the largest |score| (base 2)."""
    qi, qsc = q_codes(q)
    total, most = np.zeros(len(kq)), 0.0
    for g in range(len(q)):
        s = oracle.scores_q8(qi[g], qsc[g], kq, ks, sm_scale)
        w = np.exp(s - s.max())
        total += w / w.sum()
        most = max(most, np.abs(s).max() / np.log(2))
    return total, most
