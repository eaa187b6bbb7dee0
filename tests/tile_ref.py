"""Plain 64-bit forms of the prompt attention, the decode over shared prefixes and
the cache read back, on caches drawn at random, with the tolerance that their
arithmetic allows.

Tolerance of an output (base-2 scores).  A score is a sum over 128 dims of
q_d k_d times three factors: with B the largest sum of |q_d k_d| over a row's
tokens, in the score's units, it is off by at most 2^-19 B: the query as a pair
of 11-bit parts 2^-22, sixteen accumulation steps of the tensor cores that each
cut off below 2^-23 of what they hold 2^-19 together, the rest rounded into
that bound's slack (a step's cut is half as large on average).  A weight is then
off by the factor 2^(+-2^-19 B), in the numerator and the sum alike, and the sum
over the tokens (again 16 values per step) by 2^-18 of A = sum p_t |v_t|.  bf16
outputs take weights of 11 bits: 2^-11 A more.  The output's own rounding is half
a step of its type."""
import math

import torch

from int8_quantized_kv_gb300 import kvq8

SM = 1.0 / math.sqrt(128.0)
LOG2E = 1.4426950408889634


def random_cache(num_blocks, nkv, seed, spread=None):
    """N(0, 1) rows, quantised; spread: factors of the rows' sizes drawn from 2^+-spread."""
    g = torch.Generator("cuda").manual_seed(seed)

    def rows(shape, dim):
        x = torch.randn(shape, generator=g, device="cuda")
        if spread:
            at = list(shape)
            at[dim] = 1
            x = x * torch.exp2(spread * (2 * torch.rand(at, generator=g, device="cuda") - 1))
        s = x.abs().amax(dim, keepdim=True) / torch.full((1,), 127.0, device="cuda")
        return torch.round(x / s).clamp_(-127, 127).to(torch.int8), s.squeeze(dim)

    k, ks = rows((num_blocks, nkv, 256, 128), 3)
    v, vs = rows((num_blocks, nkv, 4, 128, 64), 3)
    return kvq8.KVCache(k, v, ks.contiguous(), vs.reshape(num_blocks, nkv, 256).contiguous())


def random_table(batch, max_blocks, seed, spare=2):
    n = batch * max_blocks + spare
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n, generator=g)[:batch * max_blocks].to(torch.int32).reshape(batch, max_blocks).cuda(), n


def rows64(cache, blocks, h, t):
    """K and V values of positions t through a block-table row, kv head h."""
    t = t.long()
    p, s = blocks.long()[t // 256], t % 256
    d = torch.arange(128, device=t.device)
    at = ((d // 16) ^ (s[:, None] & 7)) * 16 + d % 16
    k = cache.k_pool[p, h, s].gather(1, at).double() * cache.k_scale[p, h, s].double()[:, None]
    v = cache.v_pool[p, h, s // 64, :, s % 64].double() * cache.v_scale[p, h, s].double()[:, None]
    return k, v


def q_values(q):
    """The query's 32-blocks as the values their codes stand for (non-finite blocks: zeros)."""
    x = q.float().reshape(-1, 4, 32)
    x = torch.where(torch.isfinite(x).all(-1, keepdim=True), x, torch.zeros_like(x))
    m = x.abs().amax(-1, keepdim=True)
    m = torch.where(m < 1e-6, torch.ones_like(m), m)
    c = torch.round(x * (torch.full_like(m, 127.0) / m)).clamp(-128, 127)
    inv = torch.full_like(m, 1.0) / torch.full_like(m, 127.0)
    return (c.double() * (m * inv).double()).reshape(q.shape)


def attend(q, k, v, lims, sm=SM, bf16=False):
    """(out [m, 128], tolerance [m, 1] before the output's own rounding) of query rows q [m, 128],
    row i over the tokens t < lims[i] (none: 0)."""
    qd = q_values(q)
    t = torch.arange(k.shape[0], device=k.device)
    seen = t[None] < lims[:, None]
    s = torch.where(seen, qd @ k.T * (sm * LOG2E), -math.inf)
    p = torch.where(seen, torch.exp2(s - s.amax(1, keepdim=True)), 0.0)
    p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    size = torch.where(seen, qd.abs() @ k.abs().T * abs(sm * LOG2E), 0.0)
    B = size.amax(1, keepdim=True) if k.shape[0] else torch.zeros_like(qd[:, :1])
    A = (p @ v.abs()).amax(1, keepdim=True)
    grow = torch.exp2(2 * 2.0 ** -19 * B) - 1
    return p @ v, A * (grow + 2.0 ** -18 + (2.0 ** -11 if bf16 else 0.0))


def check(got, want, tol, what=""):
    """got: outputs of any type; want, tol in 64 bits."""
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps / 2   # half a subnormal step
    d = (got.double() - want).abs()
    ok = d <= tol + half * (want.abs() + tol) + tiny
    if not bool(ok.all()):
        r = (d / (tol + half * want.abs() + tiny)).max().item()
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {r:.3g} times the tolerance; first at {i}: got {got.flatten()[i].item()!r}, "
                             f"want {want.flatten()[i].item()!r}; {int((~ok).sum())} of {ok.numel()} off")
