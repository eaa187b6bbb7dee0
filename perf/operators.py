"""The operators around the int8 KV cache: what is measured of them.

Each case is one call of one operator (key "op"):

  norm_rope  norm_rope_append: per-head norm of queries and keys, position
             rotation and quantise-append of K and V, in one pass
  window     decode_attn_window / decode_step_window: one new token over a
             sliding window and the first tokens (sinks)
  weights    decode_attn_weights / decode_step_weights: one new token over the
             whole context, with the attention weight of every token added up
  evict      evict: the tokens of largest accumulated weight, the first and the
             last ones are kept, compacted into other cache blocks

With own = False, run() computes them by elementary torch operations on the
same cache layout; with own = True through the framework's binding.
"""
import math

import torch

own = False

HD, BS = 128, 256
SM = 1.0 / math.sqrt(HD)
EPS = 1e-6
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # the smallest call: one sequence, one token, before every layer's decode
        dict(name="norm_rope_token_b1", op="norm_rope", batch=1, n_new=1, nqh=16, nkv=8, dtype="bf16", start=4000,
             ragged=False, interleaved=False, norm=True, moved=0),
        # a serving batch's step after evictions (positions run ahead of the slots)
        dict(name="norm_rope_token_b64", op="norm_rope", batch=64, n_new=1, nqh=32, nkv=8, dtype="fp32", start=1531,
             ragged=False, interleaved=False, norm=True, moved=20000),
        # padded prompts of unequal length, appended behind a prefix of odd length
        dict(name="norm_rope_ragged", op="norm_rope", batch=6, n_new=1111, nqh=32, nkv=8, dtype="bf16", start=77,
             ragged=True, interleaved=False, norm=True, moved=0),
        # a batch of long prompts
        dict(name="norm_rope_prefill", op="norm_rope", batch=8, n_new=4096, nqh=16, nkv=8, dtype="fp32", start=0,
             ragged=False, interleaved=False, norm=True, moved=0),
        # one sequence, a short window: latency
        dict(name="window_b1", op="window", batch=1, nqh=32, nkv=8, ctx_lo=5000, ctx_hi=5000, window=1024, sinks=4,
             step=False),
        # the layers of one step folded into the batch, with the new token's append
        dict(name="window_28layers_step", op="window", batch=28, nqh=16, nkv=8, ctx_lo=8192, ctx_hi=8192,
             window=4096, sinks=4, step=True),
        # a ragged serving batch: some contexts shorter than the window
        dict(name="window_b64_ragged", op="window", batch=64, nqh=32, nkv=8, ctx_lo=512, ctx_hi=32768, window=4096,
             sinks=16, step=False),
        # one short odd sequence, wide groups
        dict(name="weights_b1_odd", op="weights", batch=1, nqh=64, nkv=8, ctx_lo=1401, ctx_hi=1401, step=False),
        # 28 layers at 8K, with the new token's append
        dict(name="weights_28layers_step", op="weights", batch=28, nqh=16, nkv=8, ctx_lo=8192, ctx_hi=8192, step=True),
        # the largest: four 128K contexts
        dict(name="weights_b4_128k", op="weights", batch=4, nqh=32, nkv=8, ctx_lo=131072, ctx_hi=131072, step=False),
        # one sequence past its budget by less than a block
        dict(name="evict_b1", op="evict", batch=1, nkv=8, ctx_lo=2200, ctx_hi=2200, keep=2048, first=4, recent=512),
        # 28 layers halved
        dict(name="evict_28layers", op="evict", batch=28, nkv=8, ctx_lo=8192, ctx_hi=8192, keep=4096, first=4,
             recent=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "window", "weights", "evict"])
    nqh, nkv = rng.choice([(16, 8), (32, 8), (64, 8), (8, 8), (8, 2), (5, 5), (12, 3)])
    if op == "norm_rope":
        n_new = 1 if rng.random() < 0.35 else _log(rng, 2, 4096)
        batch = _log(rng, 1, max(1, min(64, 8 * 4096 * 32 // (n_new * (nqh + 2 * nkv)))))
        return dict(op=op, batch=batch, n_new=n_new, nqh=nqh, nkv=nkv, dtype=rng.choice(sorted(DTYPES)),
                    start=rng.choice([0, rng.randrange(1, 5000)]), ragged=n_new > 1 and rng.random() < 0.5,
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, moved=rng.choice([0, rng.randrange(1, 60000)]))
    batch = _log(rng, 1, 64)
    rows = (1 if op == "evict" else 4) * 131072 * 8             # an evicted row is read and written
    hi = _log(rng, 1, min(131072, rows // (batch * nkv)))
    lo = hi if rng.random() < 0.4 else rng.randrange(1, hi + 1)
    c = dict(op=op, batch=batch, nkv=nkv, ctx_lo=lo, ctx_hi=hi)
    if op == "evict":
        keep = rng.randrange(1, hi + 1)
        first = min(keep, rng.choice([0, 1, 4, 16]))
        return dict(c, keep=keep, first=first, recent=rng.randrange(0, keep - first + 1))
    c.update(nqh=nqh, step=rng.random() < 0.5)
    if op == "window":
        c.update(window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 16, 100, 700]))
    return c


# ----------------------------------------------------------------- inputs ---
def _lens(c):
    """Context lengths, from ctx_lo to ctx_hi (the case alone says them)."""
    b, lo, hi = c["batch"], c["ctx_lo"], c["ctx_hi"]
    return [hi if b == 1 else lo + (hi - lo) * ((i * 37) % b) // (b - 1 if math.gcd(37, b) == 1 else b) for i in range(b)]


def _n_tokens(c):
    return [c["n_new"] if not c["ragged"] else 1 + (c["n_new"] - 1) * ((i * 5) % c["batch"]) // max(1, c["batch"] - 1)
            for i in range(c["batch"])]


def _quant_rows(x, dim):
    a = x.abs().amax(dim, keepdim=True) / 127.0
    return torch.round(x / a).clamp_(-127, 127).to(torch.int8), a.squeeze(dim)


def _cache(g, num_blocks, nkv):
    """Pools holding quantised N(0, 1) rows in the cache's own order (the K
    rows' chunk order needs no permutation: the values are alike anyhow)."""
    dev = "cuda"
    kp = torch.empty((num_blocks, nkv, BS, HD), dtype=torch.int8, device=dev)
    vp = torch.empty((num_blocks, nkv, 4, HD, 64), dtype=torch.int8, device=dev)
    ks = torch.empty((num_blocks, nkv, BS), device=dev)
    vs = torch.empty((num_blocks, nkv, BS), device=dev)
    per = max(1, (1 << 26) // (nkv * BS * HD))
    for i in range(0, num_blocks, per):
        n = min(per, num_blocks - i)
        kp[i:i + n], ks[i:i + n] = _quant_rows(torch.randn((n, nkv, BS, HD), generator=g, device=dev), 3)
        v, s = _quant_rows(torch.randn((n, nkv, 4, HD, 64), generator=g, device=dev), 3)
        vp[i:i + n], vs[i:i + n] = v, s.reshape(n, nkv, BS)
    return kp, vp, ks, vs


def _inv_freq(device):
    return 1.0 / (1e6 ** (torch.arange(HD // 2, dtype=torch.float64, device=device) / (HD // 2)))


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(dev).manual_seed(seed * 7919 + 13)
    st = {"case": c}
    batch, nkv = c["batch"], c["nkv"]
    if c["op"] == "norm_rope":
        nqh, n = c["nqh"], c["n_new"]
        width = (nqh + 2 * nkv) * HD
        x = torch.randn((batch, n, width), generator=g, device=dev)
        x *= 0.5 + 2.5 * torch.rand((width,), generator=g, device=dev)        # channels differ in spread
        x = x.to(DTYPES[c["dtype"]])
        st["q"] = x[..., :nqh * HD].unflatten(-1, (nqh, HD))
        st["k"] = x[..., nqh * HD:(nqh + nkv) * HD].unflatten(-1, (nkv, HD))
        st["v"] = x[..., (nqh + nkv) * HD:].unflatten(-1, (nkv, HD))
        st["qw"] = 1.0 + 0.2 * torch.randn(HD, generator=g, device=dev) if c["norm"] else None
        st["kw"] = 1.0 + 0.2 * torch.randn(HD, generator=g, device=dev) if c["norm"] else None
        n_pos = c["start"] + c["moved"] + n
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * _inv_freq(dev)
        st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["start"] = torch.full((batch,), c["start"], dtype=torch.int32, device=dev)
        st["positions"] = (c["start"] + c["moved"] + torch.arange(n, dtype=torch.int32, device=dev)).expand(batch, n).contiguous()
        st["n_tokens"] = torch.tensor(_n_tokens(c), dtype=torch.int32, device=dev)
        mb = (c["start"] + n + BS - 1) // BS
        nb = batch * mb
        st["table"] = torch.randperm(nb, generator=g, device=dev).to(torch.int32).reshape(batch, mb)
        st["kp"] = torch.zeros((nb, nkv, BS, HD), dtype=torch.int8, device=dev)
        st["vp"] = torch.zeros((nb, nkv, 4, HD, 64), dtype=torch.int8, device=dev)
        st["ks"], st["vs"] = torch.zeros((nb, nkv, BS), device=dev), torch.zeros((nb, nkv, BS), device=dev)
        st["ws"] = torch.rand((nb, nkv, BS), generator=g, device=dev)
        st["out"] = torch.zeros((batch, n, nqh, HD), device=dev)
    else:
        lens = _lens(c)
        mb = max(1, (max(lens) + BS - 1) // BS)
        nb = batch * mb
        dmb = (c["keep"] + BS - 1) // BS if c["op"] == "evict" else 0
        ids = torch.randperm(nb + batch * dmb, generator=g, device=dev).to(torch.int32)
        st["table"] = ids[:nb].reshape(batch, mb).contiguous()
        st["kp"], st["vp"], st["ks"], st["vs"] = _cache(g, nb + batch * dmb, nkv)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        if c["op"] == "evict":
            # accumulated weights: heavy-tailed, with many ties at zero
            w = torch.rand((nb + batch * dmb, nkv, BS), generator=g, device=dev)
            st["ws"] = torch.where(w > 0.2, w.pow(-0.7) - 1.0, torch.zeros_like(w))
            st["dst"] = ids[nb:].reshape(batch, dmb).contiguous()
            st["kept"] = torch.zeros((batch, nkv, c["keep"]), dtype=torch.int32, device=dev)
            st["new_lens"] = torch.zeros((batch,), dtype=torch.int32, device=dev)
        else:
            nqh = c["nqh"]
            st["q"] = 1.5 * torch.randn((batch, nqh, HD), generator=g, device=dev)
            st["k_new"] = torch.randn((batch, nkv, HD), generator=g, device=dev)
            st["v_new"] = torch.randn((batch, nkv, HD), generator=g, device=dev)
            st["out"] = torch.zeros((batch, nqh, HD), device=dev)
            if c["op"] == "window":
                st["windows"] = torch.full((batch,), c["window"], dtype=torch.int32, device=dev)
            else:
                st["ws"] = torch.rand((nb, nkv, BS), generator=g, device=dev)
    if own:
        from int8_quantized_kv_gb300 import kvq8
        st["kvq8"] = kvq8
        st["cache"] = kvq8.KVCache(st["kp"], st["vp"], st["ks"], st["vs"])
        if c["op"] == "window":
            st["work"] = kvq8.alloc_workspace(batch, c["nqh"], nkv, st["table"].shape[1])
        elif c["op"] == "weights":
            st["work"] = kvq8.alloc_weights_workspace(batch, c["nqh"], nkv, st["table"].shape[1])
    return st


# -------------------------------------------------------- the plain forms ---
def _dequant_q(q):
    """The query in 32-value blocks, as the values its codes stand for."""
    x = q.unflatten(-1, (HD // 32, 32))
    m = x.abs().amax(-1, keepdim=True)
    m = torch.where(m < 1e-6, torch.ones_like(m), m)
    codes = torch.round(x * (127.0 / m)).clamp(-128, 127)
    inv127 = torch.full((), 127.0, device=q.device).reciprocal()
    return (codes * (m * inv127)).flatten(-2)


def _row_codes(x):
    """The int8 rule of a K/V row in 32 bits: (codes, scale)."""
    s = x.abs().amax(-1, keepdim=True) / 127.0
    codes = torch.where(s == 0, torch.zeros_like(x), torch.round(x / s)).clamp(-127, 127)
    return codes.to(torch.int8), s.squeeze(-1)


def _chunks(slot):
    """Byte places of the 128 dims of the K row in a slot."""
    d = torch.arange(HD, device=slot.device)
    return ((d // 16) ^ (slot[..., None] & 7)) * 16 + d % 16


def _k_rows(st, phys, slot):
    """K codes [b, n, h, 128] in dim order of the places (phys, slot) [b, n]."""
    rows = st["kp"][phys, :, slot]
    return rows.gather(-1, _chunks(slot)[:, :, None, :].expand_as(rows))


def _put_k(st, phys, slot, codes):
    rows = torch.empty_like(codes).scatter_(-1, _chunks(slot)[:, :, None, :].expand_as(codes), codes)
    st["kp"][phys, :, slot] = rows


def _v_rows(st, phys, slot):
    return st["vp"][phys, :, slot // 64, :, slot % 64]


def _put_v(st, phys, slot, codes):
    st["vp"][phys, :, slot // 64, :, slot % 64] = codes


def _place(table, t):
    """(physical block, slot) of the positions t [b, n]; positions past the table: its last entry."""
    t = t.clamp(0, table.shape[1] * BS - 1).long()
    return table.long().gather(1, t // BS), t % BS


def _plain_norm_rope(st):
    # in 64 bits: a code next to a border depends on the last bits of its value
    c = st["case"]

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.double()
        cs = st["rope"][st["positions"].long()].double()[:, :, None, :]
        cos, sin = cs[..., :HD // 2], cs[..., HD // 2:]
        a, b = (y[..., 0::2], y[..., 1::2]) if c["interleaved"] else (y[..., :HD // 2], y[..., HD // 2:])
        z = (a * cos - b * sin, b * cos + a * sin)
        return torch.stack(z, -1).flatten(-2) if c["interleaved"] else torch.cat(z, -1)

    q, k = turned(st["q"], st["qw"]), turned(st["k"], st["kw"])
    top = k.abs().amax(-1, keepdim=True)
    kc = torch.where(top == 0, torch.zeros_like(k), torch.round(127.0 * k / top)).to(torch.int8)
    ks = (top.squeeze(-1) / 127.0).float()
    vc, vs = _row_codes(st["v"].float())
    i = torch.arange(c["n_new"], device=q.device)
    real = i < st["n_tokens"][:, None]                       # rows behind a sequence's last token stay as they were
    phys, slot = _place(st["table"], st["start"][:, None] + i)
    r3, r4 = real[:, :, None], real[:, :, None, None]
    st["out"].copy_(torch.where(r4, q.float(), st["out"]))
    _put_k(st, phys, slot, torch.where(r4, kc, _k_rows(st, phys, slot)))
    _put_v(st, phys, slot, torch.where(r4, vc, _v_rows(st, phys, slot)))
    for name, new in (("ks", ks), ("vs", vs), ("ws", torch.zeros_like(ks))):
        st[name][phys, :, slot] = torch.where(r3, new, st[name][phys, :, slot])


def _plain_append(st):
    """The step's new token into position ctx_lens - 1."""
    phys, slot = _place(st["table"], st["lens"][:, None] - 1)
    for x, put, scale in (("k_new", _put_k, "ks"), ("v_new", _put_v, "vs")):
        codes, s = _row_codes(st[x][:, None])
        put(st, phys, slot, codes)
        st[scale][phys, :, slot] = s


def _plain_attention(st, phys, slot, seen):
    """(out, weights [b, h, g, n]) of the query over the places (phys, slot) where `seen` [b, n]."""
    c = st["case"]
    qd = _dequant_q(st["q"]).unflatten(1, (c["nkv"], -1))                                  # b h g d
    s = qd @ _k_rows(st, phys, slot).float().permute(0, 2, 3, 1)                           # b h g n
    s = s * (st["ks"][phys, :, slot].transpose(1, 2)[:, :, None] * SM)
    s = torch.where(seen[:, None, None], s, torch.full_like(s, -math.inf))
    w = torch.exp(s - s.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    v = _v_rows(st, phys, slot).float() * st["vs"][phys, :, slot][..., None]
    return (w @ v.permute(0, 2, 1, 3)).flatten(1, 2), w


def _plain_window(st):
    c, lens = st["case"], st["lens"][:, None].long()
    if c["step"]:
        _plain_append(st)
    dev = lens.device
    w, s = min(c["window"], c["ctx_hi"]), min(c["sinks"], c["ctx_hi"])
    t = torch.cat([torch.arange(s, device=dev).expand(c["batch"], s),
                   lens - w + torch.arange(w, device=dev)], 1)
    first = torch.arange(s + w, device=dev) < s
    # a sink inside the window counts once: as one of the window's
    seen = torch.where(first, t < lens - w, t >= 0)
    phys, slot = _place(st["table"], t)
    out, _ = _plain_attention(st, phys, slot, seen)
    st["out"].copy_(out)


def _plain_weights(st):
    c, lens = st["case"], st["lens"][:, None].long()
    if c["step"]:
        _plain_append(st)
        phys, slot = _place(st["table"], lens - 1)
        st["ws"][phys, :, slot] = 0.0                        # the new token's sum starts here
    t = torch.arange(c["ctx_hi"], device=lens.device).expand(c["batch"], c["ctx_hi"])
    phys, slot = _place(st["table"], t)
    out, w = _plain_attention(st, phys, slot, t < lens)
    st["out"].copy_(out)
    st["ws"][phys, :, slot] += w.sum(2).transpose(1, 2)      # (a weight of 0 where nothing is seen)


def _plain_evict(st):
    c, lens = st["case"], st["lens"][:, None].long()
    keep, dev, hi = c["keep"], lens.device, c["ctx_hi"]
    t = torch.arange(hi, device=dev).expand(c["batch"], hi)
    phys, slot = _place(st["table"], t)
    key = st["ws"][phys, :, slot].transpose(1, 2)                                          # b h t
    key = torch.where(((t < c["first"]) | (t >= lens - c["recent"]))[:, None], torch.full_like(key, math.inf), key)
    key = torch.where((t < lens)[:, None], key, torch.full_like(key, -math.inf))
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    n = lens.clamp(max=keep)[:, None]                                                      # b 1 1
    j = torch.arange(keep, device=dev)
    src = torch.where(j < n, best, torch.full_like(best, hi)).sort(-1).values
    real = (j < n).expand_as(src)
    st["kept"].copy_(torch.where(real, src, torch.full_like(src, -1)))
    st["new_lens"].copy_(lens[:, 0].clamp(max=keep))
    src = src.clamp(max=hi - 1)
    dp, ds = _place(st["dst"], j.expand(c["batch"], keep))
    hh = torch.arange(c["nkv"], device=dev)[None, :, None]
    sp, ss = st["table"].long()[torch.arange(c["batch"], device=dev)[:, None, None], src // BS], src % BS
    dp, ds = dp[:, None], ds[:, None]
    d = torch.arange(HD, device=dev)
    r4 = real[..., None]
    k = st["kp"][sp[..., None], hh[..., None], ss[..., None], _chunks(ss)]
    at = (dp[..., None], hh[..., None], ds[..., None], _chunks(ds))
    st["kp"][at] = torch.where(r4, k, st["kp"][at])
    v = st["vp"][sp[..., None], hh[..., None], (ss // 64)[..., None], d, (ss % 64)[..., None]]
    at = (dp[..., None], hh[..., None], (ds // 64)[..., None], d, (ds % 64)[..., None])
    st["vp"][at] = torch.where(r4, v, st["vp"][at])
    for name in ("ks", "vs", "ws"):
        st[name][dp, hh, ds] = torch.where(real, st[name][sp, hh, ss], st[name][dp, hh, ds])


# -------------------------------------------------------------------- run ---
def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        kvq8 = st["kvq8"]
        if op == "norm_rope":
            kvq8.norm_rope_append(st["q"], st["k"], st["v"], st["qw"], st["kw"], EPS, st["rope"], st["start"],
                                  st["table"], st["cache"], st["out"], positions=st["positions"],
                                  n_tokens=st["n_tokens"], interleaved=c["interleaved"], weight_sum=st["ws"])
        elif op == "window":
            if c["step"]:
                kvq8.decode_step_window(st["q"], st["k_new"], st["v_new"], st["cache"], st["table"], st["lens"],
                                        st["windows"], c["sinks"], st["out"], st["work"])
            else:
                kvq8.decode_attn_window(st["q"], st["cache"], st["table"], st["lens"], st["windows"], c["sinks"],
                                        st["out"], st["work"])
        elif op == "weights":
            if c["step"]:
                kvq8.decode_step_weights(st["q"], st["k_new"], st["v_new"], st["cache"], st["table"], st["lens"],
                                         st["out"], st["ws"], st["work"])
            else:
                kvq8.decode_attn_weights(st["q"], st["cache"], st["table"], st["lens"], st["out"], st["ws"],
                                         st["work"])
        else:
            kvq8.evict(st["cache"], st["ws"], st["table"], st["lens"], c["keep"], st["dst"], st["kept"],
                       st["new_lens"], n_first=c["first"], n_recent=c["recent"])
    else:
        {"norm_rope": _plain_norm_rope, "window": _plain_window, "weights": _plain_weights, "evict": _plain_evict}[op](st)
    # int8 codes stand for themselves; their scales are outputs beside them
    pools = {"k_codes": st["kp"], "v_codes": st["vp"], "k_scale": st["ks"], "v_scale": st["vs"]}
    if op == "norm_rope":
        return {"q": st["out"], "weight_sum": st["ws"], **pools}
    if op == "evict":
        return {"kept": st["kept"], "new_lens": st["new_lens"], "weight_sum": st["ws"], **pools}
    got = {"out": st["out"]}
    if op == "weights":
        got["weight_sum"] = st["ws"]
    return {**got, **pools} if c["step"] else got


def work(case):
    c = case
    if c["op"] == "norm_rope":
        n = sum(_n_tokens(c))
        size = 4 if c["dtype"] == "fp32" else 2
        heads = c["nqh"] + 2 * c["nkv"]
        return {"bytes": n * (heads * HD * size + c["nqh"] * HD * 4 + c["nkv"] * (2 * HD + 12) + HD * 4),
                "flops": n * (c["nqh"] + c["nkv"]) * HD * 8}
    nkv = c["nkv"]
    if c["op"] == "evict":
        return {"bytes": sum(nkv * (4 * n + min(n, c["keep"]) * (2 * (2 * HD + 8) + 4 + 4)) for n in _lens(c)),
                "flops": sum(nkv * n for n in _lens(c))}
    seen = sum(min(n, c["sinks"] + c["window"]) if c["op"] == "window" else n for n in _lens(c))
    per = 2 * HD + 8 + (8 if c["op"] == "weights" else 0)
    new = c["batch"] * nkv * (2 * HD * 4 + 2 * HD + 8) if c["step"] else 0
    return {"bytes": seen * nkv * per + 2 * c["batch"] * c["nqh"] * HD * 4 + new, "flops": seen * c["nqh"] * HD * 4}


# --------------------------------------------- the definitions in 64 bits ---
def exact(case, seed):
    c, st = case, prepare(case, seed)
    dev = "cuda"
    batch, nkv = c["batch"], c["nkv"]
    place = lambda b, t: (st["table"][b, t // BS].long(), t % BS)  # noqa: E731
    if c["op"] == "norm_rope":
        # rotation as a product of complex numbers, its angles from the positions
        for b, n in enumerate(_n_tokens(c)):
            turn = torch.exp(1j * st["positions"][b, :n].double()[:, None, None] * _inv_freq(dev))
            res = []
            for x, w in ((st["q"][b, :n], st["qw"]), (st["k"][b, :n], st["kw"])):
                x = x.double()
                if w is not None:
                    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / HD + EPS) * w.double()
                pairs = x.reshape(*x.shape[:-1], 64, 2) if c["interleaved"] else x.reshape(*x.shape[:-1], 2, 64).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                res.append((z if c["interleaved"] else z.transpose(-1, -2)).reshape(x.shape))
            p, s = place(b, c["start"] + torch.arange(n, device=dev))
            st["out"] = st["out"].double()
            st["out"][b, :n] = res[0]
            for name, v in (("ks", res[1]), ("vs", st["v"][b, :n].double())):
                st[name] = st[name].double()
                st[name][p, :, s] = v.abs().amax(-1) / 127.0
            st["ws"][p, :, s] = 0.0
        return {"q": st["out"], "weight_sum": st["ws"].double(), "k_codes": None, "v_codes": None,
                "k_scale": st["ks"], "v_scale": st["vs"]}
    lens = _lens(c)
    if c["op"] == "evict":
        ws, ks, vs = st["ws"], st["ks"], st["vs"]
        kept = []
        for b, n in enumerate(lens):
            for h in range(nkv):
                p, s = place(b, torch.arange(n, device=dev))
                w = ws[p, h, s].double()
                w[:c["first"]] = 1e300
                w[max(0, n - c["recent"]):] = 1e300
                # the m-th largest value; what is above it stays, and of its equals the first ones
                m = min(n, c["keep"])
                edge = torch.kthvalue(w, n - m + 1).values
                same = (w == edge).nonzero()[:, 0]
                over = (w > edge).nonzero()[:, 0]
                src = torch.cat([over, same[:m - len(over)]]).sort().values
                kept.append((b, h, src))
        new = [x.clone() for x in (ws, ks, vs)]
        for b, h, src in kept:
            p, s = place(b, src)
            j = torch.arange(len(src), device=dev)
            for x, y in zip(new, (ws, ks, vs)):
                x[st["dst"][b, j // BS].long(), h, j % BS] = y[p, h, s]
        return {"kept": None, "new_lens": None, "weight_sum": new[0].double(), "k_codes": None, "v_codes": None,
                "k_scale": new[1].double(), "v_scale": new[2].double()}
    G = c["nqh"] // nkv
    out = torch.zeros((batch, c["nqh"], HD), dtype=torch.float64, device=dev)
    sums = st["ws"].double() if c["op"] == "weights" else None
    perm = torch.tensor([[(((d // 16) ^ r) * 16 + d % 16) for d in range(HD)] for r in range(8)], device=dev)
    # the codes of the query and the new token are those of the 32-bit rules
    qb = st["q"].reshape(batch, c["nqh"], 4, 32)
    top = qb.abs().amax(-1, keepdim=True)
    top = torch.where(top < 1e-6, 1.0, top)
    qd = (torch.round(qb * (127.0 / top)).double() * top.double() / 127.0).reshape(batch, c["nqh"], HD)
    scales = {"ks": st["ks"].double(), "vs": st["vs"].double()}
    for b, n in enumerate(lens):
        t = torch.arange(n, device=dev)
        if c["op"] == "window":
            t = t[(t < c["sinks"]) | (t >= n - c["window"])]
        p, s = place(b, t)
        if c["step"]:
            for x, name in (("k_new", "ks"), ("v_new", "vs")):
                scales[name][p[-1], :, s[-1]] = st[x][b].double().abs().amax(-1) / 127.0
        for h in range(nkv):
            k = st["kp"][p, h, s].gather(1, perm[s % 8]).double() * st["ks"][p, h, s].double()[:, None]
            v = st["vp"][p, h, s // 64, :, s % 64].double() * st["vs"][p, h, s].double()[:, None]
            if c["step"]:
                for x, rows in (("k_new", k), ("v_new", v)):
                    y = st[x][b, h]
                    a = y.abs().max() / 127.0
                    rows[-1] = torch.round(y / a).double() * a.double()
            pr = torch.softmax(qd[b, h * G:(h + 1) * G] @ k.T * SM, -1)
            out[b, h * G:(h + 1) * G] = pr @ v
            if sums is not None:
                if c["step"]:
                    sums[p[-1], h, s[-1]] = 0.0
                sums[p, h, s] += pr.sum(0)
    got = {"out": out}
    if sums is not None:
        got["weight_sum"] = sums
    if c["step"]:
        got.update(k_codes=None, v_codes=None, k_scale=scales["ks"], v_scale=scales["vs"])
    return got
