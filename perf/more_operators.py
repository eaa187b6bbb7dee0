"""Prompts, shared prefixes and reading back: what is measured of these operators
on the int8 KV cache.

Each case is one call of one operator (key "op"):

  prompt  prompt_attn: several new query tokens per sequence, each over the
          tokens up to its own position (the cache holds them already)
  shared  decode_attn_shared / decode_step_shared: one new token per row, where
          groups of rows share their first tokens, read once for the group
  read    read_cache: K and V rows of given positions as the values their codes
          stand for

With own = False, run() computes them by elementary torch operations on the
same cache layout; with own = True through the framework's binding.
"""
import math

import torch

own = False

HD, BS = 128, 256
SM = 1.0 / math.sqrt(HD)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # five drafted tokens per sequence verified in one call, contexts of unequal length
        dict(name="prompt_verify_b8", op="prompt", batch=8, n_new=5, ragged=False, start_lo=700, start_hi=9001, nqh=32,
             nkv=8, q="fp32", out="fp32"),
        # padded prompts of unequal length behind a prefix of odd length
        dict(name="prompt_ragged", op="prompt", batch=6, n_new=1111, ragged=True, start_lo=77, start_hi=77, nqh=32,
             nkv=8, q="fp32", out="fp32"),
        # one layer's prompt of the 28-layer model, 16-bit in and out
        dict(name="prompt_4096_bf16", op="prompt", batch=1, n_new=4096, ragged=False, start_lo=0, start_hi=0, nqh=16,
             nkv=8, q="bf16", out="bf16"),
        # one chunk of a 128K prompt: the largest
        dict(name="prompt_chunk_128k", op="prompt", batch=1, n_new=512, ragged=False, start_lo=130560, start_hi=130560,
             nqh=32, nkv=8, q="fp32", out="fp32"),
        # the smallest call: four samples of one short prompt
        dict(name="shared_b4", op="shared", groups=1, rows=4, uneven=False, prefix_lo=513, prefix_hi=513, tail_lo=1,
             tail_hi=65, nqh=16, nkv=8, step=False),
        # the layers of one step folded into the batch: eight requests behind one system prompt
        dict(name="shared_28layers_step", op="shared", groups=28, rows=8, uneven=False, prefix_lo=4096, prefix_hi=4096,
             tail_lo=100, tail_hi=700, nqh=16, nkv=8, step=True),
        # several prompts with unequal numbers of samples each
        dict(name="shared_groups", op="shared", groups=5, rows=24, uneven=True, prefix_lo=900, prefix_hi=12345,
             tail_lo=1, tail_hi=2000, nqh=32, nkv=8, step=False),
        # many requests about one long document
        dict(name="shared_b128_32k", op="shared", groups=1, rows=128, uneven=False, prefix_lo=32768, prefix_hi=32768,
             tail_lo=50, tail_hi=1500, nqh=32, nkv=8, step=False),
        # one short stretch read back
        dict(name="read_b1", op="read", batch=1, n=300, ragged=False, start=77, nkv=8, out="bf16"),
        # padded rows of unequal length
        dict(name="read_ragged_bf16", op="read", batch=12, n=3000, ragged=True, start=133, nkv=8, out="bf16"),
        # the append benchmark's rows read back
        dict(name="read_b8_4096", op="read", batch=8, n=4096, ragged=False, start=0, nkv=8, out="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "shared", "shared", "read"])
    nqh, nkv = rng.choice([(16, 8), (32, 8), (64, 8), (8, 8), (8, 2), (5, 5), (12, 3)])
    kind = lambda: rng.choice(sorted(DTYPES))  # noqa: E731
    if op == "prompt":
        n = _log(rng, 1, 4096)
        # rows * context of the largest listed case, and its cache
        hi = _log(rng, n, max(n, min(131072, 512 * 131072 * 32 // (n * nqh))))
        batch = _log(rng, 1, max(1, min(64, 512 * 131072 * 32 // (n * nqh * hi), 4 * 131072 // hi)))
        hi -= n
        return dict(op=op, batch=batch, n_new=n, ragged=n > 1 and rng.random() < 0.5,
                    start_lo=hi if rng.random() < 0.4 else rng.randrange(0, hi + 1), start_hi=hi, nqh=nqh, nkv=nkv,
                    q=kind(), out=kind())
    if op == "shared":
        groups = _log(rng, 1, 28)
        rows = _log(rng, 1, max(1, 256 // groups))
        hi = _log(rng, 1, min(32768, 128 * 32768 * 32 // (groups * rows * nqh), 4 * 131072 // groups))
        t = _log(rng, 1, min(2000, max(1, 2 * 131072 // (groups * rows))))
        return dict(op=op, groups=groups, rows=rows, uneven=rng.random() < 0.5,
                    prefix_lo=hi if rng.random() < 0.5 else rng.randrange(1, hi + 1), prefix_hi=hi,
                    tail_lo=rng.randrange(1, t + 1), tail_hi=t, nqh=nqh, nkv=nkv, step=rng.random() < 0.5)
    n = _log(rng, 1, 4096)
    batch = _log(rng, 1, max(1, min(64, 8 * 4096 // n)))
    return dict(op=op, batch=batch, n=n, ragged=n > 1 and rng.random() < 0.5, start=rng.choice([0, rng.randrange(1, 5000)]),
                nkv=nkv, out=kind())


# ----------------------------------------------------------------- inputs ---
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, out of order (the case alone says them)."""
    step = next(s for s in (37, 31, 29, 23) if math.gcd(s, n) == 1)
    return [hi if n == 1 else lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _n_tokens(c, n):
    return _spread(1, n, c["batch"]) if c["ragged"] else [n] * c["batch"]


def _group_sizes(c):
    """Rows of each group: all alike, or from 1 on with the same sum of rows at most."""
    return _spread(1, c["rows"], c["groups"]) if c["uneven"] else [c["rows"]] * c["groups"]


def _shared_rows(c):
    """(group, prefix length, context length) of every row."""
    sizes, prefix = _group_sizes(c), _spread(c["prefix_lo"], c["prefix_hi"], c["groups"])
    tails = _spread(c["tail_lo"], c["tail_hi"], sum(sizes))
    group = [g for g, m in enumerate(sizes) for _ in range(m)]
    return [(g, prefix[g], prefix[g] + t) for g, t in zip(group, tails)]


def _quant_rows(x, dim):
    a = x.abs().amax(dim, keepdim=True) * (1.0 / 127.0)
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


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(dev).manual_seed(seed * 7919 + 17)
    st = {"case": c}
    nkv = c["nkv"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    if c["op"] == "shared":
        rows = _shared_rows(c)
        batch, mb = len(rows), (max(n for _, _, n in rows) + BS - 1) // BS
        # the whole blocks of a group's prefix are listed in all its rows; a prefix that ends inside a block is
        # copied into each row's own block
        first = [next(b for b, r in enumerate(rows) if r[0] == j) for j in range(c["groups"])]
        table = torch.arange(batch * mb).reshape(batch, mb)
        col = torch.arange(mb)
        lead = i32([first[r[0]] for r in rows]).long().cpu()
        full = torch.tensor([r[1] // BS for r in rows])
        table = torch.where(col < full[:, None], table[lead], table)
        used = col < torch.tensor([(r[2] + BS - 1) // BS for r in rows])[:, None]
        ids = torch.unique(table[used])
        place = torch.full((batch * mb,), -1, dtype=torch.int64)
        place[ids] = torch.randperm(len(ids), generator=torch.Generator().manual_seed(seed))
        st["table"] = torch.where(used, place[table], -1).to(torch.int32).to(dev)
        st["kp"], st["vp"], st["ks"], st["vs"] = _cache(g, len(ids), nkv)
        t, p = st["table"].long(), i32([r[1] for r in rows]).long()
        edge = t.gather(1, (p // BS).clamp(max=mb - 1)[:, None])[:, 0].clamp(min=0)
        part = torch.arange(BS, device=dev) < (p % BS)[:, None]                       # b slot
        src = edge[lead.to(dev)]
        for name in ("ks", "vs"):
            x = st[name]
            x[edge] = torch.where(part[:, None], x[src], x[edge])
        st["kp"][edge] = torch.where(part[:, None, :, None], st["kp"][src], st["kp"][edge])
        st["vp"][edge] = torch.where(part.reshape(batch, 1, 4, 1, 64), st["vp"][src], st["vp"][edge])
        sizes = _group_sizes(c)
        st["starts"] = i32([sum(sizes[:j]) for j in range(len(sizes) + 1)])
        st["shared"] = i32(_spread(c["prefix_lo"], c["prefix_hi"], c["groups"]))
        st["lens"], st["group"] = i32([r[2] for r in rows]), i32([r[0] for r in rows]).long()
        st["q"] = 1.5 * torch.randn((batch, c["nqh"], HD), generator=g, device=dev)
        st["k_new"] = torch.randn((batch, nkv, HD), generator=g, device=dev)
        st["v_new"] = torch.randn((batch, nkv, HD), generator=g, device=dev)
        st["out"] = torch.zeros((batch, c["nqh"], HD), device=dev)
    else:
        batch = c["batch"]
        n = c["n_new"] if c["op"] == "prompt" else c["n"]
        starts = _spread(c["start_lo"], c["start_hi"], batch) if c["op"] == "prompt" else [c["start"]] * batch
        mb = (max(starts) + n + BS - 1) // BS
        st["start"], st["n_tokens"] = i32(starts), i32(_n_tokens(c, n))
        st["table"] = torch.randperm(batch * mb, generator=g, device=dev).to(torch.int32).reshape(batch, mb)
        st["kp"], st["vp"], st["ks"], st["vs"] = _cache(g, batch * mb, nkv)
        kind = DTYPES[c["out"]]
        if c["op"] == "prompt":
            st["q"] = (1.5 * torch.randn((batch, n, c["nqh"], HD), generator=g, device=dev)).to(DTYPES[c["q"]])
            st["out"] = torch.zeros((batch, n, c["nqh"], HD), dtype=kind, device=dev)
        else:
            st["k"] = torch.zeros((batch, n, nkv, HD), dtype=kind, device=dev)
            st["v"] = torch.zeros((batch, n, nkv, HD), dtype=kind, device=dev)
    if own:
        from int8_quantized_kv_gb300 import kvq8
        st["kvq8"] = kvq8
        st["cache"] = kvq8.KVCache(st["kp"], st["vp"], st["ks"], st["vs"])
        if c["op"] == "prompt":
            st["work"] = kvq8.alloc_prompt_workspace(batch, n, c["nqh"], nkv, mb)
        elif c["op"] == "shared":
            st["work"] = kvq8.alloc_shared_workspace(batch, c["groups"], c["nqh"], nkv, mb)
    return st


# -------------------------------------------------------- the plain forms ---
def _over(a, x):
    """a / x of a number and a tensor, as one division per value."""
    return torch.full_like(x, a) / x


def _q_values(q):
    """The query in 32-value blocks, as the values its codes stand for."""
    x = q.float().unflatten(-1, (HD // 32, 32))
    m = x.abs().amax(-1, keepdim=True)
    m = torch.where(m < 1e-6, torch.ones_like(m), m)
    codes = torch.round(x * _over(127.0, m)).clamp(-128, 127)
    inv127 = _over(1.0, torch.full_like(m, 127.0))
    return (codes * (m * inv127)).flatten(-2)


def _row_codes(x):
    """The int8 rule of a K/V row in 32 bits: (codes, scale)."""
    m = x.abs().amax(-1, keepdim=True)
    s = m / torch.full_like(m, 127.0)
    codes = torch.where(s == 0, torch.zeros_like(x), torch.round(x / s)).clamp(-127, 127)
    return codes.to(torch.int8), s.squeeze(-1)


def _chunks(slot):
    """Byte places of the 128 dims of the K row in a slot."""
    d = torch.arange(HD, device=slot.device)
    return ((d // 16) ^ (slot[..., None] & 7)) * 16 + d % 16


def _k_codes(st, phys, slot):
    """K codes [b, n, h, 128] in dim order of the places (phys, slot) [b, n]."""
    rows = st["kp"][phys, :, slot]
    return rows.gather(-1, _chunks(slot)[:, :, None, :].expand_as(rows))


def _keys(st, phys, slot):
    return _k_codes(st, phys, slot).float() * st["ks"][phys, :, slot][..., None]


def _values(st, phys, slot):
    return st["vp"][phys, :, slot // 64, :, slot % 64].float() * st["vs"][phys, :, slot][..., None]


def _place(table, t):
    """(physical block, slot) of the positions t [b, n]; places that the table does not have: block 0."""
    t = t.clamp(0, table.shape[1] * BS - 1).long()
    return table.long().gather(1, t // BS).clamp(min=0), t % BS


def _plain_prompt(st):
    c = st["case"]
    dev, n = st["q"].device, c["n_new"]
    i = torch.arange(n, device=dev)
    t = torch.arange(st["table"].shape[1] * BS, device=dev).expand(c["batch"], -1)
    phys, slot = _place(st["table"], t)
    q = _q_values(st["q"]).unflatten(2, (c["nkv"], -1)).permute(0, 2, 3, 1, 4)             # b h g n d
    s = q.flatten(2, 3) @ _keys(st, phys, slot).permute(0, 2, 3, 1)                         # b h gn t
    s = (s * SM).unflatten(2, (-1, n))
    seen = t[:, None] <= (st["start"][:, None] + i)[:, :, None]                             # b n t
    s.masked_fill_(~seen[:, None, None], -math.inf)
    s = torch.exp_(s.sub_(s.amax(-1, keepdim=True)))
    total = s.sum(-1, keepdim=True)
    o = s.flatten(2, 3) @ _values(st, phys, slot).transpose(1, 2)
    o = (o.unflatten(2, (-1, n)) / total).permute(0, 3, 1, 2, 4).flatten(2, 3)              # b n hg d
    real = (i < st["n_tokens"][:, None])[:, :, None, None]         # rows behind a sequence's last token stay as they were
    st["out"].copy_(torch.where(real, o.to(st["out"].dtype), st["out"]))


def _plain_append(st):
    """The step's new token into position ctx_lens - 1."""
    phys, slot = _place(st["table"], st["lens"][:, None] - 1)
    codes, s = _row_codes(st["k_new"][:, None])
    st["kp"][phys, :, slot] = torch.empty_like(codes).scatter_(-1, _chunks(slot)[:, :, None, :].expand_as(codes), codes)
    st["ks"][phys, :, slot] = s
    st["vp"][phys, :, slot // 64, :, slot % 64], st["vs"][phys, :, slot] = _row_codes(st["v_new"][:, None])


def _plain_shared(st):
    c, group = st["case"], st["group"]
    if c["step"]:
        _plain_append(st)
    dev, batch = group.device, len(group)
    lens, prefix = st["lens"].long()[:, None], st["shared"].long()[group][:, None]
    q = _q_values(st["q"]).unflatten(1, (c["nkv"], -1))                                     # b h g d
    # the prefix: the rows of a group beside each other (places behind its last row repeat another's)
    starts = st["starts"].long()
    m = c["rows"]
    member = torch.arange(batch, device=dev) - starts[group]
    at = (starts[:-1, None] + torch.arange(m, device=dev)).clamp(max=batch - 1)             # j m
    t = torch.arange(c["prefix_hi"], device=dev).expand(c["groups"], -1)
    phys, slot = _place(st["table"][starts[:-1]], t)
    k, v = _keys(st, phys, slot).permute(0, 2, 3, 1), _values(st, phys, slot).transpose(1, 2)
    s1 = (q[at].transpose(1, 2).flatten(2, 3) @ k).unflatten(2, (m, -1))                    # j h m g t
    s1 = (s1 * SM).masked_fill_((t >= st["shared"][:, None])[:, None, None, None], -math.inf)
    # each row's own tokens
    own_t = prefix + torch.arange(c["tail_hi"], device=dev)
    phys, slot = _place(st["table"], own_t)
    s2 = q @ _keys(st, phys, slot).permute(0, 2, 3, 1)                                      # b h g t
    s2 = (s2 * SM).masked_fill_((own_t >= lens)[:, None, None], -math.inf)
    top1 = s1.amax(-1, keepdim=True)
    top = torch.maximum(top1.transpose(1, 2)[group, member], s2.amax(-1, keepdim=True))      # b h g 1
    w1 = torch.exp_(s1.sub_(top[at].transpose(1, 2)))
    w2 = torch.exp_(s2.sub_(top))
    o1 = (w1.flatten(2, 3) @ v).unflatten(2, (m, -1)).transpose(1, 2)[group, member]         # b h g d
    o2 = w2 @ _values(st, phys, slot).transpose(1, 2)
    total = w1.sum(-1, keepdim=True).transpose(1, 2)[group, member] + w2.sum(-1, keepdim=True)
    st["out"].copy_(((o1 + o2) / total).flatten(1, 2))


def _plain_read(st):
    i = torch.arange(st["case"]["n"], device=st["start"].device)
    phys, slot = _place(st["table"], st["start"][:, None] + i)
    real = (i < st["n_tokens"][:, None])[:, :, None, None]
    for name, rows in (("k", _keys), ("v", _values)):
        x = rows(st, phys, slot).to(st[name].dtype)
        st[name].copy_(torch.where(real, x, st[name]))


# -------------------------------------------------------------------- run ---
def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        kvq8 = st["kvq8"]
        if op == "prompt":
            kvq8.prompt_attn(st["q"], st["cache"], st["table"], st["start"], st["out"], st["work"],
                             n_tokens=st["n_tokens"])
        elif op == "shared":
            args = (st["cache"], st["table"], st["lens"], st["starts"], st["shared"], st["out"], st["work"])
            if c["step"]:
                kvq8.decode_step_shared(st["q"], st["k_new"], st["v_new"], *args)
            else:
                kvq8.decode_attn_shared(st["q"], *args)
        else:
            kvq8.read_cache(st["cache"], st["table"], st["start"], st["k"], st["v"], n_tokens=st["n_tokens"])
    else:
        {"prompt": _plain_prompt, "shared": _plain_shared, "read": _plain_read}[op](st)
    if op == "read":
        return {"k": st["k"], "v": st["v"]}
    got = {"out": st["out"]}
    if op == "shared" and c["step"]:
        # int8 codes stand for themselves; their scales are outputs beside them
        got.update(k_codes=st["kp"], v_codes=st["vp"], k_scale=st["ks"], v_scale=st["vs"])
    return got


def work(case):
    c = case
    size = lambda name: 4 if c[name] == "fp32" else 2  # noqa: E731
    per = c["nkv"] * (2 * HD + 8)
    if c["op"] == "read":
        n = sum(_n_tokens(c, c["n"]))
        return {"bytes": n * (per + 2 * c["nkv"] * HD * size("out")), "flops": n * 2 * c["nkv"] * HD}
    if c["op"] == "prompt":
        bounds = list(zip(_spread(c["start_lo"], c["start_hi"], c["batch"]), _n_tokens(c, c["n_new"])))
        rows = sum(n for _, n in bounds)
        return {"bytes": sum(p + n for p, n in bounds) * per + rows * c["nqh"] * HD * (size("q") + size("out")),
                "flops": sum(n * p + n * (n + 1) // 2 for p, n in bounds) * c["nqh"] * HD * 4}
    rows = _shared_rows(c)
    prefix = sum(_spread(c["prefix_lo"], c["prefix_hi"], c["groups"]))
    new = len(rows) * c["nkv"] * (2 * HD * 4 + 2 * HD + 8) if c["step"] else 0
    return {"bytes": (prefix + sum(n - p for _, p, n in rows)) * per + 2 * len(rows) * c["nqh"] * HD * 4 + new,
            "flops": sum(n for _, _, n in rows) * c["nqh"] * HD * 4}


# --------------------------------------------- the definitions in 64 bits ---
def exact(case, seed):
    c, st = case, prepare(case, seed)
    dev, nkv = "cuda", c["nkv"]
    perm = torch.tensor([[(((d // 16) ^ r) * 16 + d % 16) for d in range(HD)] for r in range(8)], device=dev)

    def rows64(row, h, t):
        p, s = st["table"][row, t // BS].long(), t % BS
        k = st["kp"][p, h, s].gather(1, perm[s % 8]).double() * st["ks"][p, h, s].double()[:, None]
        return k, st["vp"][p, h, s // 64, :, s % 64].double() * st["vs"][p, h, s].double()[:, None]

    if c["op"] == "read":
        got = {name: st[name].double() for name in ("k", "v")}
        for b, n in enumerate(_n_tokens(c, c["n"])):
            for h in range(nkv):
                got["k"][b, :n, h], got["v"][b, :n, h] = rows64(b, h, c["start"] + torch.arange(n, device=dev))
        return got
    G = c["nqh"] // nkv
    # the query's codes are those of the 32-bit rule
    x = st["q"].float().reshape(-1, 4, 32)
    top = x.abs().amax(2, keepdim=True)
    top[top < 1e-6] = 1.0
    factor = torch.tensor(127.0, device=dev).expand(top.shape).contiguous().div(top)
    qd = (torch.round(x * factor).double() * top.double() / 127.0).reshape(st["q"].shape)
    out = st["out"].double()
    if c["op"] == "prompt":
        starts = _spread(c["start_lo"], c["start_hi"], c["batch"])
        for b, n in enumerate(_n_tokens(c, c["n_new"])):
            t = torch.arange(starts[b] + n, device=dev)
            late = t > (starts[b] + torch.arange(n, device=dev))[:, None]
            for h in range(nkv):
                k, v = rows64(b, h, t)
                for j in range(h * G, h * G + G):
                    s = qd[b, :n, j] @ k.T * SM
                    s[late] = -math.inf
                    out[b, :n, j] = torch.softmax(s, -1) @ v
        return {"out": out}
    scales = {"ks": st["ks"].double(), "vs": st["vs"].double()}
    rows = _shared_rows(c)
    first = {}
    for b, (g, p, n) in enumerate(rows):
        first.setdefault(g, b)
    for h in range(nkv):
        seen = {}
        for b, (g, p, n) in enumerate(rows):
            if g not in seen:
                seen = {g: rows64(first[g], h, torch.arange(p, device=dev))}
            k, v = rows64(b, h, torch.arange(p, n, device=dev))
            if c["step"]:
                w, s = st["table"][b, (n - 1) // BS], (n - 1) % BS
                for y, name, r in ((st["k_new"][b, h], "ks", k), (st["v_new"][b, h], "vs", v)):
                    a = y.abs().max() / torch.tensor(127.0, device=dev)
                    r[-1] = torch.round(y / a).double() * a.double()
                    scales[name][w, h, s] = y.abs().max().double() / 127.0
            k, v = torch.cat([seen[g][0], k]), torch.cat([seen[g][1], v])
            out[b, h * G:(h + 1) * G] = torch.softmax(qd[b, h * G:(h + 1) * G] @ k.T * SM, -1) @ v
    got = {"out": out}
    if c["step"]:
        got.update(k_codes=None, v_codes=None, k_scale=scales["ks"], v_scale=scales["vs"])
    return got
