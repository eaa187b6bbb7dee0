"""The operators around the int8 cache together, as a serving loop uses them,
and on other streams, in captured graphs and with shared workspaces."""
import numpy as np
import pytest
import torch

import cache_ops_ref as ref
from int8_quantized_kv_gb300 import kvq8
from kvq8_harness import assert_close, k_rows_logical, v_rows_logical

pytestmark = pytest.mark.gpu
HD = 128


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Loop:
    """Two sequences of one layer: prompt, decode with weights, eviction, decode on."""

    def __init__(self, seed=0):
        self.nqh, self.nkv, self.batch = 8, 2, 2
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.blocks, self.dblocks = 4, 2
        ids = rng.permutation(2 * (self.blocks + self.dblocks)).astype(np.int32)
        self.table = ids[:8].reshape(2, 4)
        self.dst = ids[8:].reshape(2, 2)
        self.nb = len(ids)
        self.cache = kvq8.alloc_cache(self.nb, self.nkv)
        self.wsum = kvq8.alloc_weight_sum(self.nb, self.nkv)
        self.inv = _dev(1e4 ** (-np.arange(64) / 64.0))
        self.rope = kvq8.rope_table(self.inv, 4096)
        self.qw, self.kw = (_dev((1 + 0.2 * rng.standard_normal(HD)).astype(np.float32)) for _ in range(2))
        self.ws = kvq8.alloc_weights_workspace(2, self.nqh, self.nkv, self.blocks)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self, n):
        x = self.rng.standard_normal((2, n, self.nqh + 2 * self.nkv, HD)).astype(np.float32)
        t = torch.from_numpy(x).bfloat16().cuda()
        return t[:, :, :8], t[:, :, 8:10], t[:, :, 10:]

    def append(self, n, start, table, positions, n_tokens=None):
        q, k, v = self.rows(n)
        out = torch.zeros((2, n, self.nqh, HD), device="cuda")
        kvq8.norm_rope_append(q, k, v, self.qw, self.kw, 1e-6, self.rope, _dev(np.asarray(start, np.int32)),
                              _dev(table), self.cache, out, positions=_dev(np.asarray(positions, np.int32)),
                              n_tokens=None if n_tokens is None else _dev(np.asarray(n_tokens, np.int32)),
                              weight_sum=self.wsum, dev_status=self.status)
        return out

    def unit(self, table, b, h, L):
        """The cached rows of a unit as they stand: (kq, ks, vq, vs)."""
        t = np.arange(L)
        phys, slot = table[b, t // 256], t % 256
        c = [x.cpu().numpy() for x in self.cache]
        return (k_rows_logical(c[0], phys, h, slot), c[2][phys, h, slot], v_rows_logical(c[1], phys, h, slot),
                c[3][phys, h, slot])

    def check_decode(self, q, out, table, lens, seen=None):
        for b in range(2):
            for h in range(self.nkv):
                kq, ks, vq, vs = self.unit(table, b, h, lens[b])
                vis = np.arange(lens[b]) if seen is None else seen[b]
                want = ref.decode(q[b, h * 4:(h + 1) * 4].cpu().numpy(), kq[vis], ks[vis], vq[vis], vs[vis])
                assert_close(out[b, h * 4:(h + 1) * 4].cpu().numpy(), want, f"b={b} h={h}")


def test_prompt_decode_evict_decode(gpu_lib):
    s = Loop()
    lens = np.array([700, 333])
    s.append(700, [0, 0], s.table, np.tile(np.arange(700), (2, 1)), n_tokens=lens)
    out = torch.empty((2, s.nqh, HD), device="cuda")
    sums = np.zeros((2, s.nkv, 1024))
    pos = lens.copy()
    for step in range(6):
        q = s.append(1, lens, s.table, pos[:, None])[:, 0].contiguous()
        lens, pos = lens + 1, pos + 1
        kvq8.decode_attn_weights(q, s.cache, _dev(s.table), _dev(lens.astype(np.int32)), out, s.wsum, s.ws,
                                 dev_status=s.status)
        torch.cuda.synchronize()
        s.check_decode(q, out, s.table, lens)
        for b in range(2):
            for h in range(s.nkv):
                kq, ks, vq, vs = s.unit(s.table, b, h, lens[b])
                sums[b, h, :lens[b]] += ref.weights(q[b, h * 4:(h + 1) * 4].cpu().numpy(), kq, ks)[0]
    t = np.arange(1024)
    got = s.wsum.cpu().numpy()
    for b in range(2):
        for h in range(s.nkv):
            w = got[s.table[b, t // 256], h, t % 256]
            assert np.all(np.abs(w - sums[b, h])[:lens[b]] <= 1e-4 * sums[b, h][:lens[b]])
            assert not w[lens[b]:].any()
    # evict to 300 tokens and carry on in the new blocks
    kept = torch.empty((2, s.nkv, 300), dtype=torch.int32, device="cuda")
    new_lens = torch.empty((2,), dtype=torch.int32, device="cuda")
    before = {(b, h): s.unit(s.table, b, h, lens[b]) for b in range(2) for h in range(s.nkv)}
    kvq8.evict(s.cache, s.wsum, _dev(s.table), _dev(lens.astype(np.int32)), 300, _dev(s.dst), kept, new_lens,
               n_first=4, n_recent=64, dev_status=s.status)
    torch.cuda.synchronize()
    k, n = kept.cpu().numpy(), new_lens.cpu().numpy()
    assert n.tolist() == [300, 300]
    for (b, h), rows in before.items():
        t = np.arange(lens[b])
        w = got[s.table[b, t // 256], h, t % 256].astype(np.float64)
        w[:4] = w[lens[b] - 64:] = np.inf
        want = np.sort(np.lexsort((t, -w))[:300])
        assert np.array_equal(k[b, h], want)
        for x, y in zip(rows, s.unit(s.dst, b, h, 300)):
            assert np.array_equal(x[want], y)
    lens = n.copy()
    for step in range(3):
        q = s.append(1, lens, s.dst, pos[:, None])[:, 0].contiguous()
        lens, pos = lens + 1, pos + 1
        kvq8.decode_attn_weights(q, s.cache, _dev(s.dst), _dev(lens.astype(np.int32)), out, s.wsum,
                                 kvq8.alloc_weights_workspace(2, s.nqh, s.nkv, 2), dev_status=s.status)
        torch.cuda.synchronize()
        s.check_decode(q, out, s.dst, lens)
    # and the same cache through a window
    kvq8.decode_attn_window(q, s.cache, _dev(s.dst), _dev(lens.astype(np.int32)),
                            torch.tensor([50, 100], dtype=torch.int32, device="cuda"), 4, out,
                            kvq8.alloc_workspace(2, s.nqh, s.nkv, 2), dev_status=s.status)
    torch.cuda.synchronize()
    s.check_decode(q, out, s.dst, lens, [np.r_[0:4, lens[0] - 50:lens[0]], np.r_[0:4, lens[1] - 100:lens[1]]])
    assert int(s.status.item()) == 0


def _state(seed, lens=(900, 513), step=True):
    """Buffers of one call of each operator, made from the seed."""
    rng = np.random.default_rng(seed)
    batch, nqh, nkv, mb = len(lens), 8, 4, 4
    nb = batch * (mb + 2)
    ids = rng.permutation(nb).astype(np.int32)
    st = dict(table=_dev(ids[:batch * mb].reshape(batch, mb)), dst=_dev(ids[batch * mb:].reshape(batch, 2)),
              lens=_dev(np.array(lens, np.int32)), windows=_dev(np.array([200, 70][:batch], np.int32)))
    st["cache"] = kvq8.KVCache(_dev(rng.integers(-127, 128, (nb, nkv, 256, HD), np.int8)),
                               _dev(rng.integers(-127, 128, (nb, nkv, 4, HD, 64), np.int8)),
                               _dev(rng.random((nb, nkv, 256), np.float32) * 0.02),
                               _dev(rng.random((nb, nkv, 256), np.float32) * 0.02))
    st["wsum"] = _dev(rng.random((nb, nkv, 256), np.float32))
    for n, heads in (("q", nqh), ("k", nkv), ("v", nkv)):
        st[n] = _dev(rng.standard_normal((batch, heads, HD), np.float32))
    st["rope"] = kvq8.rope_table(_dev(1e4 ** (-np.arange(64) / 64.0)), 2048)
    st["start"] = st["lens"] - 1
    st["out"] = [torch.zeros((batch, nqh, HD), device="cuda") for _ in range(3)]
    st["kept"] = torch.zeros((batch, nkv, 300), dtype=torch.int32, device="cuda")
    st["new_lens"] = torch.zeros((batch,), dtype=torch.int32, device="cuda")
    st["ws"] = kvq8.alloc_weights_workspace(batch, nqh, nkv, mb)
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


def _all(st, stream=None):
    """One call of every operator; they share one workspace."""
    kw = dict(dev_status=st["status"], stream=stream)
    o = st["out"]
    kvq8.norm_rope_append(st["q"][:, None], st["k"][:, None], st["v"][:, None], None, None, 0.0, st["rope"],
                          st["start"], st["table"], st["cache"], o[0][:, None], weight_sum=st["wsum"], **kw)
    kvq8.decode_attn_window(o[0], st["cache"], st["table"], st["lens"], st["windows"], 4, o[1], st["ws"], **kw)
    kvq8.decode_step_weights(o[0], st["k"], st["v"], st["cache"], st["table"], st["lens"], o[2], st["wsum"], st["ws"],
                             **kw)
    kvq8.evict(st["cache"], st["wsum"], st["table"], st["lens"], 300, st["dst"], st["kept"], st["new_lens"],
               n_first=4, n_recent=30, **kw)


def _result(st):
    torch.cuda.synchronize()
    assert int(st["status"].item()) == 0
    return [x.cpu().numpy() for x in (*st["out"], st["kept"], st["new_lens"], st["wsum"], *st["cache"])]


def test_other_streams_and_graphs_give_the_same_bits(gpu_lib):
    st = _state(1)
    _all(st)
    want = _result(st)
    side = torch.cuda.Stream()
    st = _state(1)
    torch.cuda.synchronize()
    _all(st, stream=side)
    assert all(np.array_equal(x, y) for x, y in zip(_result(st), want))
    st = _state(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _all(st)
    assert all(np.array_equal(x, y) for x, y in zip(_result(st), want))
    # captured, and replayed with other contents in the same buffers
    st, other = _state(1), _state(2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _all(st)
    for src, ref in ((_state(1), want), (other, None), (_state(1), want)):
        for name in ("table", "dst", "q", "k", "v", "wsum", "lens", "start", "windows"):
            st[name].copy_(src[name])
        for x, y in zip(st["cache"], src["cache"]):
            x.copy_(y)
        g.replay()
        got = _result(st)
        if ref is None:
            _all(src)
            ref = _result(src)
        assert all(np.array_equal(x, y) for x, y in zip(got, ref))


def test_two_graphs_share_a_workspace(gpu_lib):
    a, b = _state(3), _state(4)
    b["ws"] = a["ws"]
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        _all(a)
    with torch.cuda.graph(gb):
        _all(b)
    ga.replay()
    gb.replay()
    got = _result(a), _result(b)
    for seed, r in ((3, got[0]), (4, got[1])):
        st = _state(seed)
        _all(st)
        assert all(np.array_equal(x, y) for x, y in zip(r, _result(st)))


def test_back_to_back_calls_do_not_overlap_wrongly(gpu_lib):
    # every kernel may start before the one ahead of it ends; 40 chained rounds equal 40 separate ones
    a, b = _state(5), _state(5)
    for _ in range(40):
        _all(a)
    for _ in range(40):
        _all(b)
        torch.cuda.synchronize()
    assert all(np.array_equal(x, y) for x, y in zip(_result(a), _result(b)))


def test_binding_refuses_wrong_tensors(gpu_lib):
    st = _state(6)
    o = torch.zeros_like(st["q"])
    for name, bad in (("q", st["q"].half()), ("q", st["q"].transpose(1, 2)), ("lens", st["lens"].long()),
                      ("windows", st["windows"][:1]), ("table", st["table"].long()), ("out", o[:1])):
        a = dict(q=st["q"], table=st["table"], lens=st["lens"], windows=st["windows"], out=o)
        a[name] = bad
        with pytest.raises(ValueError):
            kvq8.decode_attn_window(a["q"], st["cache"], a["table"], a["lens"], a["windows"], 4, a["out"], st["ws"])
    with pytest.raises(ValueError):
        kvq8.decode_attn_weights(st["q"], st["cache"], st["table"], st["lens"], o, st["wsum"][:1], st["ws"])
    with pytest.raises(kvq8.Kvq8Error):
        kvq8.decode_attn_weights(st["q"], st["cache"], st["table"], st["lens"], o, st["wsum"], st["ws"][:256])
    with pytest.raises(ValueError):
        kvq8.evict(st["cache"], st["wsum"], st["table"], st["lens"], 299, st["dst"], st["kept"], st["new_lens"])
    with pytest.raises(kvq8.Kvq8Error):
        kvq8.evict(st["cache"], st["wsum"], st["table"], st["lens"], 300, st["dst"], st["kept"], st["new_lens"],
                   n_first=301)
    with pytest.raises(ValueError):
        kvq8.norm_rope_append(st["q"][:, None], st["k"][:, None].bfloat16(), st["v"][:, None], None, None, 1e-6,
                              st["rope"], st["start"], st["table"], st["cache"], o[:, None])
    with pytest.raises(kvq8.Kvq8Error):
        kvq8.norm_rope_append(st["q"][:, None], st["k"][:, None], st["v"][:, None],
                              torch.ones(HD, device="cuda"), None, 1e-6, st["rope"], st["start"], st["table"],
                              st["cache"], o[:, None])


def test_streams_at_once(gpu_lib):
    want = []
    for i in range(4):
        st = _state(10 + i)
        for _ in range(10):
            _all(st)
        want.append(_result(st))
    states, streams = [_state(10 + i) for i in range(4)], [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(10):         # the calls of the four streams overlap
        for st, s in zip(states, streams):
            _all(st, stream=s)
    for st, ref_ in zip(states, want):
        assert all(np.array_equal(x, y) for x, y in zip(_result(st), ref_))


def test_page_locked_host_buffers(gpu_lib):
    # q, the new rows and out in host memory, read and written by the kernels
    a, b = _state(20), _state(20)
    kw = dict(dev_status=a["status"])
    o = torch.zeros_like(a["q"])
    kvq8.decode_step_window(a["q"], a["k"], a["v"], a["cache"], a["table"], a["lens"], a["windows"], 4, o, a["ws"], **kw)
    w = torch.zeros_like(a["q"])
    kvq8.decode_step_weights(a["q"], a["k"], a["v"], a["cache"], a["table"], a["lens"], w, a["wsum"], a["ws"], **kw)
    host = {n: b[n].cpu().pin_memory() for n in ("q", "k", "v")}
    oh, wh = torch.zeros_like(host["q"]).pin_memory(), torch.zeros_like(host["q"]).pin_memory()
    q, k, v = (kvq8.HostMapped(host[n]) for n in ("q", "k", "v"))
    kvq8.decode_step_window(q, k, v, b["cache"], b["table"], b["lens"], b["windows"], 4, kvq8.HostMapped(oh), b["ws"])
    kvq8.decode_step_weights(q, k, v, b["cache"], b["table"], b["lens"], kvq8.HostMapped(wh), b["wsum"], b["ws"])
    torch.cuda.synchronize()
    assert torch.equal(o.cpu(), oh) and torch.equal(w.cpu(), wh) and torch.equal(a["wsum"], b["wsum"])
    with pytest.raises(ValueError):
        kvq8.decode_step_window(q, k, v, b["cache"], b["table"], b["lens"], b["windows"], 4, o[:1], b["ws"])


def test_pools_past_32_bits(gpu_lib):
    # block ids whose tiles lie beyond 2^32 bytes (and 2^31 tokens' worth of codes) of the pools
    nb, nkv, nqh = 20000, 8, 16
    cache, wsum = kvq8.alloc_cache(nb, nkv), torch.empty((nb, nkv, 256), device="cuda")
    assert cache.k_pool.numel() > 2**32
    small, small_sum = kvq8.alloc_cache(8, nkv), torch.empty((8, nkv, 256), device="cuda")
    high = np.array([[19999, 19990, 19001], [18003, 17777, 16500]], np.int32)     # the last: destinations
    low = np.array([[0, 1, 2], [3, 4, 5]], np.int32)
    rng = np.random.default_rng(21)
    L = 700
    x = torch.from_numpy(rng.standard_normal((1, L, nqh + 2 * nkv, HD), np.float32)).cuda()
    rope = kvq8.rope_table(_dev(1e4 ** (-np.arange(64) / 64.0)), 1024)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = []
    for c, w, t in ((cache, wsum, high), (small, small_sum, low)):
        table, dst = _dev(t[:1]), _dev(t[1:])
        out = torch.empty((1, L, nqh, HD), device="cuda")
        kvq8.norm_rope_append(x[:, :, :nqh], x[:, :, nqh:nqh + nkv], x[:, :, nqh + nkv:], None, None, 0.0, rope,
                              torch.zeros(1, dtype=torch.int32, device="cuda"), table, c, out, weight_sum=w)
        q = out[:, -1].contiguous()
        o1, o2 = torch.empty_like(q), torch.empty_like(q)
        ws = kvq8.alloc_weights_workspace(1, nqh, nkv, 3)
        kvq8.decode_attn_window(q, c, table, lens, torch.tensor([90], dtype=torch.int32, device="cuda"), 4, o1, ws)
        kvq8.decode_attn_weights(q, c, table, lens, o2, w, ws)
        kept = torch.empty((1, nkv, 600), dtype=torch.int32, device="cuda")
        new = torch.empty((1,), dtype=torch.int32, device="cuda")
        kvq8.evict(c, w, table, lens, 600, dst, kept, new, n_recent=10)
        ids = torch.from_numpy(t.reshape(-1).astype(np.int64)).cuda()
        live = torch.arange(768, device="cuda").reshape(3, 256)
        mask = torch.cat([live < L, live < 600])[:, None]                          # [6][1][256]
        pools = [torch.where(mask, p[ids], 0) for p in (c.k_scale, c.v_scale, w)]
        pools.append(torch.where(mask[..., None], c.k_pool[ids], 0))
        pools.append(torch.where(mask.reshape(6, 1, 4, 1, 64), c.v_pool[ids], 0))
        got.append([y.cpu() for y in (out, o1, o2, kept, new, *pools)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_largest_batch(gpu_lib):
    # 65535 sequences of one token: each output row is its value row as the cache holds it
    B = 65535
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((B, 1, 3, HD), generator=g, device="cuda")
    ids = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32)
    table, dst = ids[:B, None].contiguous(), ids[B:, None].contiguous()
    cache, wsum = kvq8.alloc_cache(2 * B, 1), torch.full((2 * B, 1, 256), 9.0, device="cuda")
    rope = kvq8.rope_table(_dev(1e4 ** (-np.arange(64) / 64.0)), 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.empty((B, 1, 1, HD), device="cuda")
    kvq8.norm_rope_append(x[:, :, :1], x[:, :, 1:2], x[:, :, 2:], None, None, 0.0, rope,
                          torch.zeros(B, dtype=torch.int32, device="cuda"), table, cache, q, weight_sum=wsum,
                          dev_status=status)
    assert torch.equal(q, x[:, :, :1])                       # position 0 turns nothing
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    scale = cache.v_scale[table[:, 0].long(), 0, 0]
    want = cache.v_pool[table[:, 0].long(), 0, 0, :, 0].float() * scale[:, None]
    assert (want - x[:, 0, 2]).abs().max().item() <= 0.51 * scale.max().item()
    ws = kvq8.alloc_weights_workspace(B, 1, 1, 1)
    q = q[:, 0]
    for out in (torch.zeros_like(q), torch.zeros_like(q)):
        kvq8.decode_attn_window(q, cache, table, lens, lens, 0, out, ws, dev_status=status)
        assert (out[:, 0] - want).abs().max().item() <= 1e-5
        out.zero_()
        kvq8.decode_attn_weights(q, cache, table, lens, out, wsum, ws, dev_status=status)
        assert (out[:, 0] - want).abs().max().item() <= 1e-5
    assert (wsum[table[:, 0].long(), 0, 0] - 2.0).abs().max().item() <= 1e-5
    kept, new = torch.empty((B, 1, 1), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    kvq8.evict(cache, wsum, table, lens, 1, dst, kept, new, dev_status=status)
    assert not kept.any() and torch.equal(new, lens) and int(status.item()) == 0
    kvq8.decode_attn_window(q, cache, dst, new, lens, 0, out, ws)
    assert (out[:, 0] - want).abs().max().item() <= 1e-5


@pytest.mark.parametrize("between", ["turn", "rows"])
@pytest.mark.parametrize("batch, nkv, keep", [(1, 2, 1024), (2, 1, 1500), (28, 8, 1024)])
def test_step_with_the_cache_ready_two_calls_behind(gpu_lib, batch, nkv, keep, between):
    # a step that may read the cache before the call ahead of it ends still sees
    # what the eviction before that call wrote
    rng = np.random.default_rng(40)
    nqh, n_dst = 2 * nkv, keep // 256 + 1
    nb = batch * (8 + n_dst)
    ids = rng.permutation(nb).astype(np.int32)
    table, dst = _dev(ids[:8 * batch].reshape(batch, 8)), _dev(ids[8 * batch:].reshape(batch, n_dst))
    cache, wsum = kvq8.alloc_cache(nb, nkv), torch.rand((nb, nkv, 256), device="cuda")
    rows = torch.randn((batch, 2048, nkv, HD), device="cuda")
    kvq8.quantize_append(rows, rows, torch.zeros(batch, dtype=torch.int32, device="cuda"), table, cache)
    lens, after = (torch.full((batch,), n, dtype=torch.int32, device="cuda") for n in (2048, keep + 1))
    kept = torch.empty((batch, nkv, keep), dtype=torch.int32, device="cuda")
    new_lens = torch.empty_like(lens)
    q, k, v = (torch.randn((batch, n, HD), device="cuda") for n in (nqh, nkv, nkv))
    ws, status = kvq8.alloc_workspace(batch, nqh, nkv, 8), torch.zeros(1, dtype=torch.int32, device="cuda")
    other, rope = kvq8.alloc_cache(1, 1), kvq8.rope_table(_dev(1e4 ** (-np.arange(64) / 64.0)), 16)
    x = torch.randn((1, 1, 1, HD), device="cuda")
    zero, q_out = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.empty((1, 1, 1, HD), device="cuda")
    many, o = torch.randn((1, 40, 1, HD), device="cuda"), torch.empty_like(q)

    def calls(ready):
        kvq8.evict(cache, wsum, table, lens, keep, dst, kept, new_lens, 4, 64, dev_status=status)
        if between == "rows":
            kvq8.quantize_append(many, many, zero[0], zero, other, dev_status=status)
        else:
            kvq8.norm_rope_append(x, x, x, None, None, 1e-6, rope, zero[0], zero, other, q_out, dev_status=status)
        kvq8.decode_step(q, k, v, cache, dst, after, o, ws, dev_status=status, cache_ready=ready)

    calls(False)
    torch.cuda.synchronize()
    want = o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(True)
    for _ in range(20):
        for c in cache:
            c[dst.flatten().long()] = 0
        o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    assert int(status.item()) == 0


@pytest.mark.parametrize("raw", [False, True])
def test_rope_table_on_another_stream(gpu_lib, raw):
    # the table's memory must not be one that the current stream still writes
    inv = _dev(1e4 ** (-np.arange(64) / 64.0))
    want = kvq8.rope_table(inv, 1000).cpu()
    side = torch.cuda.Stream()
    torch.cuda._sleep(1000)          # (its first launch may wait for the device)
    x = torch.full((1000, HD), 7.0, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    x.fill_(7.0)
    del x
    table = kvq8.rope_table(inv, 1000, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert torch.equal(table.cpu(), want)
