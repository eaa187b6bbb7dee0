"""Decode over shared prefixes against its 64-bit form and against the plain decode of
the same tokens: groups of every size, prefixes that end anywhere, rows shorter than
the prefix, empty rows and groups, steps, broken groups and tables, graphs and streams."""
import pytest
import torch

import tile_ref as ref
from int8_quantized_kv_gb300 import kvq8

pytestmark = pytest.mark.gpu


class Shared:
    """sizes[g] rows in group g, prefix[g] tokens shared, lens[b] tokens in each row."""

    def __init__(self, sizes, prefix, lens, nqh, nkv, seed, step=False, size=1.5, spread=None, table=None):
        self.batch, self.nqh, self.nkv, self.step = sum(sizes), nqh, nkv, step
        self.sizes, self.prefix, self.lens = sizes, prefix, lens
        self.first = [sum(sizes[:g]) for g in range(len(sizes))]
        self.group = [g for g, m in enumerate(sizes) for _ in range(m)]
        self.mb = max(1, max(max(lens, default=1), max(prefix, default=1)) // 256 + 1)
        table, nb = table or ref.random_table(self.batch, self.mb, seed)
        self.cache = ref.random_cache(nb, nkv, seed, spread)
        # a row's whole blocks below the prefix are nobody's (its own entries are not looked at), but in the row
        # that the prefix is read through: the first one that has all of it, else the longest
        self.lead = []
        for g, m in enumerate(sizes):
            rows = range(self.first[g], self.first[g] + m)
            has = [min(prefix[g], lens[b] - (1 if step else 0)) for b in rows]
            self.lead.append(rows[has.index(max(has))] if m else None)
            for b in rows:
                if b != self.lead[g]:
                    table[b, :min(prefix[g], max(lens[b] - (1 if step else 0), 0)) // 256] = -1
        self.table = table
        g = torch.Generator("cuda").manual_seed(seed + 1)
        self.q = size * torch.randn((self.batch, nqh, 128), generator=g, device="cuda")
        self.k_new = torch.randn((self.batch, nkv, 128), generator=g, device="cuda")
        self.v_new = torch.randn((self.batch, nkv, 128), generator=g, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.starts_d, self.prefix_d, self.lens_d = i32(self.first + [self.batch]), i32(prefix), i32(lens)
        self.out = torch.full_like(self.q, float("nan"))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = kvq8.alloc_shared_workspace(self.batch, len(sizes), nqh, nkv, self.mb)
        self.ws.fill_(0xFF)

    def run(self, stream=None):
        args = (self.cache, self.table, self.lens_d, self.starts_d, self.prefix_d, self.out, self.ws)
        if self.step:
            kvq8.decode_step_shared(self.q, self.k_new, self.v_new, *args, dev_status=self.status, stream=stream)
        else:
            kvq8.decode_attn_shared(self.q, *args, dev_status=self.status, stream=stream)
        torch.cuda.synchronize()
        return self.out

    def check(self, rows=None, what=""):
        G = self.nqh // self.nkv
        for b in range(self.batch) if rows is None else rows:
            L = self.lens[b]
            if L == 0:
                assert not self.out[b].any(), f"row {b} is empty"
                continue
            g = self.group[b]
            s = max(0, min(self.prefix[g], L - 1 if self.step else L))
            for h in range(self.nkv):
                k1, v1 = ref.rows64(self.cache, self.table[self.lead[g]], h, torch.arange(s, device="cuda"))
                k2, v2 = ref.rows64(self.cache, self.table[b], h, torch.arange(s, L, device="cuda"))
                want, tol = ref.attend(self.q[b, h * G:(h + 1) * G], torch.cat([k1, k2]), torch.cat([v1, v2]),
                                       torch.full((G,), L, device="cuda"))
                ref.check(self.out[b, h * G:(h + 1) * G], want, tol, f"{what} b={b} h={h} L={L} shared={s}")


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("step", [False, True])
def test_prefixes_that_end_anywhere(gpu_lib, G, step):
    prefix = [1, 63, 64, 65, 128, 200, 256, 257, 511, 512, 700, 0]
    sizes = [2, 1, 3, 2, 4, 1, 2, 2, 5, 1, 3, 2]
    lens = []
    for m, p in zip(sizes, prefix):
        lens += [p + (1 if i == 0 else 37 * i * i + 1) for i in range(m)]
    c = Shared(sizes, prefix, lens, 2 * G, 2, 200 + G, step)
    c.run()
    c.check()
    assert c.status.item() == 0


@pytest.mark.parametrize("nqh,nkv", [(1, 1), (5, 5), (12, 3), (64, 8), (16, 8)])
def test_heads(gpu_lib, nqh, nkv):
    c = Shared([3, 6], [300, 1000], [301, 400, 999, 1001, 1100, 1000, 2000, 1005, 1256], nqh, nkv, 211)
    c.run()
    c.check()


@pytest.mark.parametrize("m", [1, 15, 16, 17, 31, 32, 33, 40, 64, 65, 130])
def test_one_group_of_many_rows(gpu_lib, m):
    c = Shared([m], [900], [901 + (i * 7) % 50 for i in range(m)], 8, 2, 213 + m)
    c.run()
    c.check()


def test_long_prefixes(gpu_lib):
    c = Shared([40, 3], [20011, 33000], [20012 + 11 * i for i in range(40)] + [33001, 33300, 35000], 8, 2, 215)
    c.run()
    c.check()


@pytest.mark.parametrize("step", [False, True])
def test_rows_shorter_than_the_prefix_and_empty_rows(gpu_lib, step):
    lens = [0, 100, 1, 700, 0, 699, 701, 0, 0, 0, 5, 300, 1024]
    c = Shared([7, 2, 4], [700, 300, 1024], lens, 8, 2, 217, step)
    c.run()
    c.check()
    assert c.status.item() == 0


def test_empty_groups(gpu_lib):
    c = Shared([0, 2, 0, 0, 1, 0], [5, 400, 7, 900, 100, 3], [450, 401, 130], 8, 2, 219)
    c.run()
    c.check()
    assert c.status.item() == 0


def test_groups_of_one_and_no_prefix_match_the_plain_decode(gpu_lib):
    for prefix in ([0, 0, 0], [100, 1000, 640]):
        c = Shared([1, 1, 1], prefix, [333, 1500, 641], 8, 2, 221)
        c.run()
        ws, plain = kvq8.alloc_workspace(3, 8, 2, c.mb), torch.empty_like(c.q)
        kvq8.decode_attn(c.q, c.cache, c.table, c.lens_d, plain, ws)
        torch.cuda.synchronize()
        assert (plain - c.out).abs().max().item() <= 1e-5 * plain.abs().max().item()


def test_step_appends_as_the_plain_step(gpu_lib):
    sizes, prefix = [3, 2], [256, 130]
    lens = [257, 512, 300, 131, 400]
    c = Shared(sizes, prefix, lens, 8, 2, 223, step=True)
    other = kvq8.KVCache(*(x.clone() for x in c.cache))
    own = c.table.clone()                                        # a table in which every row names its own blocks
    for b in range(5):
        own[b, :prefix[c.group[b]] // 256] = c.table[c.lead[c.group[b]], :prefix[c.group[b]] // 256]
    c.run()
    ws, out = kvq8.alloc_workspace(5, 8, 2, c.mb), torch.empty_like(c.q)
    kvq8.decode_step(c.q, c.k_new, c.v_new, other, own, c.lens_d, out, ws)
    torch.cuda.synchronize()
    for x, y in zip(c.cache, other):
        assert torch.equal(x, y)
    c.check()


def test_groups_that_do_not_cut_the_batch(gpu_lib):
    for starts in ([0, 2, 1, 5], [1, 2, 3, 5], [0, 2, 3, 4], [0, 2, 3, 6], [0, 2**31 - 1, -2**31, 5], [0, -1, 3, 5]):
        c = Shared([5], [300], [400, 301, 500, 350, 600], 8, 2, 225)
        c.table, _ = ref.random_table(5, c.mb, 225)              # every row has its own blocks
        c.starts_d = torch.tensor(starts, dtype=torch.int32, device="cuda")
        c.prefix_d = torch.tensor([100, 300, 200], dtype=torch.int32, device="cuda")
        c.ws = kvq8.alloc_shared_workspace(5, 3, 8, 2, c.mb)
        c.ws.fill_(0xFF)
        c.run()
        assert c.status.item() == kvq8.DEV_BAD_GROUPS, starts
        c.prefix = [0]
        c.check(what=str(starts))


def test_bad_lengths(gpu_lib):
    c = Shared([2, 2], [256, 100], [300, 400, 200, 150], 8, 2, 227)
    c.table, _ = ref.random_table(4, c.mb, 227)
    c.prefix_d[0] = -5
    c.run()
    assert c.status.item() == kvq8.DEV_BAD_CTX_LEN
    c.prefix[0] = 0
    c.check()
    c = Shared([2, 2], [256, 100], [300, 511, 200, 150], 8, 2, 229)
    assert c.mb == 2
    c.lens_d[1], c.lens_d[3] = 100000, -4
    c.lens[1], c.lens[3] = 512, 0
    c.lens_d[0], c.lens[0] = 200, 200
    c.lead[0] = 1
    c.table, _ = ref.random_table(4, 2, 229)
    c.prefix_d[0], c.prefix[0] = 2**31 - 1, 512                  # all of row 1, which has all of it
    c.run()
    assert c.status.item() == kvq8.DEV_BAD_CTX_LEN
    c.check()


def test_bad_blocks_of_the_prefix_are_skipped_and_flagged(gpu_lib):
    c = Shared([20], [1024], [1030 + i for i in range(20)], 8, 2, 231)
    c.table[0, 2] = 10**6
    c.run()
    assert c.status.item() == kvq8.DEV_BAD_BLOCK_ID
    for b in (0, 7, 19):
        for h in range(2):
            t = torch.cat([torch.arange(512), torch.arange(768, 1024)]).cuda()
            k1, v1 = ref.rows64(c.cache, c.table[0], h, t)
            k2, v2 = ref.rows64(c.cache, c.table[b], h, torch.arange(1024, c.lens[b], device="cuda"))
            k, v = torch.cat([k1, k2]), torch.cat([v1, v2])
            want, tol = ref.attend(c.q[b, 4 * h:4 * h + 4], k, v, torch.full((4,), len(k), device="cuda"))
            ref.check(c.out[b, 4 * h:4 * h + 4], want, tol)


def test_uneven_sizes(gpu_lib):
    for size, spread in ((1e-3, 10.0), (30.0, 2.0), (0.0, 12.0)):
        c = Shared([9, 30], [500, 1300], [501 + 20 * i for i in range(9)] + [1301 + 3 * i for i in range(30)], 8, 2, 233,
                   size=size, spread=spread)
        c.run()
        c.check(what=f"{size} {spread}")


def test_non_finite_queries(gpu_lib):
    c = Shared([4], [300], [310, 301, 400, 555], 8, 2, 235)
    c.q[1, 3, 100] = float("nan")
    c.q[2] = float("inf")
    c.run()
    assert c.status.item() == kvq8.DEV_NONFINITE
    c.check()


def test_many_groups(gpu_lib):
    sizes = [1 + i % 3 for i in range(700)]
    prefix = [(i * 11) % 200 for i in range(700)]
    lens = [prefix[g] + 1 + (7 * g) % 40 for g in range(700) for _ in range(sizes[g])]
    c = Shared(sizes, prefix, lens, 2, 1, 237)
    c.run()
    assert c.status.item() == 0
    c.check(rows=[0, 1, 2, 3, 500, 501, 702, 1000, c.batch - 1])
    assert torch.isfinite(c.out).all()


def test_same_bits_again_in_a_graph_and_on_another_stream(gpu_lib):
    c = Shared([30, 5], [3000, 400], [3001 + 9 * i for i in range(30)] + [401, 500, 700, 450, 410], 8, 2, 239, step=True)
    want = c.run().clone()
    side = torch.cuda.Stream()
    for again in range(3):
        c.out.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        c.run(stream=side if again else None)
        assert torch.equal(c.out, want)
    graph = torch.cuda.CUDAGraph()
    other = Shared([3], [100], [150, 101, 300], 8, 2, 241)
    other_want = other.run().clone()
    with torch.cuda.graph(graph):
        kvq8.decode_step_shared(c.q, c.k_new, c.v_new, c.cache, c.table, c.lens_d, c.starts_d, c.prefix_d, c.out, c.ws)
        kvq8.decode_attn_shared(other.q, other.cache, other.table, other.lens_d, other.starts_d, other.prefix_d, other.out,
                                c.ws)                             # one workspace, in turn
    for _ in range(3):
        c.out.fill_(float("nan"))
        other.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(other.out, other_want)


def test_replayed_with_other_lengths(gpu_lib):
    # groups and lengths are device data: a captured call follows them
    c = Shared([2, 3], [300, 200], [900, 900, 900, 900, 900], 8, 2, 243)
    c.table, _ = ref.random_table(5, c.mb, 243)
    graph = torch.cuda.CUDAGraph()
    c.run()
    with torch.cuda.graph(graph):
        kvq8.decode_attn_shared(c.q, c.cache, c.table, c.lens_d, c.starts_d, c.prefix_d, c.out, c.ws)
    for first, prefix, lens in (([0, 4], [800, 0], [801, 850, 900, 890, 5]), ([0, 0], [10, 64], [65, 64, 300, 700, 900])):
        c.starts_d.copy_(torch.tensor(first + [5]))
        c.prefix_d.copy_(torch.tensor(prefix))
        c.lens_d.copy_(torch.tensor(lens))
        c.lens, c.prefix, c.lead = lens, prefix, [0, first[1]]
        c.group = [1 if b >= first[1] else 0 for b in range(5)]
        if first[1] == 0:
            c.lead = [None, 0]
        graph.replay()
        torch.cuda.synchronize()
        c.check(what=str(first))


@pytest.mark.parametrize("level", [-300.0, 300.0])
def test_rows_that_see_nothing_of_the_prefixs_later_part(gpu_lib, level):
    # the rows that end early in a prefix which several CTAs share: the later records hold nothing of them
    c = Shared([5], [1500], [1501, 100, 300, 129, 1700], 4, 2, 245)
    c.q.fill_(1.0)
    c.q += 0.01 * torch.randn(c.q.shape, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    c.cache.k_pool.fill_(100)
    c.cache.k_scale.fill_(level / (100 * 128 * ref.SM))
    c.run()
    c.check(what=f"level={level}")


def test_step_captured_and_replayed(gpu_lib):
    # each replay appends the tokens that then stand in k_new, v_new, at the lengths that then stand in ctx_lens
    c = Shared([3, 2], [300, 128], [301, 340, 500, 129, 200], 8, 2, 247, step=True)
    graph = torch.cuda.CUDAGraph()
    c.run()
    with torch.cuda.graph(graph):
        kvq8.decode_step_shared(c.q, c.k_new, c.v_new, c.cache, c.table, c.lens_d, c.starts_d, c.prefix_d, c.out, c.ws)
    g = torch.Generator("cuda").manual_seed(7)
    for _ in range(3):
        c.lens_d += 1
        c.lens = [n + 1 for n in c.lens]
        for x in (c.q, c.k_new, c.v_new):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        c.check()
        for b in range(5):                                       # the token stands in the cache
            for h in range(2):
                k, v = ref.rows64(c.cache, c.table[b], h, torch.tensor([c.lens[b] - 1], device="cuda"))
                for got, x in ((k, c.k_new[b, h]), (v, c.v_new[b, h])):
                    assert (got[0] - x.double()).abs().max() <= x.abs().max().double() / 127 * 0.5001


def test_blocks_past_32_bits(gpu_lib):
    c = Shared([3, 2], [600, 128], [601, 640, 800, 129, 200], 8, 8, 249, step=True)
    before = [x.clone() for x in c.cache]
    want = c.run().clone()
    spare = 2**32 // (8 * 256 * 128)
    big = kvq8.KVCache(*(torch.empty((spare + x.shape[0],) + x.shape[1:], dtype=x.dtype, device="cuda") for x in c.cache))
    for x, y in zip(big, before):
        x[spare:] = y
    small = c.cache
    c.cache = big
    c.table = torch.where(c.table >= 0, c.table + spare, c.table)
    c.out.fill_(float("nan"))
    assert torch.equal(c.run(), want)
    for x, y in zip(big, small):
        assert torch.equal(x[spare:], y)
    assert c.status.item() == 0


def test_two_calls_at_once(gpu_lib):
    a = Shared([20, 5], [2000, 400], [2001 + 9 * i for i in range(20)] + [401, 500, 700, 450, 410], 8, 2, 251)
    b = Shared([4], [3000], [3001, 3100, 3300, 3500], 16, 2, 253)
    wa, wb = a.run().clone(), b.run().clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.out.zero_()
        b.out.zero_()
        torch.cuda.synchronize()
        for x, s in ((a, sa), (b, sb)):
            kvq8.decode_attn_shared(x.q, x.cache, x.table, x.lens_d, x.starts_d, x.prefix_d, x.out, x.ws, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.out, wa) and torch.equal(b.out, wb)


@pytest.mark.parametrize("rows", [4, 16, 32])
def test_long_sums_do_not_shrink(gpu_lib, rows):
    # 20 groups x 8 heads, so that every CTA has some 450 stages of a tile; even weights and values of one sign: each output
    # is the mean of 60000 values.  A step of the tensor cores cuts off less than 2^-23 of its accumulator, which grows evenly
    # over at most 12 stages of 16 steps; weights and sums 2^-18
    prefix = 60000
    mb = prefix // 256 + 1                                       # only the blocks that are looked at, or 640 rows need 147 GB
    table = torch.full((20 * rows, mb), -1, dtype=torch.int32, device="cuda")
    table[:, -1] = 20 * mb + torch.arange(20 * rows)
    table[::rows] = torch.arange(20 * mb, dtype=torch.int32, device="cuda").reshape(20, mb)
    c = Shared([rows] * 20, [prefix] * 20, [prefix + 1 + b % 5 for b in range(20 * rows)], 32, 8, 255,
               table=(table, 20 * mb + 20 * rows))
    c.cache.v_pool.abs_()
    c.q.zero_()
    c.run()
    for b in (0, 20 * rows - 1):
        for h in (0, 7):
            k1, v1 = ref.rows64(c.cache, c.table[c.lead[c.group[b]]], h, torch.arange(prefix, device="cuda"))
            k2, v2 = ref.rows64(c.cache, c.table[b], h, torch.arange(prefix, c.lens[b], device="cuda"))
            want = torch.cat([v1, v2]).mean(0)
            r = ((c.out[b, 4 * h:4 * h + 4].double() - want).abs() / want).max().item()
            assert r <= 96 * 2.0 ** -23 + 2.0 ** -18, f"b={b} h={h}: {r:.3g} off"


def test_ready_steps_between_shared_ones(gpu_lib):
    # a step with the cache declared ready may start while the call ahead of it runs: what that call appended is there all
    # the same, and the other way round; captured, replayed over a cache whose new slots were overwritten, bit for bit
    batch, nkv, G, L0, n, prefix = 6, 2, 4, 330, 8, 300
    g = torch.Generator("cuda").manual_seed(257)
    rows = lambda *s: torch.randn((*s, 128), generator=g, device="cuda")  # noqa: E731
    old_k, old_v = rows(batch, L0, nkv), rows(batch, L0, nkv)
    for x in (old_k, old_v):
        x[1:4, :prefix], x[5, :prefix] = x[0, :prefix], x[4, :prefix]
    k, v = rows(n, batch, nkv), 5 * rows(n, batch, nkv)
    q = (k[:, :, :, None] + 0.3 * rows(n, batch, nkv, G)).flatten(2, 3).contiguous()   # along the new tokens' keys
    table, nb = ref.random_table(batch, 2, 257)
    cache = kvq8.alloc_cache(nb, nkv, "cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [i32(*[L0 + i + 1] * batch) for i in range(n)]
    starts, shared, zero, status = i32(0, 4, 6), i32(prefix, prefix), i32(*[0] * batch), i32(0)
    ws, wd = kvq8.alloc_shared_workspace(batch, 2, nkv * G, nkv, 2), kvq8.alloc_workspace(batch, nkv * G, nkv, 2)
    out = torch.empty_like(q)

    def reset():
        for x, y in zip(cache, (99, -99, 0.5, 9.0)):
            x.fill_(y)
        out.fill_(float("nan"))
        kvq8.quantize_append(old_k, old_v, zero, table, cache)
        torch.cuda.synchronize()

    def steps(ready, sync):
        for i in range(n):
            args = (q[i], k[i], v[i], cache, table, lens[i])
            if i % 2:
                kvq8.decode_step(*args, out[i], wd, dev_status=status, cache_ready=ready)
            else:
                kvq8.decode_step_shared(*args, starts, shared, out[i], ws, dev_status=status)
            if sync:
                torch.cuda.synchronize()

    reset()
    steps(False, True)
    want, want_cache = out.clone(), [x.clone() for x in cache]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(True, False)
    for _ in range(20):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(x, y) for x, y in zip(cache, want_cache))
    assert status.item() == 0


@pytest.mark.parametrize("by", [-85, 85])
def test_values_of_any_size(gpu_lib, by):
    c = Shared([3, 20, 9], [300, 700, 256], [301 + 3 * i for i in range(3)] + [701 + 30 * i for i in range(20)] +
               [257 + i for i in range(9)], 8, 2, 259, spread=3.0)
    c.cache.v_scale.mul_(2.0 ** by)
    c.run()
    c.check(what=f"2^{by}")
