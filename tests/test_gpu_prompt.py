"""Prompt attention against its 64-bit form: every group size and type, lengths and
positions next to tile, quarter and block edges, padding, strides, masks that leave
a row empty, steep scores, uneven scales, broken tables, graphs and streams."""
import math

import pytest
import torch

import tile_ref as ref
from int8_quantized_kv_gb300 import kvq8

pytestmark = pytest.mark.gpu
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


class Prompt:
    def __init__(self, starts, n_new, nqh, nkv, seed, q=torch.float32, out=torch.float32, n_tokens=None, spread=None,
                 size=1.5):
        self.batch, self.n_new, self.nqh, self.nkv = len(starts), n_new, nqh, nkv
        self.starts, self.ns = list(starts), [n_new] * len(starts) if n_tokens is None else list(n_tokens)
        mb = (max(max(starts), 0) + n_new + 255) // 256
        self.table, nb = ref.random_table(self.batch, mb, seed)
        self.cache = ref.random_cache(nb, nkv, seed, spread)
        g = torch.Generator("cuda").manual_seed(seed + 1)
        self.q = (size * torch.randn((self.batch, n_new, nqh, 128), generator=g, device="cuda")).to(q)
        self.out = torch.full((self.batch, n_new, nqh, 128), float("nan"), dtype=out, device="cuda")
        self.start_d = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.n_d = None if n_tokens is None else torch.tensor(self.ns, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = kvq8.alloc_prompt_workspace(self.batch, n_new, nqh, nkv, mb)
        self.ws.fill_(0xFF)                                     # NaN wherever a partial result is not written

    def run(self, sm_scale=None, stream=None):
        kvq8.prompt_attn(self.q, self.cache, self.table, self.start_d, self.out, self.ws, n_tokens=self.n_d,
                         sm_scale=sm_scale, dev_status=self.status, stream=stream)
        torch.cuda.synchronize()
        return self.out

    def check(self, out=None, sm=ref.SM, what=""):
        out = self.out if out is None else out
        G = self.nqh // self.nkv
        cap = self.table.shape[1] * 256
        for b, (p, n) in enumerate(zip(self.starts, self.ns)):
            n = max(0, min(n, self.n_new))
            assert torch.isnan(out[b, n:].float()).all(), f"{what} b={b}: padding was written"
            if n == 0:
                continue
            lims = (p + 1 + torch.arange(n, device="cuda")).clamp(0, cap)
            t = torch.arange(int(lims.max()), device="cuda")
            for h in range(self.nkv):
                k, v = ref.rows64(self.cache, self.table[b], h, t)
                rows = self.q[b, :n, h * G:(h + 1) * G].reshape(-1, 128)
                want, tol = ref.attend(rows, k, v, lims.repeat_interleave(G), sm, out.dtype is torch.bfloat16)
                ref.check(out[b, :n, h * G:(h + 1) * G].reshape(-1, 128), want, tol, f"{what} b={b} h={h} start={p} n={n}")


EDGES = [0, 1, 62, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700]


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n_new", [1, 2, 5, 17, 64, 65])
def test_small_calls_at_every_edge(gpu_lib, G, n_new):
    c = Prompt(EDGES, n_new, 2 * G, 2, 100 * G + n_new)
    c.run()
    c.check()
    assert c.status.item() == 0


@pytest.mark.parametrize("q", sorted(KINDS))
@pytest.mark.parametrize("out", sorted(KINDS))
def test_types(gpu_lib, q, out):
    c = Prompt([0, 37, 300], 77, 8, 2, 7, KINDS[q], KINDS[out])
    c.run()
    c.check()


@pytest.mark.parametrize("nqh,nkv", [(1, 1), (5, 5), (12, 3), (8, 2), (64, 8), (16, 8)])
def test_heads(gpu_lib, nqh, nkv):
    c = Prompt([130, 0], 150, nqh, nkv, 9)
    c.run()
    c.check()


@pytest.mark.parametrize("n_new,start", [(128, 0), (129, 0), (500, 0), (1000, 3), (37, 4000), (8, 9000), (1, 30000),
                                         (3, 40007)])
@pytest.mark.parametrize("G", [1, 4])
def test_long(gpu_lib, n_new, start, G):
    c = Prompt([start], n_new, 2 * G, 2, n_new + G)
    c.run()
    c.check()


def test_padding_is_neither_read_nor_written(gpu_lib):
    ns = [0, 1, 5, 64, 65, 199, 200, 300, -3]
    c = Prompt([0, 3, 70, 0, 256, 11, 0, 5, 9], 200, 8, 4, 21, n_tokens=ns)
    for b, n in enumerate(ns):
        c.q[b, max(n, 0):] = float("nan")
    c.run()
    c.check()
    assert c.status.item() == 0


def test_strides(gpu_lib):
    for kind in (torch.float32, torch.bfloat16):
        c = Prompt([5, 300], 70, 8, 2, 23, kind, kind)
        plain = c.run().clone()
        packed = torch.full((2, 70, 16 * 128), float("nan"), dtype=kind, device="cuda")
        packed[..., 512:1536] = c.q.flatten(2)
        wide = torch.full((2, 70, 11 * 128 + 8), 3.0, dtype=kind, device="cuda")
        c.q = packed[..., 512:1536].unflatten(-1, (8, 128))
        c.out = wide[..., 136:1160].unflatten(-1, (8, 128))
        c.run()
        assert torch.equal(c.out, plain)
        assert bool((wide[..., :136] == 3).all()) and bool((wide[..., 1160:] == 3).all())


def test_behind_the_last_token_anything_may_stand(gpu_lib):
    c = Prompt([60, 200, 0], 70, 8, 2, 25)
    want = c.run().clone()
    cap = c.table.shape[1] * 256
    for b, p in enumerate(c.starts):
        for t in range(p + 70, cap):
            blk, s = int(c.table[b, t // 256]), t % 256
            c.cache.k_scale[blk, :, s] = float("nan")
            c.cache.v_scale[blk, :, s] = float("inf")
            c.cache.k_pool[blk, :, s] = -128
    c.out.fill_(float("nan"))
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("size", [0.0, 1e-8, 1e-3, 40.0, 3e4])
def test_query_sizes(gpu_lib, size):
    # flat to one-hot softmax; blocks below the query rule's 1e-6 are zeros
    c = Prompt([200, 5], 40, 8, 2, 27, size=size)
    c.run()
    c.check(what=f"size={size}")


def test_rows_and_blocks_of_one_tile_of_very_unequal_size(gpu_lib):
    c = Prompt([333], 64, 8, 2, 29)
    g = torch.Generator("cuda").manual_seed(5)
    c.q *= torch.exp2(12 * torch.rand((1, 64, 8, 1), generator=g, device="cuda") - 10)
    c.q *= torch.exp2(6 * torch.rand((1, 64, 8, 4), generator=g, device="cuda") - 6).repeat_interleave(32, -1)
    c.run()
    c.check()


@pytest.mark.parametrize("spread", [3.0, 12.0])
def test_uneven_scales(gpu_lib, spread):
    for sm in (ref.SM, ref.SM * 2.0 ** -8):
        c = Prompt([1000, 64], 90, 8, 2, 31, spread=spread)
        c.run(sm_scale=sm)
        c.check(sm=sm)


@pytest.mark.parametrize("shape", ["rising", "falling", "spike", "cliff"])
def test_steep_scores(gpu_lib, shape):
    # scores that rise, fall or jump over the context, so that the running maximum moves tile after tile
    c = Prompt([1500], 60, 8, 2, 33)
    L = 1560
    t = torch.arange(L, device="cuda", dtype=torch.float32)
    gain = {"rising": t / 4, "falling": (L - t) / 4, "spike": 300.0 * (t == 1040), "cliff": 300.0 * (t >= 777)}[shape]
    c.q.fill_(1.0)
    c.q += 0.01 * torch.randn(c.q.shape, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    p, s = c.table[0].long()[t.long() // 256], t.long() % 256
    c.cache.k_pool[p, :, s] = 100
    c.cache.k_scale[p, :, s] = ((gain - 100) / (100 * 128 * ref.SM))[:, None]
    c.run()
    c.check(what=shape)


def test_scale_of_zero_and_below(gpu_lib):
    for sm in (0.0, -ref.SM):
        c = Prompt([100], 30, 4, 2, 35)
        c.run(sm_scale=sm)
        c.check(sm=sm)


def test_values_whose_scale_falls_and_rises_by_far(gpu_lib):
    # the weight of the later tokens far above the earlier ones', their values far below, and the other way round
    for up in (1, -1):
        c = Prompt([1000], 33, 4, 2, 37)
        L = 1033
        t = torch.arange(L, device="cuda")
        p, s = c.table[0].long()[t // 256], t % 256
        step = torch.where(t < 500, 0.0, 1.0)
        c.q.fill_(1.0)
        c.cache.k_pool[p, :, s] = 100
        c.cache.k_scale[p, :, s] = (step * 40 / (100 * 128 * ref.SM))[:, None]
        c.cache.v_scale[p, :, s] *= torch.exp2(-20.0 * up * step)[:, None]
        c.run()
        c.check(what=f"up={up}")


def test_positions_outside_the_table(gpu_lib):
    c = Prompt([-5, 0, 250], 12, 4, 2, 39)                       # one block per sequence
    c.table = c.table[:, :1].contiguous()
    c.run()
    c.check()
    assert c.status.item() == kvq8.DEV_BAD_POSITION
    assert not c.out[0, :5].any()
    c = Prompt([10], 4, 4, 2, 39)
    c.start_d.fill_(2**31 - 2)
    c.starts = [255]
    c.run()
    assert c.status.item() == kvq8.DEV_BAD_POSITION
    c.check()


def test_bad_blocks_are_skipped_and_flagged(gpu_lib):
    c = Prompt([1000, 1000], 60, 8, 2, 41)
    c.table[0, 1], c.table[0, 3] = -1, 10**6
    c.run()
    assert c.status.item() == kvq8.DEV_BAD_BLOCK_ID
    G = 4
    t = torch.cat([torch.arange(256), torch.arange(512, 768), torch.arange(1024, 1060)]).cuda()
    lims = torch.searchsorted(t, 1001 + torch.arange(60, device="cuda")).repeat_interleave(G)
    for h in range(2):
        k, v = ref.rows64(c.cache, c.table[0], h, t)
        want, tol = ref.attend(c.q[0, :, h * G:(h + 1) * G].reshape(-1, 128), k, v, lims)
        ref.check(c.out[0, :, h * G:(h + 1) * G].reshape(-1, 128), want, tol)
    c.table[0], c.table[1] = -1, -7                              # nothing left: rows of zeros
    c.run()
    assert not c.out.any()


def test_non_finite_queries(gpu_lib):
    c = Prompt([50, 0], 40, 8, 2, 43)
    c.q[0, 3, 1, 40] = float("nan")
    c.q[0, 20, 7, 127] = float("inf")
    c.q[1, 0, 0] = -float("inf")
    c.run()
    assert c.status.item() == kvq8.DEV_NONFINITE
    c.check()


def test_many_sequences(gpu_lib):
    c = Prompt([(i * 37) % 90 for i in range(3000)], 2, 2, 1, 45)
    c.run()
    assert c.status.item() == 0
    pick = Prompt.__new__(Prompt)
    pick.__dict__.update(c.__dict__)
    for lo in (0, 1400, 2990):
        pick.starts, pick.ns = c.starts[lo:lo + 10], c.ns[lo:lo + 10]
        pick.q, pick.table = c.q[lo:lo + 10], c.table[lo:lo + 10]
        pick.check(out=c.out[lo:lo + 10])
    assert torch.isfinite(c.out).all()


def test_a_row_is_the_decode_of_its_context(gpu_lib):
    c = Prompt([0, 400], 70, 8, 2, 47)
    out = c.run()
    ws = kvq8.alloc_workspace(2, 8, 2, c.table.shape[1])
    one = torch.empty((2, 8, 128), device="cuda")
    for i in (0, 1, 33, 69):
        kvq8.decode_attn(c.q[:, i].contiguous(), c.cache, c.table, c.start_d + i + 1, one, ws)
        torch.cuda.synchronize()
        assert (one - out[:, i]).abs().max().item() <= 1e-5 * out[:, i].abs().max().item()


def test_same_bits_again_in_a_graph_and_on_another_stream(gpu_lib):
    c = Prompt([100, 2000], 129, 8, 2, 49)
    want = c.run().clone()
    side = torch.cuda.Stream()
    for again in range(3):
        c.out.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        c.run(stream=side if again else None)
        assert torch.equal(c.out, want)
    graph = torch.cuda.CUDAGraph()
    other = Prompt([700], 40, 8, 2, 51)
    other_want = other.run().clone()
    with torch.cuda.graph(graph):
        for x in (c, other):
            kvq8.prompt_attn(x.q, x.cache, x.table, x.start_d, x.out, c.ws, dev_status=x.status)   # one workspace, in turn
    for _ in range(3):
        c.out.fill_(float("nan"))
        other.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(other.out, other_want)


def test_two_calls_at_once(gpu_lib):
    a, b = Prompt([900], 200, 8, 2, 53), Prompt([30, 500], 150, 8, 2, 55)
    wa, wb = a.run().clone(), b.run().clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.out.zero_()
        b.out.zero_()
        torch.cuda.synchronize()
        for x, s in ((a, sa), (b, sb)):
            kvq8.prompt_attn(x.q, x.cache, x.table, x.start_d, x.out, x.ws, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.out, wa) and torch.equal(b.out, wb)


def test_binding_refusals(gpu_lib):
    c = Prompt([10], 8, 8, 2, 57)
    args = lambda **k: [{**dict(q=c.q, cache=c.cache, block_table=c.table, start_pos=c.start_d, out=c.out,  # noqa: E731
                                workspace=c.ws), **k}]
    for bad in (dict(q=c.q.double()), dict(q=c.q.cpu()), dict(out=c.out[:, :4]), dict(out=c.out.cpu()),
                dict(start_pos=c.start_d.long()), dict(block_table=c.table.cpu()), dict(n_tokens=c.start_d.long()),
                dict(out=c.out.transpose(1, 2).contiguous().transpose(1, 2)), dict(workspace=c.ws.float())):
        with pytest.raises(ValueError):
            kvq8.prompt_attn(**args(**bad)[0])
    with pytest.raises(kvq8.Kvq8Error) as e:
        kvq8.prompt_attn(**args(workspace=c.ws[:4096])[0])
    assert e.value.status == kvq8.ERR_WORKSPACE
    with pytest.raises(kvq8.Kvq8Error) as e:
        kvq8.prompt_attn(**args(sm_scale=math.inf)[0])
    assert e.value.status == kvq8.ERR_INVALID_ARG
    packed = torch.zeros((1, 8, 8 * 128 + 2), device="cuda")     # rows not 16 bytes apart
    with pytest.raises(kvq8.Kvq8Error) as e:
        kvq8.prompt_attn(**args(q=packed[..., :1024].unflatten(-1, (8, 128)))[0])
    assert e.value.status == kvq8.ERR_INVALID_ARG
    empty = kvq8.prompt_attn(c.q[:, :0], c.cache, c.table, c.start_d, c.out[:, :0], c.ws)
    assert empty is None


@pytest.mark.parametrize("level", [-300.0, 300.0])
def test_rows_that_see_nothing_of_a_tiles_later_part(gpu_lib, level):
    # few tiles: every CTA has one stage of one, so the records of the stages behind a row's position hold nothing of it
    c = Prompt([60, 0], 300, 4, 2, 59)
    c.q.fill_(1.0)
    c.q += 0.01 * torch.randn(c.q.shape, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    c.cache.k_pool.fill_(100)
    c.cache.k_scale.fill_(level / (100 * 128 * ref.SM))
    c.run()
    c.check(what=f"level={level}")


def test_replayed_with_other_positions(gpu_lib):
    # positions and counts are device data: a captured call follows them
    c = Prompt([900, 900, 900], 40, 8, 2, 61, n_tokens=[40, 40, 40])
    c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq8.prompt_attn(c.q, c.cache, c.table, c.start_d, c.out, c.ws, n_tokens=c.n_d, dev_status=c.status)
    for starts, ns in (([0, 300, 12], [40, 1, 17]), ([883, 0, 0], [0, 0, 5]), ([0, 0, 0], [0, 0, 0]), ([64, 63, 900], [40, 39, 38])):
        c.start_d.copy_(torch.tensor(starts))
        c.n_d.copy_(torch.tensor(ns))
        c.starts, c.ns = starts, ns
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(what=str(starts))
    assert c.status.item() == 0


def test_blocks_past_32_bits(gpu_lib):
    # a pool of more than 2^32 bytes of K, of V, and the sequence's blocks at its end
    c = Prompt([600], 70, 8, 8, 63)
    nb, spare = c.table.numel() + 2, 2**32 // (8 * 256 * 128)
    big = kvq8.KVCache(*(torch.empty((spare + nb,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in c.cache))
    for x, y in zip(big, c.cache):
        x[spare:] = y
    want = c.run().clone()
    c.cache, c.table = big, c.table + spare
    c.out.fill_(float("nan"))
    assert torch.equal(c.run(), want)
    assert c.status.item() == 0


def test_most_sequences_empty(gpu_lib):
    ns = [0] * 20000
    ns[0], ns[9999], ns[19999] = 3, 2, 1
    c = Prompt([5] * 20000, 3, 8, 4, 65, n_tokens=ns)
    c.run()
    assert c.status.item() == 0
    assert torch.isnan(c.out.flatten(2)).all(2).sum().item() == 3 * 20000 - 6
    pick = Prompt.__new__(Prompt)
    pick.__dict__.update(c.__dict__)
    for b in (0, 9999, 19999):
        pick.starts, pick.ns, pick.table = [5], [ns[b]], c.table[b:b + 1]
        pick.q = c.q[b:b + 1]
        pick.check(out=c.out[b:b + 1])


# 160 tiles of each height, so that every CTA has some 450 stages of a tile.
LONG_RUNS = [(20, 2), (20, 12), (5, 128)]
# Outputs of values of one sign.  A step of the tensor cores cuts off less than 2^-23 of its accumulator, which grows evenly
# over a run of at most 12 stages of 16 steps: 12 * 16 / 2 * 2^-23; queries, weights and the runs' sum: 2^-18.
LONG_TOL = 96 * 2.0 ** -23 + 2.0 ** -18


def _long(batch, n_new, seed, out):
    c = Prompt([60000 + 7 * b for b in range(batch)], n_new, 32, 8, seed, out=out)
    c.cache.v_pool.abs_()
    return c


def _check_long(c, tol, what):
    for b in (0, c.batch - 1):
        for i in (0, c.n_new - 1):
            L = c.starts[b] + i + 1
            for h in (0, 7):
                k, v = ref.rows64(c.cache, c.table[b], h, torch.arange(L, device="cuda"))
                rows = c.q[b, i, 4 * h:4 * h + 4]
                want, _ = ref.attend(rows, k, v, torch.full((4,), L, device="cuda"))
                half = torch.finfo(c.out.dtype).eps / 2
                r = ((c.out[b, i, 4 * h:4 * h + 4].double() - want).abs() / want).max().item()
                assert r <= tol + half, f"{what} b={b} i={i} h={h}: {r:.3g} off, {tol + half:.3g} allowed"


@pytest.mark.parametrize("batch,n_new", LONG_RUNS)
def test_long_sums_do_not_shrink(gpu_lib, batch, n_new):
    # even weights: each output is the mean of 60000 values, which one accumulator would cut by 1e-4
    for out in (torch.float32, torch.float16) if n_new == 128 else (torch.float32,):
        c = _long(batch, n_new, 67, out)
        c.q.zero_()
        c.run()
        _check_long(c, LONG_TOL, str(out))


@pytest.mark.parametrize("batch,n_new", LONG_RUNS)
def test_totals_move_with_their_references(gpu_lib, batch, n_new):
    # the last 300 tokens weigh 2^8 times as much as the others, which are still two fifths of the output
    c = _long(batch, n_new, 69, torch.float32)
    c.q.fill_(1.0)
    for b, p in enumerate(c.starts):
        t = torch.arange(p + n_new, device="cuda")
        blk, s = c.table[b].long()[t // 256], t % 256
        c.cache.k_pool[blk, :, s] = 100
        c.cache.k_scale[blk, :, s] = ((t >= p - 300).float() * 8 / (100 * 128 * ref.SM * ref.LOG2E))[:, None]
    c.run()
    # (scores of 8 in size: 2 * 2^-19 * 8 of ln 2 each)
    _check_long(c, LONG_TOL + 16 * 2.0 ** -19, "cliff")


def test_long_sums_in_bf16(gpu_lib):
    # the weights' 11 bits and the cut of up to 256 stages, both far below bf16's half step
    c = _long(5, 128, 71, torch.bfloat16)
    c.q.zero_()
    c.run()
    _check_long(c, 2.0 ** -11 + 256 * 8 / 2 * 2.0 ** -23 + 2.0 ** -18, "bf16")


@pytest.mark.parametrize("by", [-85, 85])
@pytest.mark.parametrize("n_new", [2, 10, 90])
def test_values_of_any_size(gpu_lib, by, n_new):
    c = Prompt([700, 0, 130], n_new, 8, 2, 73, spread=3.0)
    c.cache.v_scale.mul_(2.0 ** by)
    c.run()
    c.check(what=f"2^{by}")


def test_rows_of_zeros_among_the_values(gpu_lib):
    # their scale is 0: they count in the sum alone; first all of them, then every third
    for n_new in (2, 90):
        c = Prompt([700, 0], n_new, 8, 2, 75)
        for b in range(2):
            t = torch.arange(c.starts[b] + n_new, device="cuda")
            t = t[(t < 300) | (t % 3 == 0)]
            blk, s = c.table[b].long()[t // 256], t % 256
            c.cache.v_scale[blk, :, s] = 0.0
            c.cache.v_pool[blk, :, s // 64, :, s % 64] = 0
        c.run()
        c.check()


@pytest.mark.parametrize("spread", [6, 11, 13, 40])
def test_rows_of_one_tile_of_any_size(gpu_lib, spread):
    # queries of 2^-spread .. 1 beside each other, rows of zeros among them, in tiles of 128 rows (which take one unit for
    # rows of like size), and one row whose scores leave all others' far behind
    c = Prompt([150, 600], 70, 8, 2, 77)
    g = torch.Generator("cuda").manual_seed(79)
    c.q *= torch.exp2(-spread * torch.rand((2, 70, 8, 1), generator=g, device="cuda"))
    c.q[0, 5], c.q[1, 40, 3] = 0.0, 0.0
    c.run()
    c.check(what=f"spread={spread}")
    c.q[1, 20, 2] *= 2.0 ** 60
    c.run()
    keep = torch.ones(2, 70, 8, dtype=torch.bool, device="cuda")
    keep[1, 20, 2] = False
    want = c.out.clone()
    c.q[1, 20, 2] = 0.0
    c.run()
    d = (c.out - want)[keep]
    assert torch.isfinite(want).all() and d.abs().max().item() <= 2.0 ** -17 * want.abs().max().item()
