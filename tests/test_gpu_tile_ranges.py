"""Prompts and shared prefixes at the ends of what their inputs may be: rows of zeros among
the values beside values of any size, queries whose 32-blocks are of very unequal size, flat
to one-hot weights with keys of any size, as much work in one group as 32 bits do not count."""
import pytest
import torch

import tile_bounds
import tile_ref as ref
from int8_quantized_kv_gb300 import kvq8
from test_gpu_prompt import Prompt
from test_gpu_shared import Shared

pytestmark = pytest.mark.gpu

# New query tokens per sequence with four heads to a kv head: tiles of 16, 32, 64 and 128 rows.
HEIGHTS = [3, 6, 12, 40]


def _places(blocks, t):
    return blocks.long()[t // 256], t % 256


def _zeros(cache, blocks, t):
    blk, s = _places(blocks, t)
    cache.v_scale[blk, :, s] = 0.0
    cache.v_pool[blk, :, s // 64, :, s % 64] = 0


def _larger(cache, blocks, t, by):
    blk, s = _places(blocks, t)
    cache.v_scale[blk, :, s] *= 2.0 ** by


def _mixed_values(cache, blocks, n, by, where):
    """Tokens [0, n): rows of zeros before, behind or between rows 2^by times as large as drawn."""
    t = torch.arange(n, device="cuda")
    zero = {"first": t < n // 2, "last": t >= n // 2, "between": (t // 150) % 2 == 0}[where]
    _zeros(cache, blocks, t[zero])
    _larger(cache, blocks, t[~zero], by)


@pytest.mark.parametrize("where", ["first", "last", "between"])
@pytest.mark.parametrize("by", [-40, 40, 44, 85])
@pytest.mark.parametrize("n_new", HEIGHTS)
def test_prompt_rows_of_zeros_beside_values_of_any_size(gpu_lib, n_new, by, where):
    # a tile shared by many CTAs (each has a stage or two, so the records differ), and tiles that a CTA has whole
    for starts, size in (([700], 0.0), ([700, 333], 1.5), ([400 + 3 * i for i in range(90)], 0.0)):
        c = Prompt(starts, n_new, 8, 2, 301, size=size)
        for b, p in enumerate(starts):
            _mixed_values(c.cache, c.table[b], p + n_new, by, where)
        c.run()
        for b in range(0, len(starts), 17):
            one = Prompt.__new__(Prompt)
            one.__dict__.update(c.__dict__)
            one.starts, one.ns, one.q, one.table = c.starts[b:b + 1], c.ns[b:b + 1], c.q[b:b + 1], c.table[b:b + 1]
            one.check(out=c.out[b:b + 1], what=f"2^{by} {where} size={size} of {len(starts)}")


@pytest.mark.parametrize("where", ["first", "last", "between"])
@pytest.mark.parametrize("by", [-40, 40, 85])
@pytest.mark.parametrize("rows", HEIGHTS)
def test_shared_rows_of_zeros_beside_values_of_any_size(gpu_lib, rows, by, where):
    # in the prefix, and the rows' own tokens of the other kind: zeros behind large values, and the other way round
    for size, own in ((0.0, "zeros"), (1.5, "large"), (0.0, "as drawn")):
        prefix = 900
        c = Shared([rows], [prefix], [prefix + 1 + (5 * i) % 70 for i in range(rows)], 8, 2, 303, size=size)
        _mixed_values(c.cache, c.table[c.lead[0]], prefix, by, where)
        for b in range(rows):
            t = torch.arange(prefix, c.lens[b], device="cuda")
            if own == "zeros":
                _zeros(c.cache, c.table[b], t)
            elif own == "large":
                _larger(c.cache, c.table[b], t, by)
        c.run()
        c.check(what=f"2^{by} {where} size={size} own={own}")


def test_shared_prefix_of_zeros_and_large_values_of_the_rows_own(gpu_lib):
    # the records of the prefix and of the rows' own tokens far apart, either way
    for prefix_by, own_by in ((None, 60), (60, None), (-85, 60), (85, -60)):
        c = Shared([6, 20], [700, 300], [701 + 7 * i for i in range(6)] + [301 + 3 * i for i in range(20)], 8, 2, 305, size=0.0)
        for b in range(c.batch):
            p = c.prefix[c.group[b]]
            if b == c.lead[c.group[b]]:
                t = torch.arange(p, device="cuda")
                _zeros(c.cache, c.table[b], t) if prefix_by is None else _larger(c.cache, c.table[b], t, prefix_by)
            t = torch.arange(p, c.lens[b], device="cuda")
            _zeros(c.cache, c.table[b], t) if own_by is None else _larger(c.cache, c.table[b], t, own_by)
        c.run()
        c.check(what=f"prefix {prefix_by}, own {own_by}")


@pytest.mark.parametrize("n_new", HEIGHTS)
@pytest.mark.parametrize("many", [False, True])
def test_many_rows_of_zeros_below_large_values_of_higher_scores(gpu_lib, n_new, many):
    # 4000 rows of zeros, then 100 rows of values near 2^36 whose scores are 10 higher (base 2): the zeros still take
    # 4000 / (4000 + 100 * 2^10) of the weight
    starts = [4100] * (90 if many else 1)
    c = Prompt(starts, n_new, 8, 2, 307)
    c.q.fill_(1.0)
    for b in range(len(starts)):
        t = torch.arange(4100 + n_new, device="cuda")
        blk, s = _places(c.table[b], t)
        c.cache.k_pool[blk, :, s] = 100
        c.cache.k_scale[blk, :, s] = ((t >= 4000).float() * 10 / (100 * 128 * ref.SM * ref.LOG2E))[:, None]
        _zeros(c.cache, c.table[b], t[:4000])
        _larger(c.cache, c.table[b], t[4000:], 36)
    c.run()
    for b in {0, len(starts) - 1}:
        one = Prompt.__new__(Prompt)
        one.__dict__.update(c.__dict__)
        one.starts, one.ns, one.q, one.table = c.starts[b:b + 1], c.ns[b:b + 1], c.q[b:b + 1], c.table[b:b + 1]
        one.check(out=c.out[b:b + 1])


def _only_block(cache, blocks, n, block, nkv):
    """K rows of the tokens [0, n): zero outside one 32-block."""
    t = torch.arange(n, device="cuda")
    blk, s = _places(blocks, t)
    d = torch.arange(128, device="cuda")
    keep = torch.zeros(128, dtype=torch.bool, device="cuda")
    keep[32 * block:32 * block + 32] = True
    at = ((d // 16) ^ (s[:, None] & 7)) * 16 + d % 16              # byte place of each dim
    mask = torch.zeros((n, 128), dtype=torch.int8, device="cuda").scatter_(1, at, keep.to(torch.int8).expand(n, -1))
    for h in range(nkv):
        cache.k_pool[blk, h, s] *= mask


@pytest.mark.parametrize("down,rows_apart", [(22, 0), (16, 0), (8, 10), (14, 10), (3, 40)])
@pytest.mark.parametrize("n_new", HEIGHTS)
def test_keys_that_meet_a_small_part_of_the_query(gpu_lib, n_new, down, rows_apart):
    # one 32-block of each query is 2^-down of the row's largest, and the keys are zero outside it; rows of a tile up to
    # 2^rows_apart apart.  (Rows of 2^4, so that no block falls below the query rule's 1e-6.)
    c = Prompt([300, 0], n_new, 8, 2, 309)
    g = torch.Generator("cuda").manual_seed(11)
    apart = torch.randint(0, 2, (2, n_new, 8, 1), generator=g, device="cuda").float()
    c.q *= 16.0 * torch.exp2(rows_apart * apart)
    c.q[..., 64:96] *= 2.0 ** -down
    for b, p in enumerate(c.starts):
        _only_block(c.cache, c.table[b], p + n_new, 2, 2)
    # scores of some hundreds in size for the rows of 16
    c.run(sm_scale=ref.SM * 2.0 ** (down - 1))
    c.check(sm=ref.SM * 2.0 ** (down - 1), what=f"2^-{down}, rows 2^{rows_apart} apart")


# (query size, spread of the cache's rows, factor of the scores): flat to one-hot weights, keys of one size and of any.
WEIGHTS = [(1e-3, 0.0, 1.0), (1.5, 0.0, 1.0), (40.0, 0.0, 1.0), (1e3, 0.0, 1.0), (3e4, 0.0, 1.0), (1.5, 3.0, 1.0), (1.5, 12.0, 1.0),
           (1.5, 12.0, 2.0 ** -8), (45.0, 10.0, 1.0)]
# Scores of 2^26 and more, whose own steps are wider than the weights' range.
HUGE = [(3e4, 12.0, 1.0), (3e4, 12.0, -1.0), (1e8, 12.0, 1.0), (1e20, 3.0, 1.0)]


@pytest.mark.parametrize("size,spread,factor", WEIGHTS + HUGE)
@pytest.mark.parametrize("n_new", HEIGHTS)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_prompt_weights_flat_to_one_hot(gpu_lib, out, n_new, size, spread, factor):
    c = Prompt([200, 5, 700], n_new, 8, 2, 313, out=out, size=size, spread=spread)
    c.run(sm_scale=ref.SM * factor)
    for b, p in enumerate(c.starts):
        lims = (p + 1 + torch.arange(n_new, device="cuda")).repeat_interleave(4)
        for h in range(2):
            k, v = ref.rows64(c.cache, c.table[b], h, torch.arange(p + n_new, device="cuda"))
            rows = c.q[b, :, 4 * h:4 * h + 4].reshape(-1, 128)
            want, tol, decided = tile_bounds.attend(rows, k, v, lims, ref.SM * factor, out is torch.bfloat16)
            assert tile_bounds.sharp(want, tol, decided, 0.9)
            tile_bounds.check(c.out[b, :, 4 * h:4 * h + 4], want, tol, f"b={b} h={h}")


@pytest.mark.parametrize("size,spread,factor", [w for w in WEIGHTS + HUGE if w[2] == 1.0])
@pytest.mark.parametrize("rows", HEIGHTS)
def test_shared_weights_flat_to_one_hot(gpu_lib, rows, size, spread, factor):
    c = Shared([rows], [600], [601 + (11 * i) % 150 for i in range(rows)], 8, 2, 315, size=size, spread=spread)
    c.run()
    for h in range(2):
        k1, v1 = ref.rows64(c.cache, c.table[c.lead[0]], h, torch.arange(600, device="cuda"))
        for b in range(rows):
            k2, v2 = ref.rows64(c.cache, c.table[b], h, torch.arange(600, c.lens[b], device="cuda"))
            want, tol, decided = tile_bounds.attend(c.q[b, 4 * h:4 * h + 4], torch.cat([k1, k2]), torch.cat([v1, v2]),
                                                    torch.full((4,), c.lens[b], device="cuda"))
            assert tile_bounds.sharp(want, tol, decided, 0.5)      # of four rows
            tile_bounds.check(c.out[b, 4 * h:4 * h + 4], want, tol, f"b={b} h={h}")


@pytest.mark.slow
def test_shared_group_of_more_work_than_31_bits_count(gpu_lib):
    # 65535 rows of 8 heads in tiles of 16 (65534 empty groups lower the average), each over 72000 stages: 2.36e9 with the
    # tiles' own cost, so that the last tenth of the CTAs begin beyond 2^31.  Four blocks stand for the whole prefix, and
    # equal weights make every row the mean of their values.
    batch, G, n, blocks = 65535, 8, 36000, 5
    prefix = n * 256
    cache = ref.random_cache(blocks, 1, 311)
    table = torch.full((batch, n + 1), -1, dtype=torch.int32, device="cuda")
    table[0, :n] = torch.arange(n, device="cuda") % 4
    table[:, n] = 4
    starts = torch.full((batch + 1,), batch, dtype=torch.int32, device="cuda")
    starts[0] = 0
    shared = torch.full((batch,), prefix, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), prefix + 1, dtype=torch.int32, device="cuda")
    q = torch.zeros((batch, G, 128), device="cuda")
    out = torch.full_like(q, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kvq8.alloc_shared_workspace(batch, batch, G, 1, n + 1)
    kvq8.decode_attn_shared(q, cache, table, lens, starts, shared, out, ws, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    _, v = ref.rows64(cache, torch.arange(4, device="cuda"), 0, torch.arange(1024, device="cuda"))
    _, last = ref.rows64(cache, torch.tensor([4], device="cuda"), 0, torch.zeros(1, device="cuda"))
    want = (v.mean(0) * prefix + last[0]) / (prefix + 1)
    # 9000 runs of eight stages are added to a total of 24 bits, each off by half a step (2^-25 of it) at most; within a
    # run LONG_TOL of test_gpu_prompt, of the largest of its sums of values
    tol = (9000 * 2.0 ** -25 + 96 * 2.0 ** -23 + 2.0 ** -18) * v.abs().mean(0).max()
    for part in out.split(4096):
        assert bool(((part.double() - want).abs() <= tol).all())
