"""Decode with accumulated attention weights: the output is the plain decode's
and the sums are those of the oracle's softmax weights.

Tolerance of a sum, against weights p of the 64-bit softmax over the same
codes: a score s (base 2) is a sum of four exact integers times scales, five
roundings and two products: off by at most 8 * 2^-24 |s|; |s| <= 64 on these
inputs, so 2^s is off by 64 * 8 * 2^-24 * ln 2 < 2.2e-5 of itself, the sum in
the denominator by as much again, and the base-2 exponential, the division and
the G additions add less than 2e-6: within 1e-4 of p.  Below that, values under
2^-126 of the maximum are lost: 1e-30.  An addition to a sum that is there
rounds once: 2^-24 of it."""
import numpy as np
import pytest
import torch

import cache_ops_ref as ref
from int8_quantized_kv_gb300 import kvq8
from int8_quantized_kv_gb300 import workloads as wl
from kvq8_harness import Case, StepCase, assert_close

pytestmark = pytest.mark.gpu


def _run(case, wsum, step=False, table=None, ws=None):
    cfg = case.cfg
    out = torch.full_like(case.q_d, float("nan"))
    if ws is None:
        ws = kvq8.alloc_weights_workspace(cfg.batch, cfg.nqh, cfg.nkv, case.max_blocks)
        ws.fill_(255)                                        # NaN patterns: nothing stale may count
    args = (case.cache, case.table_d if table is None else table, case.lens_d, out, wsum, ws)
    if step:
        kvq8.decode_step_weights(case.q_d, case.k_new_d, case.v_new_d, *args, dev_status=case.status)
    else:
        kvq8.decode_attn_weights(case.q_d, *args, dev_status=case.status)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def _unit_weights(case, b, h, L, step):
    G = case.cfg.group
    kq, ks, _, _ = ref.unit_rows(*wl.unit_kv(case.cfg, b, h, L), step)
    p, most = ref.weights(case.q[b, h * G:(h + 1) * G], kq, ks)
    assert most <= 64
    return p


def _check_sums(case, before, after, step=False, lens=None):
    """Every slot of every block: the listed ones as the oracle says, the others untouched."""
    cfg = case.cfg
    want = before.astype(np.float64)
    tol = np.zeros_like(want)
    for b in range(cfg.batch):
        L = int(case.lens[b]) if lens is None else lens[b]
        if L == 0:
            continue
        t = np.arange(L)
        phys, slot = case.table[b, t // 256], t % 256
        for h in range(cfg.nkv):
            p = _unit_weights(case, b, h, L, step)
            if step:
                want[phys[-1], h, slot[-1]] = 0.0
            want[phys, h, slot] += p
            tol[phys, h, slot] = 1e-4 * p + 1e-30 + 2.0**-24 * np.abs(want[phys, h, slot])
    err = np.abs(after.astype(np.float64) - want)
    assert np.all(err <= tol), f"worst {np.max(err - tol)} at {np.unravel_index(np.argmax(err - tol), err.shape)}"


def _sums(case, seed=1):
    x = np.random.default_rng(seed).random((case.num_blocks, case.cfg.nkv, 256), np.float32)
    return x, torch.from_numpy(x).cuda()


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_output_and_sums(gpu_lib, G):
    lens = [1, 3, 0, 64, 65, 511, 512, 513, 700, 1025, 1301]
    cfg = wl.Workload("s", 800 + G, batch=len(lens), nqh=2 * G, nkv=2)
    case = Case(cfg, lens=lens)
    before, wsum = _sums(case)
    plain = case.decode()
    got = _run(case, wsum)
    assert_close(got[8, :G], ref.decode(case.q[8, :G], *ref.unit_rows(*wl.unit_kv(cfg, 8, 0, lens[8]))), "out")
    assert_close(got, plain, "against the plain decode")
    _check_sums(case, before, wsum.cpu().numpy())
    assert case.status_bits() == 0


def test_sums_add_up_over_calls_and_to_the_group_size(gpu_lib):
    cfg = wl.Workload("s", 820, batch=3, nqh=16, nkv=4)
    case = Case(cfg, lens=[900, 17, 2000])
    wsum = kvq8.alloc_weight_sum(case.num_blocks, 4)
    for i in range(3):
        _run(case, wsum)
    # each call adds weights that sum to G per unit, each sum of 3 * 2^-24 relative roundings and
    # weights within 1e-4 of themselves
    w = wsum.cpu().numpy().astype(np.float64)
    for b, L in enumerate([900, 17, 2000]):
        t = np.arange(L)
        for h in range(4):
            assert abs(w[case.table[b, t // 256], h, t % 256].sum() - 3 * 4) <= 3 * 4 * 1.1e-4


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_step_starts_the_new_tokens_sum(gpu_lib, G):
    lens = [1, 64, 65, 257, 512, 1301, 0]
    cfg = wl.Workload("s", 830 + G, batch=len(lens), nqh=2 * G, nkv=2)
    case = StepCase(cfg, lens=lens)
    before, wsum = _sums(case, 2)
    # whatever the new token's slot held, NaN included, is gone
    for b, L in enumerate(lens):
        if L:
            wsum[int(case.table[b, (L - 1) // 256]), :, (L - 1) % 256] = float("nan")
    got = _run(case, wsum, step=True)
    _check_sums(case, before, wsum.cpu().numpy(), step=True)
    pools = case.host_pools()
    for b in range(cfg.batch):
        for h in range(2):
            if lens[b]:
                for x, y in zip(case.gather_unit(pools, b, h), ref.unit_rows(*wl.unit_kv(cfg, b, h, lens[b]), True)):
                    assert np.array_equal(x, y)
    # the token is in the cache now: the same decode without the append
    assert np.array_equal(got, _run(case, torch.zeros_like(wsum)))


def test_steep_scores(gpu_lib):
    # all weight on one late token: the others' sums grow by next to nothing
    L, G = 700, 4
    q, k, v = wl.steered_unit(3, L, G, "spike")
    cache = kvq8.alloc_cache(3, 1)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    kvq8.quantize_append(torch.from_numpy(k)[None, :, None].contiguous().cuda(),
                         torch.from_numpy(v)[None, :, None].contiguous().cuda(),
                         torch.zeros(1, dtype=torch.int32, device="cuda"), table, cache)
    wsum = kvq8.alloc_weight_sum(3, 1)
    out = torch.empty((1, G, 128), device="cuda")
    kvq8.decode_attn_weights(torch.from_numpy(q)[None].cuda(), cache, table,
                             torch.tensor([L], dtype=torch.int32, device="cuda"), out, wsum,
                             kvq8.alloc_weights_workspace(1, G, 1, 3))
    t = np.arange(L)
    w = wsum.cpu().numpy()[np.array([2, 0, 1])[t // 256], 0, t % 256]
    top = 2 * L // 3
    assert abs(w[top] - G) <= 1e-4 * G and np.all(np.delete(w, top) <= 1e-4)
    assert_close(out.cpu().numpy()[0], ref.decode(q, *ref.unit_rows(k, v)))


def test_bad_lengths_and_blocks(gpu_lib):
    cfg = wl.Workload("s", 840, batch=3, nqh=4, nkv=2)
    case = Case(cfg, lens=[600, 600, 600])
    before, wsum = _sums(case, 3)
    table = case.table.copy()
    table[0, 1], table[1, 0], table[2, :] = -1, case.num_blocks, 10**9
    got = _run(case, wsum, table=torch.from_numpy(table).cuda())
    assert case.status_bits() == kvq8.DEV_BAD_BLOCK_ID and np.all(np.isfinite(got)) and not got[2].any()
    after = wsum.cpu().numpy()
    G = cfg.group
    want = before.astype(np.float64)
    for b, vis in ((0, np.r_[0:256, 512:600]), (1, np.arange(256, 600))):
        for h in range(2):
            k, v = wl.unit_kv(cfg, b, h, 600)
            rows = ref.unit_rows(k[vis], v[vis])
            assert_close(got[b, h * G:(h + 1) * G], ref.decode(case.q[b, h * G:(h + 1) * G], *rows))
            want[case.table[b, vis // 256], h, vis % 256] += ref.weights(case.q[b, h * G:(h + 1) * G], *rows[:2])[0]
    assert np.abs(after - want).max() <= 1e-4
    untouched = np.ones(before.shape, bool)
    for b, vis in ((0, np.r_[0:256, 512:600]), (1, np.arange(256, 600))):
        untouched[case.table[b, vis // 256], :, vis % 256] = False
    assert np.array_equal(after[untouched], before[untouched])
    case.status.zero_()
    case.lens_d.copy_(torch.tensor([-1, 100000, 5], dtype=torch.int32))    # beyond the table: clamped
    got = _run(case, wsum)
    assert case.status_bits() & kvq8.DEV_BAD_CTX_LEN and not got[0].any() and np.all(np.isfinite(got[2]))


def test_many_units_of_two_heads(gpu_lib):
    # enough units and table for two CTAs per SM
    rng = np.random.default_rng(6)
    lens = rng.integers(1, 3000, 40).tolist()
    lens[3] = 0
    cfg = wl.Workload("s", 845, batch=40, nqh=8, nkv=4)
    for step in (False, True):
        case = (StepCase if step else Case)(cfg, lens=lens)
        assert cfg.batch * cfg.nkv * case.max_blocks * 4 >= 16 * 2 * 152
        before, wsum = _sums(case, 7)
        _run(case, wsum, step=step)
        _check_sums(case, before, wsum.cpu().numpy(), step=step)


def test_wide_table(gpu_lib):
    # lengths far below the table's width, and one near it in the last row
    cfg = wl.Workload("s", 850, batch=3, nqh=8, nkv=1)
    case = Case(cfg, lens=[5, 2, 40000])
    before, wsum = _sums(case, 4)
    _run(case, wsum)
    _check_sums(case, before, wsum.cpu().numpy())


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("shape", ["rise", "fall", "waves"])
def test_many_records_per_unit(gpu_lib, G, shape):
    # a unit cut into more than 32 records, whose maxima rise, fall, or do both from one to the next
    rng = np.random.default_rng(860 + G)
    lens = [30001, 70]
    u = rng.standard_normal((G, 128)).astype(np.float32)
    q = np.stack([4 * u, 4 * u])
    L = lens[0]
    t = np.arange(L) / L
    lift = {"rise": t, "fall": 1 - t, "waves": 0.5 + 0.5 * np.sin(40 * t)}[shape]
    k = 0.3 * rng.standard_normal((2, L, 1, 128)) + 0.35 * lift[None, :, None, None] * u.sum(0)
    k, v = k.astype(np.float32), rng.standard_normal((2, L, 1, 128)).astype(np.float32)
    nb = 2 * ((L + 255) // 256)
    table = rng.permutation(nb).astype(np.int32).reshape(2, -1)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache, table_d, lens_d = kvq8.alloc_cache(nb, 1), d(table), d(np.array(lens, np.int32))
    kvq8.quantize_append(d(k), d(v), torch.zeros(2, dtype=torch.int32, device="cuda"), table_d, cache)
    wsum, out = kvq8.alloc_weight_sum(nb, 1), torch.full((2, G, 128), float("nan"), device="cuda")
    ws = kvq8.alloc_weights_workspace(2, G, 1, table.shape[1])
    ws.fill_(255)
    kvq8.decode_attn_weights(d(q), cache, table_d, lens_d, out, wsum, ws)
    got, sums = out.cpu().numpy(), wsum.cpu().numpy()
    records = ws[:8].view(torch.int32)[1].item()             # the first unit's (first CTA, number) in the workspace
    assert records > 64
    for b, n in enumerate(lens):
        rows = ref.unit_rows(k[b, :n, 0], v[b, :n, 0])
        assert_close(got[b], ref.decode(q[b], *rows), f"sequence {b}")
        p, most = ref.weights(q[b], *rows[:2])
        assert most <= 64
        i = np.arange(n)
        assert np.all(np.abs(sums[table[b, i // 256], 0, i % 256] - p) <= 1e-4 * p + 1e-30)


@pytest.mark.parametrize("step", [False, True])
def test_output_of_many_units_of_two_heads(gpu_lib, step):
    # the grid of two CTAs per SM, against the plain decode over the same cache
    lens = np.random.default_rng(7).integers(1, 3000, 40)
    lens[5] = 0
    cfg = wl.Workload("s", 846, batch=40, nqh=8, nkv=4)
    case = (StepCase if step else Case)(cfg, lens=lens)
    got = _run(case, kvq8.alloc_weight_sum(case.num_blocks, 4), step=step)
    assert_close(got, case.decode(), "against the plain decode")
    for b in (0, 17, 39):
        rows = ref.unit_rows(*wl.unit_kv(cfg, b, 3, int(lens[b])), step)
        assert_close(got[b, 6:], ref.decode(case.q[b, 6:], *rows), f"sequence {b}")
    assert not got[5].any() and case.status_bits() == 0
