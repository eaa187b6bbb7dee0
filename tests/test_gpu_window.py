"""Windowed decode (sliding window + first tokens) against the oracle on the
visible rows, against the plain decode where everything is visible, and the windows, sinks and tables at which it can go wrong."""
import numpy as np
import pytest
import torch

import cache_ops_ref as ref
from int8_quantized_kv_gb300 import kvq8
from int8_quantized_kv_gb300 import workloads as wl
from kvq8_harness import Case, StepCase, assert_close

pytestmark = pytest.mark.gpu


def _visible(L, window, sinks):
    t = np.arange(L)
    return t[(t < sinks) | (t >= L - max(1, window))]


def _run(case, windows, sinks, table=None, step=False):
    cfg = case.cfg
    out = torch.full_like(case.q_d, float("nan"))
    ws = kvq8.alloc_workspace(cfg.batch, cfg.nqh, cfg.nkv, case.max_blocks)
    win = torch.tensor(windows, dtype=torch.int32, device="cuda")
    args = (case.cache, case.table_d if table is None else table, case.lens_d, win, sinks, out, ws)
    if step:
        kvq8.decode_step_window(case.q_d, case.k_new_d, case.v_new_d, *args, dev_status=case.status)
    else:
        kvq8.decode_attn_window(case.q_d, *args, dev_status=case.status)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def _check(case, got, windows, sinks, step=False):
    cfg, G = case.cfg, case.cfg.group
    for b in range(cfg.batch):
        L = int(case.lens[b])
        if L == 0:
            assert not got[b].any()
            continue
        vis = _visible(L, windows[b], sinks)
        for h in range(cfg.nkv):
            k, v = wl.unit_kv(cfg, b, h, L)
            want = ref.decode(case.q[b, h * G:(h + 1) * G], *ref.unit_rows(k[vis], v[vis], step))
            assert_close(got[b, h * G:(h + 1) * G], want, f"b={b} h={h} L={L} window={windows[b]} sinks={sinks}")


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("sinks", [0, 1, 4, 64, 65, 700])
def test_window_matches_the_oracle_on_visible_rows(gpu_lib, G, sinks):
    # per row: window 1, inside one stage, on and next to stage and block edges,
    # one that just meets the sinks, one longer than the context
    windows = [1, 2, 63, 64, 65, 255, 256, 257, 1000, 1, 640, 5000]
    lens = [1, 2, 64, 65, 700, 1024, 1025, 1090, 1003, 1300, 1341, 900]
    cfg = wl.Workload("w", 700 + G, batch=len(lens), nqh=2 * G, nkv=2)
    case = Case(cfg, lens=lens)
    got = _run(case, windows, sinks)
    _check(case, got, windows, sinks)
    assert case.status_bits() == 0


def test_window_longer_than_the_context_matches_the_plain_decode(gpu_lib):
    for nqh, nkv, batch in ((8, 8, 3), (32, 8, 3), (16, 2, 3)):
        cfg = wl.Workload("w", 720, batch=batch, nqh=nqh, nkv=nkv)
        case = Case(cfg, lens=[1500, 333, 64][:batch])
        plain = case.decode()
        got = _run(case, [1500, 5000, 64], 0)
        # (the two round the query's factor differently: equal unless a code sits on a border)
        assert_close(got, plain)
        assert np.array_equal(_run(case, [2**31 - 1] * 3, 2**31 - 1), got)
        assert np.array_equal(_run(case, [1] * 3, 1500), got)                # all are first tokens


def test_empty_and_one_token_rows(gpu_lib):
    cfg = wl.Workload("w", 721, batch=4, nqh=8, nkv=2)
    case = Case(cfg, lens=[0, 1, 0, 200])
    got = _run(case, [10, 10, 1, 10], 3)
    _check(case, got, [10, 10, 1, 10], 3)


def test_blocks_out_of_sight_are_not_looked_at(gpu_lib):
    cfg = wl.Workload("w", 722, batch=2, nqh=4, nkv=2)
    lens, windows, sinks = [2600, 2000], [300, 520], 5
    case = Case(cfg, lens=lens)
    want = _run(case, windows, sinks)
    table = case.table.copy()
    for b in range(2):
        first = (lens[b] - windows[b]) // 64 * 64 // 256
        table[b, 1:first] = (-1, 10**9)[b]                                   # given back
    # what lies in them now: NaN scales
    gone = np.concatenate([case.table[b, 1:(lens[b] - windows[b]) // 64 * 64 // 256] for b in range(2)])
    case.cache.k_scale[gone.tolist()] = float("nan")
    case.cache.v_scale[gone.tolist()] = float("inf")
    got = _run(case, windows, sinks, table=torch.from_numpy(table).cuda())
    assert np.array_equal(got, want) and case.status_bits() == 0


def test_masked_tokens_of_a_read_stage_do_not_count(gpu_lib):
    # NaN, infinite and lowest scales at masked tokens of the stages that are read
    cfg = wl.Workload("w", 723, batch=1, nqh=8, nkv=2)
    case = Case(cfg, lens=[1000])
    windows, sinks = [100], 3
    want = _run(case, windows, sinks)
    for t in list(range(3, 64)) + list(range(896, 900)):
        phys, slot = int(case.table[0, t // 256]), t % 256
        case.cache.k_scale[phys, :, slot] = (float("nan"), float("inf"), torch.finfo(torch.float32).min)[t % 3]
        case.cache.v_scale[phys, :, slot] = (float("inf"), torch.finfo(torch.float32).max, float("nan"))[t % 3]
    assert np.array_equal(_run(case, windows, sinks), want)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_step_appends_and_attends(gpu_lib, G):
    lens = [1, 64, 65, 257, 700, 1345, 0]
    windows = [1, 1, 64, 300, 30, 1000, 5]
    cfg = wl.Workload("w", 730 + G, batch=len(lens), nqh=2 * G, nkv=2)
    case = StepCase(cfg, lens=lens)
    before = [x.clone() for x in case.cache]
    got = _run(case, windows, 4, step=True)
    _check(case, got, windows, 4, step=True)
    pools = case.host_pools()
    for b in range(cfg.batch):
        for h in range(cfg.nkv):
            if lens[b]:
                for x, y in zip(case.gather_unit(pools, b, h), ref.unit_rows(*wl.unit_kv(cfg, b, h, lens[b]), True)):
                    assert np.array_equal(x, y), (b, h)
    # nothing else was written
    for x, y, name in zip(before, case.cache, ("k_pool", "v_pool", "k_scale", "v_scale")):
        diff = (x != y)
        assert int(diff.sum()) <= cfg.batch * cfg.nkv * 128, name


def test_bad_windows_lengths_and_blocks_are_flagged(gpu_lib):
    cfg = wl.Workload("w", 740, batch=3, nqh=4, nkv=2)
    case = Case(cfg, lens=[600, 600, 600])
    got = _run(case, [0, -7, 9], 2)                       # below 1: taken as 1
    assert case.status_bits() == kvq8.DEV_BAD_CTX_LEN
    _check(case, got, [1, 1, 9], 2)
    case.status.zero_()
    case.lens_d.copy_(torch.tensor([5000, -3, 600], dtype=torch.int32))   # clamped to the table
    got = _run(case, [50, 50, 50], 2)
    assert case.status_bits() & kvq8.DEV_BAD_CTX_LEN and not got[1].any()
    case.status.zero_()
    case.lens_d.copy_(torch.tensor([600, 600, 600], dtype=torch.int32))
    table = case.table.copy()
    table[0, 2], table[2, 0] = -1, case.num_blocks        # the window's block, the first tokens' block
    got = _run(case, [88, 88, 88], 2, table=torch.from_numpy(table).cuda())
    assert case.status_bits() == kvq8.DEV_BAD_BLOCK_ID
    assert np.all(np.isfinite(got))
    G = cfg.group
    for b, vis in ((0, np.arange(2)), (1, _visible(600, 88, 2)), (2, np.arange(512, 600))):
        for h in range(cfg.nkv):
            k, v = wl.unit_kv(cfg, b, h, 600)
            want = ref.decode(case.q[b, h * G:(h + 1) * G], *ref.unit_rows(k[vis], v[vis]))
            assert_close(got[b, h * G:(h + 1) * G], want, f"b={b} h={h}")


def test_many_rows_of_differing_windows(gpu_lib):
    rng = np.random.default_rng(5)
    batch = 40
    lens = rng.integers(1, 3000, batch).tolist()
    windows = rng.integers(1, 2500, batch).tolist()
    cfg = wl.Workload("w", 750, batch=batch, nqh=16, nkv=8)
    case = Case(cfg, lens=lens)
    got = _run(case, windows, 7)
    assert np.array_equal(got, _run(case, windows, 7))     # reproducible
    for b in rng.choice(batch, 6, replace=False):
        vis = _visible(lens[b], windows[b], 7)
        k, v = wl.unit_kv(cfg, int(b), 3, lens[b])
        assert_close(got[b, 6:8], ref.decode(case.q[b, 6:8], *ref.unit_rows(k[vis], v[vis])), f"b={b}")
