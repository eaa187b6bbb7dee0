"""Decode steps with the cache declared ready (KVQ8_STEP_CACHE_READY) behind
calls whose kernels may still run: what the flag's contract allows to be read
is there, whatever the calls ahead were.  Every chain is captured, replayed
over caches whose slots were overwritten meanwhile, and compared bit for bit
with the same calls without the flag and with a synchronisation after each."""
import numpy as np
import pytest
import torch

from int8_quantized_kv_gb300 import kvq8

pytestmark = pytest.mark.gpu
HD = 128


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Steps:
    """A cache that holds L0 tokens of every sequence, and n new tokens."""

    def __init__(self, batch, nkv, group, L0, n, seed):
        rng = np.random.default_rng(seed)
        self.mb = (L0 + n + 255) // 256
        nb = batch * self.mb
        self.table = _dev(rng.permutation(nb).astype(np.int32).reshape(batch, self.mb))
        self.cache, self.wsum = kvq8.alloc_cache(nb, nkv), torch.zeros((nb, nkv, 256), device="cuda")
        g = torch.Generator("cuda").manual_seed(seed)
        rows = lambda *s: torch.randn((*s, HD), generator=g, device="cuda")  # noqa: E731
        self.old = rows(batch, L0, nkv), rows(batch, L0, nkv)
        self.k, self.v = rows(n, batch, nkv), 5 * rows(n, batch, nkv)
        # queries along the new tokens' keys, so that these carry the softmax
        self.q = (self.k[:, :, :, None] + 0.3 * rows(n, batch, nkv, group)).flatten(2, 3).contiguous()
        self.lens = [torch.full((batch,), L0 + i + 1, dtype=torch.int32, device="cuda") for i in range(n)]
        self.windows = torch.full((batch,), 100, dtype=torch.int32, device="cuda")
        self.out = torch.empty_like(self.q)
        self.ws = kvq8.alloc_weights_workspace(batch, nkv * group, nkv, self.mb)
        self.zero = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reset(self):
        """The old tokens in place, every other slot something else."""
        self.cache.k_pool.fill_(99)
        self.cache.v_pool.fill_(-99)
        self.cache.k_scale.fill_(0.5)
        self.cache.v_scale.fill_(9.0)
        self.out.fill_(float("nan"))
        kvq8.quantize_append(*self.old, self.zero, self.table, self.cache)
        torch.cuda.synchronize()

    def step(self, i, kind):
        a = (self.q[i], self.k[i], self.v[i], self.cache, self.table, self.lens[i])
        if kind == "window":
            kvq8.decode_step_window(*a, self.windows, 4, self.out[i], self.ws, dev_status=self.status)
        elif kind == "weights":
            kvq8.decode_step_weights(*a, self.out[i], self.wsum, self.ws, dev_status=self.status)
        else:
            kvq8.decode_step(*a, self.out[i], self.ws, dev_status=self.status, cache_ready=kind == "ready")


def _replays(calls, reset, outs, times=10):
    """calls(ready, sync): the same bits from a graph of the flagged calls as from calls in turn."""
    reset()
    calls(False, torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    assert all(torch.isfinite(w).all() for w in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(True, lambda: None)
    for _ in range(times):
        reset()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("ahead", ["plain", "ready", "window", "weights"])
@pytest.mark.parametrize("batch, nkv, group, L0", [(1, 1, 1, 1), (1, 2, 1, 61), (1, 8, 2, 190), (3, 1, 8, 253),
                                                   (4, 8, 4, 1021), (28, 8, 2, 1533), (1, 8, 2, 8190)])
def test_token_of_the_step_ahead(gpu_lib, batch, nkv, group, L0, ahead):
    # each flagged step attends to the token that the step ahead of it appends
    n = 6
    s = Steps(batch, nkv, group, L0, n, seed=L0)

    def calls(ready, sync):
        for i in range(n):
            if ahead == "ready" and i:
                s.step(i, "ready" if ready else "plain")
            else:
                s.step(i, ahead if i % 2 == 0 and ahead != "ready" else "ready" if ready and i else "plain")
            sync()

    _replays(calls, s.reset, [s.out])
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("between", ["step", "ready", "window", "weights", "attn", "int4", "combine"])
@pytest.mark.parametrize("batch, nkv", [(1, 2), (28, 8)])
def test_rows_of_the_call_before_the_one_ahead(gpu_lib, batch, nkv, between):
    # a bulk append, a call on another cache, then a flagged step over the appended rows
    a, b = Steps(1, 2, 2, 700, 1, 50), Steps(batch, nkv, 2, 1800, 1, 51)
    four = kvq8.alloc_cache4(a.mb, 2)

    def calls(ready, sync):
        if between == "combine":
            kvq8.decode_split(a.q[0], a.cache, a.table, a.lens[0], a.ws, dev_status=a.status)
        kvq8.quantize_append(*b.old, b.zero, b.table, b.cache, dev_status=b.status)
        sync()
        if between == "attn":
            kvq8.decode_attn(a.q[0], a.cache, a.table, a.lens[0], a.out[0], a.ws, dev_status=a.status)
        elif between == "combine":
            kvq8.decode_combine(1, 4, 2, a.mb, a.lens[0], a.ws, a.out[0])
        elif between == "int4":
            kvq8.decode_step4(a.q[0], a.k[0], a.v[0], four, a.table, a.lens[0], a.out[0], a.ws, dev_status=a.status)
        else:
            a.step(0, between if ready or between != "ready" else "plain")
        sync()
        b.step(0, "ready" if ready else "plain")

    def reset():
        a.reset()
        b.reset()
        for x in (*b.cache, *four):
            x.zero_()
        torch.cuda.synchronize()

    _replays(calls, reset, [a.out, b.out])
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0
