"""Eviction by accumulated weight: the kept lists, the copied codes, scales and
weights are exact, and nothing else is written."""
import numpy as np
import pytest
import torch

from int8_quantized_kv_gb300 import kvq8
from kvq8_harness import k_rows_logical, v_rows_logical

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, lens, keep, nkv, seed=0, weights=None, dst_blocks=None, table_blocks=None):
        rng = np.random.default_rng(seed)
        self.lens, self.keep, self.nkv = list(lens), keep, nkv
        batch = len(lens)
        self.mb = max(1, max((n + 255) // 256 for n in lens)) if table_blocks is None else table_blocks
        self.dmb = (keep + 255) // 256 if dst_blocks is None else dst_blocks
        ids = rng.permutation(batch * (self.mb + self.dmb) + 2).astype(np.int32)
        self.nb = len(ids)
        self.table = ids[:batch * self.mb].reshape(batch, self.mb)
        self.dst = ids[batch * self.mb:batch * (self.mb + self.dmb)].reshape(batch, self.dmb)
        self.kp = rng.integers(-127, 128, (self.nb, nkv, 256, 128), np.int8)
        self.vp = rng.integers(-127, 128, (self.nb, nkv, 4, 128, 64), np.int8)
        self.ks = rng.random((self.nb, nkv, 256), np.float32)
        self.vs = rng.random((self.nb, nkv, 256), np.float32)
        w = rng.random((self.nb, nkv, 256), np.float32)
        self.w = w if weights is None else weights(rng, w)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, first=0, recent=0, table=None, dst=None, lens=None):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.cache = kvq8.KVCache(d(self.kp), d(self.vp), d(self.ks), d(self.vs))
        self.wsum = d(self.w)
        self.kept = torch.full((len(self.lens), self.nkv, self.keep), -99, dtype=torch.int32, device="cuda")
        self.new_lens = torch.full((len(self.lens),), -99, dtype=torch.int32, device="cuda")
        kvq8.evict(self.cache, self.wsum, d(self.table if table is None else table),
                   d(np.array(self.lens if lens is None else lens, np.int32)), self.keep,
                   d(self.dst if dst is None else dst), self.kept, self.new_lens, n_first=first, n_recent=recent,
                   dev_status=self.status)
        torch.cuda.synchronize()
        return self.kept.cpu().numpy(), self.new_lens.cpu().numpy()

    def want(self, b, h, first, recent):
        n = self.lens[b]
        t = np.arange(n)
        w = self.w[self.table[b, t // 256], h, t % 256].astype(np.float64)
        w = np.where(np.isnan(w), -np.inf, w)
        rank = np.where(np.isnan(self.w[self.table[b, t // 256], h, t % 256]), 1, 0)
        must = (t < first) | (t >= n - recent)
        order = np.lexsort((t, rank, -w, ~must))         # forced first, then larger, then non-NaN, then lower
        return np.sort(order[:min(n, self.keep)])

    def check(self, first=0, recent=0):
        kept, new_lens = self.run(first, recent)
        kp, vp = self.kp.copy(), self.vp.copy()
        ks, vs, w = self.ks.copy(), self.vs.copy(), self.w.copy()
        for b, n in enumerate(self.lens):
            m = min(n, self.keep)
            assert new_lens[b] == m
            j = np.arange(m)
            for h in range(self.nkv):
                src = self.want(b, h, first, recent)
                assert np.array_equal(kept[b, h, :m], src), (b, h)
                assert np.all(kept[b, h, m:] == -1)
                sp, ss, dp, ds = self.table[b, src // 256], src % 256, self.dst[b, j // 256], j % 256
                rows = k_rows_logical(self.kp, sp, h, ss).reshape(m, 8, 16)
                pos = np.arange(8)[None, :] ^ (ds & 7)[:, None]
                at = np.empty_like(rows)
                np.put_along_axis(at, pos[:, :, None], rows, axis=1)
                kp[dp, h, ds] = at.reshape(m, 128)
                vp[dp, h, ds // 64, :, ds % 64] = v_rows_logical(self.vp, sp, h, ss)
                for x, y in ((ks, self.ks), (vs, self.vs), (w, self.w)):
                    x[dp, h, ds] = y[sp, h, ss]
        # every byte of the pools: the destinations' kept slots as above, all else as it was
        for got, ref, name in ((self.cache.k_pool, kp, "k"), (self.cache.v_pool, vp, "v"),
                               (self.cache.k_scale, ks, "ks"), (self.cache.v_scale, vs, "vs"), (self.wsum, w, "w")):
            got = got.cpu().numpy()
            assert np.array_equal(got.view(np.uint8), ref.view(np.uint8)), name
        assert int(self.status.item()) == 0


@pytest.mark.parametrize("keep", [1, 2, 63, 64, 65, 200, 256, 257, 700])
def test_kept_and_copied(gpu_lib, keep):
    Pool([0, 1, keep, keep + 1, max(1, keep - 1), 3 * keep + 17, 1200], keep, 2, seed=keep).check()


@pytest.mark.parametrize("first,recent", [(0, 0), (1, 0), (0, 1), (4, 64), (100, 200), (0, 300), (300, 0), (150, 150)])
def test_first_and_recent_tokens_stay(gpu_lib, first, recent):
    Pool([1, 299, 300, 301, 450, 2000], 300, 2, seed=first + recent).check(first, recent)


def _ties(rng, w):
    return (np.floor(w * 4) / 4).astype(np.float32)


def _all_equal(rng, w):
    return np.zeros_like(w)


def _signed_zeros(rng, w):
    return np.where(w < 0.5, np.float32(-0.0), np.float32(0.0)).astype(np.float32)


def _wild(rng, w):
    x = (rng.standard_normal(w.shape) * 10.0 ** rng.integers(-40, 38, w.shape)).astype(np.float32)
    x[w < 0.05] = np.nan
    x[(w >= 0.05) & (w < 0.08)] = np.inf
    x[(w >= 0.08) & (w < 0.11)] = -np.inf
    x[(w >= 0.11) & (w < 0.14)] = np.finfo(np.float32).min
    x[(w >= 0.14) & (w < 0.17)] = -0.0
    x[(w >= 0.17) & (w < 0.2)] = 0.0
    return x


def _near(rng, w):   # equal but for the last bits
    return (np.float32(1.0) + (w * 16).astype(np.int32) * np.float32(2.0**-23)).astype(np.float32)


@pytest.mark.parametrize("weights", [_ties, _all_equal, _signed_zeros, _wild, _near])
@pytest.mark.parametrize("keep", [5, 300, 1250])
def test_order_of_equal_and_odd_weights(gpu_lib, weights, keep):
    Pool([1300, 640, 1301], keep, 2, seed=keep, weights=weights).check(2, min(3, keep - 2))


def test_long_sequences_and_many_heads(gpu_lib):
    Pool([30000, 100, 12345], 5000, 1, seed=7, weights=_ties).check(4, 1000)
    Pool([3000] * 3, 1000, 8, seed=8).check(4, 100)


def test_wider_tables_than_needed(gpu_lib):
    p = Pool([500, 300], 200, 2, seed=9, dst_blocks=3, table_blocks=6)
    p.table[:, 2:], p.dst[:, 1:] = -1, -1                      # entries that no token needs
    p.check(1, 10)


def test_bad_ids_leave_the_sequence_out(gpu_lib):
    p = Pool([600, 600, 600, 600, 600, 600], 300, 2, seed=10)
    table, dst = p.table.copy(), p.dst.copy()
    table[0, 1] = -1
    table[1, 2] = p.nb
    dst[2, 1] = -5
    dst[3, 0] = table[3, 2]                                     # a destination among the sources
    dst[4, 1] = dst[4, 0]                                       # listed twice
    kept, new_lens = p.run(4, 10, table=table, dst=dst)
    assert int(p.status.item()) == kvq8.DEV_BAD_BLOCK_ID
    assert np.array_equal(new_lens, [0, 0, 0, 0, 0, 300]) and np.all(kept[:5] == -1)
    for h in range(2):
        assert np.array_equal(kept[5, h], p.want(5, h, 4, 10))
    mine = p.dst[5]
    others = np.setdiff1d(np.arange(p.nb), mine)
    for got, was in ((p.cache.k_pool, p.kp), (p.cache.v_pool, p.vp), (p.cache.k_scale, p.ks), (p.wsum, p.w)):
        assert np.array_equal(got.cpu().numpy()[others], was[others])


def test_lengths_outside_the_table(gpu_lib):
    p = Pool([600, 600], 300, 1, seed=11)
    kept, new_lens = p.run(lens=[-4, 100000])
    assert int(p.status.item()) == kvq8.DEV_BAD_CTX_LEN
    assert np.array_equal(new_lens, [0, 300]) and np.all(kept[0] == -1)
    p.lens[1] = 768
    assert np.array_equal(kept[1, 0], p.want(1, 0, 0, 0))


@pytest.mark.parametrize("longest", [16384, 40001, 131067])
def test_clusters(gpu_lib, longest):
    # tables of at least 16384 tokens: 2, 4 and 8 CTAs per unit, with short and empty sequences beside the long one,
    # keys beyond a CTA's shared memory, everything kept, and ties over the CTAs' borders
    lens = [longest, 0, 5, 3000, longest - 4097, 8193]
    Pool(lens, 3000, 1, seed=longest).check(4, 100)
    Pool(lens[:3], 9000, 2, seed=longest + 1, weights=_ties).check(0, 0)
    Pool(lens[::4], 1, 1, seed=longest + 2, weights=_all_equal).check(0, 0)
    p = Pool([longest, longest, 700], 500, 1, seed=longest + 3)
    table, dst = p.table.copy(), p.dst.copy()
    table[0, (longest - 1) // 256] = p.nb
    dst[2, 1] = table[2, 0]
    kept, new_lens = p.run(4, 10, table=table, dst=dst)
    assert int(p.status.item()) == kvq8.DEV_BAD_BLOCK_ID
    assert np.array_equal(new_lens, [0, 500, 0]) and np.all(kept[[0, 2]] == -1)
    assert np.array_equal(kept[1, 0], p.want(1, 0, 4, 10))


def test_wide_table_short_sequences(gpu_lib):
    # more units than SMs with a wide table: keys beyond a CTA's shared memory in one of them
    lens = [300] * 159 + [25000]
    Pool(lens, 200, 1, seed=5).check(0, 20)


@pytest.mark.parametrize("keep", [64, 500])
def test_lengths_in_place(gpu_lib, keep):
    # new_lens written over ctx_lens while other heads of the sequences may still wait for their selection
    p = Pool([3000, 64, 0, 501] * 15, keep, 7, seed=keep)
    kept, new_lens = p.run(4, 20)
    q = Pool([3000, 64, 0, 501] * 15, keep, 7, seed=keep)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    cache, wsum, table, dst = kvq8.KVCache(*(d(x) for x in (q.kp, q.vp, q.ks, q.vs))), d(q.w), d(q.table), d(q.dst)
    for _ in range(5):
        lens, again = d(np.array(q.lens, np.int32)), torch.empty_like(p.kept)
        kvq8.evict(cache, wsum, table, lens, keep, dst, again, lens, n_first=4, n_recent=20, dev_status=q.status)
        assert np.array_equal(lens.cpu().numpy(), new_lens) and np.array_equal(again.cpu().numpy(), kept)
    assert all(torch.equal(a, b) for a, b in zip(cache, p.cache)) and int(q.status.item()) == 0
