"""Norm + rotation + quantise-append against the formulas in 64 bits.

K codes, V codes and V scales are exact (V: in fp32, scale = max * fl(1/127),
code = round_half_even(v / scale)).  Tolerance of a query value and of a K
scale, in units of eps = 2^-24 (half a step of fp32) relative to the length of
the value's pair (u_a, u_b): the squares' sum passes 9 roundings, so its root
4.5; the mean's addition .5; the reciprocal root 2 ulp = 4; the products by r
and the weight 1 each; the rotation 2 |ac| + 3 |bs| + |y| <= 5.3.  Together
16.3 eps < 2^-19.9: 2^-19 below.  Inputs of 16 bits are exact in fp32."""
import numpy as np
import pytest
import torch

from cache_ops_ref import row_codes
from int8_quantized_kv_gb300 import kvq8
from kvq8_harness import k_rows_logical, v_rows_logical

pytestmark = pytest.mark.gpu
HD = 128
TOL = 2.0**-19
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _table(n_pos, theta=1e6):
    inv = theta ** (-np.arange(64) / 64.0)
    ang = np.arange(n_pos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _turned(x, w, eps, cs, pairs):
    """fp64 rows [..., 128] normed, weighted, rotated; the pair lengths [..., 128]."""
    u = x.astype(np.float64)
    if w is not None:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    c, s = cs[..., :64].astype(np.float64), cs[..., 64:].astype(np.float64)
    a, b = (u[..., 0::2], u[..., 1::2]) if pairs else (u[..., :64], u[..., 64:])
    y, n = np.empty_like(u), np.empty_like(u)
    ya, yb, r = a * c - b * s, b * c + a * s, np.hypot(a, b)
    if pairs:
        y[..., 0::2], y[..., 1::2], n[..., 0::2], n[..., 1::2] = ya, yb, r, r
    else:
        y[..., :64], y[..., 64:], n[..., :64], n[..., 64:] = ya, yb, r, r
    return y, n


def _k_codes(y):
    top = np.abs(y).max(-1, keepdims=True)
    v = np.where(top > 0, 127.0 * y / np.where(top > 0, top, 1.0), 0.0)
    return np.rint(v).astype(np.int8), top[..., 0] / 127.0, np.abs(np.abs(v - np.floor(v)) - 0.5)


class Case:
    def __init__(self, batch, n_new, nqh, nkv, dtype="fp32", start=0, n_pos=None, positions=None, n_tokens=None,
                 pairs=False, norm=True, packed=True, seed=0, eps=1e-6, x=None, wsum=True, table_blocks=None):
        rng = np.random.default_rng(seed)
        self.batch, self.n_new, self.nqh, self.nkv, self.pairs, self.eps = batch, n_new, nqh, nkv, pairs, eps
        self.start = np.broadcast_to(np.asarray(start, np.int32), (batch,)).copy()
        heads = nqh + 2 * nkv
        if x is None:
            x = rng.standard_normal((batch, n_new, heads, HD)) * (0.2 + 3 * rng.random((heads, HD)))
        t = torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[dtype])
        self.x = t.float().numpy()
        t = t.cuda()
        parts = (t[:, :, :nqh], t[:, :, nqh:nqh + nkv], t[:, :, nqh + nkv:])
        self.q, self.k, self.v = parts if packed else tuple(p.contiguous() for p in parts)
        w = lambda: (1 + 0.3 * rng.standard_normal(HD)).astype(np.float32) if norm else None  # noqa: E731
        self.qw, self.kw = w(), w()
        self.positions = positions
        pos = (self.start[:, None] + np.arange(n_new)) if positions is None else positions
        self.pos = np.asarray(pos)
        self.n_pos = int(max(self.pos.max() + 1, 1)) if n_pos is None else n_pos
        self.rope = _table(self.n_pos)
        need = (int(self.start.max()) + n_new + 255) // 256
        self.mb = need if table_blocks is None else table_blocks
        ids = rng.permutation(batch * self.mb + 2).astype(np.int32)
        self.nb, self.table = len(ids), ids[:batch * self.mb].reshape(batch, self.mb)
        self.n_tokens = n_tokens
        d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = kvq8.KVCache(torch.full((self.nb, nkv, 256, HD), 77, dtype=torch.int8, device="cuda"),
                                  torch.full((self.nb, nkv, 4, HD, 64), 77, dtype=torch.int8, device="cuda"),
                                  torch.full((self.nb, nkv, 256), 7.5, device="cuda"),
                                  torch.full((self.nb, nkv, 256), 7.5, device="cuda"))
        self.wsum = torch.full((self.nb, nkv, 256), 7.5, device="cuda") if wsum else None
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full((batch, n_new, nqh, HD), 7.5, device="cuda")
        self.dev = dict(qw=d(self.qw), kw=d(self.kw), rope=d(self.rope), start=d(self.start), table=d(self.table),
                        positions=d(None if positions is None else np.asarray(positions, np.int32)),
                        n_tokens=d(None if n_tokens is None else np.asarray(n_tokens, np.int32)))

    def call(self, stream=None):
        v = self.dev
        kvq8.norm_rope_append(self.q, self.k, self.v, v["qw"], v["kw"], self.eps, v["rope"], v["start"], v["table"],
                              self.cache, self.out, positions=v["positions"], n_tokens=v["n_tokens"],
                              interleaved=self.pairs, weight_sum=self.wsum, dev_status=self.status, stream=stream)

    def check(self, skip_rows=(), skip_cache=(), nonfinite=False):
        """Outputs and the whole cache; skip_rows, skip_cache: (b, i) not written (at all, to the cache)."""
        torch.cuda.synchronize()
        nqh, nkv = self.nqh, self.nkv
        out = self.out.cpu().numpy()
        kp, vp = self.cache.k_pool.cpu().numpy(), self.cache.v_pool.cpu().numpy()
        ks, vs = self.cache.k_scale.cpu().numpy(), self.cache.v_scale.cpu().numpy()
        ws = None if self.wsum is None else self.wsum.cpu().numpy()
        written = np.zeros((self.nb, nkv, 256), bool)
        for b in range(self.batch):
            real = self.n_new if self.n_tokens is None else min(self.n_new, max(0, self.n_tokens[b]))
            gone = {i for bb, i in skip_rows if bb == b}
            rows = np.array([i for i in range(real) if i not in gone], int)
            rest = np.setdiff1d(np.arange(self.n_new), rows)
            assert np.all(out[b, rest] == 7.5)
            if not len(rows):
                continue
            cs = self.rope[self.pos[b, rows]][:, None, :]
            with np.errstate(all="ignore"):
                yq, nq = _turned(self.x[b, rows][:, :nqh], self.qw, self.eps, cs, self.pairs)
                if nonfinite:
                    ok = np.isfinite(yq)
                    assert np.array_equal(ok, np.isfinite(out[b, rows]))
                    yq, nq, got = yq[ok], nq[ok], out[b, rows][ok]
                else:
                    got = out[b, rows]
                assert np.all(np.abs(got - yq) <= TOL * nq + 1e-37), np.abs(got - yq).max()
                rows = np.array([i for i in rows if (b, i) not in skip_cache], int)
                if not len(rows):
                    continue
                cs = self.rope[self.pos[b, rows]][:, None, :]
                yk, nk = _turned(self.x[b, rows][:, nqh:nqh + nkv], self.kw, self.eps, cs, self.pairs)
            bad = ~np.isfinite(yk).all(-1) | (np.abs(yk).max(-1) > np.finfo(np.float32).max)
            yk[bad] = 0.0
            codes, scale, border = _k_codes(yk)
            # the exact codes are meant: a case whose values sit on a border to within fp64 would say nothing
            assert border[~bad].min(initial=1) > 1e-10 or not self._generic
            phys, slot = self.table[b, (self.start[b] + rows) // 256], (self.start[b] + rows) % 256
            vc, vsc = row_codes(self.x[b, rows][:, nqh + nkv:])
            for h in range(nkv):
                got = k_rows_logical(kp, phys, h, slot)
                assert np.array_equal(got, codes[:, h]), (b, h, np.argwhere(got != codes[:, h])[:5])
                near = np.where(bad[:, h], 0.0, TOL * nk[:, h].max(-1) / 127.0)      # a row of zeros: exact
                assert np.all(np.abs(ks[phys, h, slot] - scale[:, h]) <= near + 1e-44)
                assert np.array_equal(v_rows_logical(vp, phys, h, slot), vc[:, h])
                assert np.array_equal(vs[phys, h, slot].view(np.uint32), vsc[:, h].view(np.uint32))
                if ws is not None:
                    assert np.all(ws[phys, h, slot] == 0.0)
                written[phys, h, slot] = True
        idle = ~written
        assert np.all(kp[idle] == 77) and np.all(ks[idle] == 7.5) and np.all(vs[idle] == 7.5)
        assert np.all(vp.transpose(0, 1, 2, 4, 3).reshape(self.nb, nkv, 256, HD)[idle] == 77)
        if ws is not None:
            assert np.all(ws[idle] == 7.5)

    _generic = True


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_one_token(gpu_lib, dtype, pairs, norm):
    c = Case(3, 1, 8, 2, dtype, start=[0, 255, 300], pairs=pairs, norm=norm, seed=1)
    c.call()
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("start,n_new", [(0, 2), (0, 16), (15, 2), (0, 64), (37, 200), (250, 700), (1, 17), (3, 61)])
def test_runs(gpu_lib, dtype, pairs, start, n_new):
    c = Case(2, n_new, 4, 2, dtype, start=[start, start + 5], pairs=pairs, seed=n_new)
    c.call()
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("nqh,nkv", [(1, 1), (5, 5), (8, 1), (12, 3), (16, 8), (64, 8)])
@pytest.mark.parametrize("n_new", [1, 33])
def test_head_layouts(gpu_lib, nqh, nkv, n_new):
    for packed in (True, False):
        c = Case(2, n_new, nqh, nkv, "bf16", start=9, packed=packed, seed=nqh, wsum=packed)
        c.call()
        c.check()


def test_many_values(gpu_lib):
    # 2.6 million K codes, exact: borders between codes are met at every distance
    for dtype, norm in (("fp32", True), ("bf16", True), ("fp32", False)):
        c = Case(2, 1300, 2, 2, dtype, start=3, norm=norm, seed=21)
        c._generic = False
        c.call()
        c.check()
    c = Case(4, 640, 8, 8, "fp16", start=0, seed=22)
    c._generic = False
    c.call()
    c.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_long_runs(gpu_lib, dtype, pairs):
    # enough new tokens for value tasks of 16 slots, with and without padding
    c = Case(4, 900, 8, 8, dtype, start=[3, 16, 255, 31], pairs=pairs, seed=23)
    c._generic = False
    c.call()
    c.check()
    c = Case(8, 1300, 8, 8, dtype, start=[5, 0, 8, 77, 1, 2, 300, 15], pairs=pairs, seed=24,
             n_tokens=[1300, 0, 1, 16, 900, 33, 1299, 640])
    c._generic = False
    for b, n in enumerate(c.n_tokens):
        c.v[b, n:] = float("nan")
    c.call()
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("n_new", [1, 40])
def test_positions_ahead_of_the_slots_and_far(gpu_lib, n_new):
    pos = np.array([[100000], [7], [131071 - n_new + 1]]) + np.arange(n_new)
    c = Case(3, n_new, 4, 2, "fp32", start=[70, 0, 255], positions=pos, seed=3)
    c.call()
    c.check()
    # any order of positions, repeated ones among them
    pos = np.random.default_rng(1).integers(0, 50, (3, n_new))
    c = Case(3, n_new, 4, 2, "fp32", start=[70, 0, 255], positions=pos, seed=4)
    c.call()
    c.check()


def test_padded_batch(gpu_lib):
    for n_tokens in ([0, 1, 45, 100, 99], [100, -3, 1000, 16, 17]):
        c = Case(5, 100, 4, 2, "bf16", start=[0, 10, 200, 33, 64], n_tokens=n_tokens, seed=5)
        # padding holds anything
        for b, n in enumerate(n_tokens):
            c.q[b, max(n, 0):] = float("nan")
            c.k[b, max(n, 0):] = float("inf")
        c.call()
        c.check()
        assert int(c.status.item()) == 0


def test_exact_ties_round_to_even(gpu_lib):
    # position 0 (no turn), no norm: 127 y / max|y| = y for a maximum of 127, with halves
    x = np.zeros((1, 1, 3, HD))
    y = np.arange(HD) - 63.5
    y[0] = 127.0
    x[0, 0, 1] = y
    x[0, 0, 2] = y
    x[0, 0, 0] = y
    c = Case(1, 1, 1, 1, "fp32", start=0, norm=False, x=x)
    c._generic = False
    c.call()
    c.check()
    kp = c.cache.k_pool.cpu().numpy()
    got = k_rows_logical(kp, np.array([c.table[0, 0]]), 0, np.array([0]))[0]
    assert got[1] == -62 and got[2] == -62 and got[63] == 0 and got[64] == 0 and got[65] == 2


def test_near_ties(gpu_lib):
    # values one fp32 step beside each border, where fp32 arithmetic alone cannot tell
    rng = np.random.default_rng(8)
    x = np.zeros((1, 64, 3, HD), np.float32)
    for i in range(64):
        m = np.float32(rng.uniform(0.3, 30))
        r = rng.integers(-126, 126, HD) + 0.5
        y = (r * np.float64(m) / 127.0).astype(np.float32)
        y = np.nextafter(y, np.where(rng.random(HD) < 0.5, np.float32(1e30), np.float32(-1e30)))
        y[rng.integers(HD)] = m
        x[0, i] = y
    c = Case(1, 64, 1, 1, "fp32", start=0, positions=np.zeros((1, 64), int), n_pos=1, norm=False, x=x)
    c._generic = False
    c.call()
    c.check()
    c = Case(1, 64, 1, 1, "fp32", start=0, positions=np.zeros((1, 64), int), n_pos=1, norm=True, x=x)
    c._generic = False
    c.call()
    c.check()


@pytest.mark.parametrize("n_new", [1, 20])
def test_large_small_and_zero_rows(gpu_lib, n_new):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((1, n_new, 12, HD))
    x *= np.array([1e-30, 1e-10, 1.0, 1e10, 1e25, 1e36, 0.0, 1e-38, 1e-3, 1e18, 1e36, 1e-10])[:, None]
    x[0, 0, 8, :] = 0.0
    x[0, 0, 9, :] = 0.0
    c = Case(1, n_new, 4, 4, "fp32", x=x, seed=9)
    c.call()
    c.check()
    assert int(c.status.item()) == 0
    c = Case(1, n_new, 4, 4, "fp32", x=np.minimum(np.abs(x), 1e37), norm=False, seed=9)
    c.call()
    c.check()


@pytest.mark.parametrize("n_new", [1, 20])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_normed_rows_up_to_the_largest_value(gpu_lib, n_new, dtype, pairs):
    # squares whose sum passes 2^128 even of much smaller rows: equal values of 1e38, the type's largest ones,
    # spread rows, one such value beside small ones, and an ordinary row in the same task
    rng = np.random.default_rng(35)
    most = float(torch.finfo(TYPES[dtype]).max)
    x = rng.standard_normal((1, n_new, 24, HD))
    for h, row in enumerate([np.full(HD, 1e38), np.full(HD, most), most * rng.choice([-1, 1], HD),
                             3e37 * np.clip(rng.standard_normal(HD), -3, 3), 1e18 * rng.standard_normal(HD), None,
                             np.where(np.arange(HD) == 77, most, 1.0), most * rng.uniform(-1, 1, HD)]):
        for first in (0, 8, 16):              # queries, keys, values
            if row is not None:
                x[:, :, first + h] = row
    c = Case(1, n_new, 8, 8, dtype, start=11, pairs=pairs, x=x, seed=36)
    c._generic = False
    c.call()
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("n_new", [1, 50])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nonfinite_rows(gpu_lib, n_new, dtype):
    rng = np.random.default_rng(10)
    for pairs in (False, True):
        x = rng.standard_normal((2, n_new, 8, HD))
        for j, (b, h) in enumerate([(0, 0), (0, 4), (0, 6), (1, 5), (1, 7), (1, 1)]):
            x[b, rng.integers(n_new), h, rng.integers(HD)] = (np.nan, np.inf, -np.inf)[j % 3]
        c = Case(2, n_new, 4, 2, dtype, start=20, x=x, pairs=pairs, seed=11)
        c.call()
        c.check(nonfinite=True)
        assert int(c.status.item()) == kvq8.DEV_NONFINITE


@pytest.mark.parametrize("n_new", [1, 30])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_weight_and_table(gpu_lib, n_new, value):
    # one weight: every key row comes out with it; one table entry: the rows at that position
    c = Case(2, n_new, 4, 2, "bf16", start=3, seed=31)
    c.kw[70] = value
    c.dev["kw"] = torch.from_numpy(c.kw).cuda()
    c.call()
    c.check()
    assert int(c.status.item()) == kvq8.DEV_NONFINITE and not c.cache.k_scale[c.table[0, 0], :, 3:3 + n_new].any()
    c = Case(2, n_new, 4, 2, "fp32", start=3, seed=32)
    c.rope[3 + n_new // 2, 64 + 17] = value
    c.dev["rope"] = torch.from_numpy(c.rope).cuda()
    c.call()
    c.check(nonfinite=True)
    assert int(c.status.item()) == kvq8.DEV_NONFINITE


def test_borders_and_several_maxima(gpu_lib):
    # rows with many values on and next to borders and the maximum taken several times, with either sign
    rng = np.random.default_rng(33)
    x = np.zeros((1, 96, 12, HD), np.float32)
    for i in range(96):
        for h in range(4, 8):
            m = np.float32(2.0 ** rng.integers(-20, 20)) * np.float32(127 if i % 2 else rng.integers(1, 2**20))
            r = rng.integers(-127, 127, HD) + (0.5 if i % 3 else rng.choice([0.0, 0.5], HD))
            y = (r * np.float64(m) / 127.0).astype(np.float32)
            step = rng.integers(-1, 2, HD)
            y = np.where(step == 0, y, np.nextafter(y, np.float32(1e38) * step.astype(np.float32)))
            y = np.clip(y, -m, m)
            y[rng.choice(HD, 1 + i % 5, replace=False)] = m * rng.choice([-1, 1]).astype(np.float32)
            x[0, i, h] = y
    for norm, pos in ((False, np.zeros((1, 96), int)), (True, np.zeros((1, 96), int)), (False, None), (True, None)):
        for pairs in (False, True):
            c = Case(1, 96, 4, 4, "fp32", start=7, positions=pos, norm=norm, pairs=pairs, x=x, seed=34)
            c._generic = False
            c.call()
            c.check()


@pytest.mark.parametrize("n_new", [1, 20])
def test_bad_positions_and_blocks(gpu_lib, n_new):
    last = n_new - 1
    # rotation positions outside the table: the token is skipped
    pos = np.tile(np.arange(n_new), (3, 1))
    pos[0, 0], pos[2, last] = -1, 64
    c = Case(3, n_new, 4, 2, "fp32", start=30, positions=np.clip(pos, 0, 63), n_pos=64, seed=12)
    c.dev["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
    c.call()
    c.check(skip_rows={(0, 0), (2, last)})
    assert int(c.status.item()) == kvq8.DEV_BAD_POSITION
    # places outside the block table or the pool: queries are written, the cache is not
    c = Case(3, n_new, 4, 2, "fp32", start=30, positions=np.tile(np.arange(n_new), (3, 1)), table_blocks=1, seed=13)
    c.start[:] = [-5, 250, 30]
    c.dev["start"] = torch.from_numpy(c.start).cuda()
    table = c.table.copy()
    table[2, 0] = c.nb
    c.dev["table"] = torch.from_numpy(table).cuda()
    c.call()
    skip = {(0, i) for i in range(n_new) if i < 5} | {(1, i) for i in range(n_new) if 250 + i >= 256}
    skip |= {(2, i) for i in range(n_new)}
    c.check(skip_cache=skip)
    want = kvq8.DEV_BAD_BLOCK_ID | kvq8.DEV_BAD_POSITION
    assert int(c.status.item()) == want


def test_value_rows_against_the_plain_append(gpu_lib):
    c = Case(2, 130, 2, 2, "fp32", start=[5, 60], packed=False, seed=14)
    c.call()
    other = kvq8.alloc_cache(c.nb, 2)
    kvq8.quantize_append(c.k, c.v, c.dev["start"], c.dev["table"], other)
    torch.cuda.synchronize()
    for b in range(2):
        t = c.start[b] + np.arange(130)
        phys, slot = c.table[b, t // 256], t % 256
        for h in range(2):
            a, b_ = c.cache.v_scale.cpu().numpy()[phys, h, slot], other.v_scale.cpu().numpy()[phys, h, slot]
            assert np.abs(a.view(np.int32) - b_.view(np.int32)).max() <= 1      # the last bit at most
            same = a == b_
            assert np.array_equal(v_rows_logical(c.cache.v_pool.cpu().numpy(), phys, h, slot)[same],
                                  v_rows_logical(other.v_pool.cpu().numpy(), phys, h, slot)[same])
            assert same.mean() > 0.5


def test_rope_table(gpu_lib):
    inv = 5e5 ** (-np.arange(64) / 64.0)
    n = 131072
    got = kvq8.rope_table(torch.from_numpy(inv).cuda(), n).cpu().numpy()
    rows = np.r_[0:50, 1000:1010, n - 50:n]
    ang = rows[:, None] * inv
    # one rounding to fp32 (2^-24 of a value up to 1), the angle's own rounding 2^-53 * 1.3e5, and the 64-bit functions
    assert np.abs(got[rows, :64] - np.cos(ang)).max() <= 2.0**-24 + 1e-10
    assert np.abs(got[rows, 64:] - np.sin(ang)).max() <= 2.0**-24 + 1e-10
    assert kvq8.rope_table(torch.from_numpy(inv).cuda(), 1).tolist()[0] == [1.0] * 64 + [0.0] * 64
