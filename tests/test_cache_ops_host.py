"""Host-side checks of the operators around the int8 cache (window, weights,
eviction, norm + rotation + append): every refusal returns before a launch, so
this runs without a GPU."""
import pytest
import torch

from int8_quantized_kv_gb300 import build as kbuild
from int8_quantized_kv_gb300 import kvq8

FAKE = 1 << 20   # a 256-aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq8.load()


def _window(lib, step, **kw):
    a = dict(q=FAKE, kn=FAKE, vn=FAKE, batch=1, nqh=8, nkv=8, hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE,
             num_blocks=4, table=FAKE, max_blocks=4, bs=256, lens=FAKE, windows=FAKE, sinks=4, sm=0.088,
             out=FAKE, ws=FAKE, ws_bytes=0, status=None, stream=None)
    a.update(kw)
    if not step:
        a.pop("kn"), a.pop("vn")
    return getattr(lib, "kvq8_decode_step_window" if step else "kvq8_decode_attn_window")(*a.values())


@pytest.mark.parametrize("step", [False, True])
def test_window_refusals(lib, step):
    need = kvq8.decode_workspace_bytes(1, 8, 8, 4)
    assert _window(lib, step, hd=64) == kvq8.ERR_UNSUPPORTED
    assert _window(lib, step, bs=128) == kvq8.ERR_UNSUPPORTED
    assert _window(lib, step, nqh=24) == kvq8.ERR_UNSUPPORTED
    assert _window(lib, step, batch=65536) == kvq8.ERR_UNSUPPORTED
    assert _window(lib, step, max_blocks=(2**31 - 1) // 256 + 1) == kvq8.ERR_UNSUPPORTED
    assert _window(lib, step, batch=-1) == kvq8.ERR_INVALID_ARG
    assert _window(lib, step, sinks=-1) == kvq8.ERR_INVALID_ARG
    assert _window(lib, step, batch=0, sinks=-1) == kvq8.ERR_INVALID_ARG
    for name in ("q", "kp", "vp", "ks", "vs", "table", "lens", "windows", "out"):
        assert _window(lib, step, ws_bytes=need, **{name: None}) == kvq8.ERR_INVALID_ARG, name
        assert _window(lib, step, ws_bytes=need, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    if step:
        assert _window(lib, step, ws_bytes=need, kn=None) == kvq8.ERR_INVALID_ARG
        assert _window(lib, step, ws_bytes=need, vn=FAKE + 4) == kvq8.ERR_INVALID_ARG
    assert _window(lib, step, ws_bytes=need, sm=float("inf")) == kvq8.ERR_INVALID_ARG
    assert _window(lib, step, ws_bytes=need - 1) == kvq8.ERR_WORKSPACE
    assert _window(lib, step, ws=FAKE + 16, ws_bytes=need) == kvq8.ERR_WORKSPACE
    assert _window(lib, step, ws=None, ws_bytes=need) == kvq8.ERR_WORKSPACE
    assert _window(lib, step, batch=0) == kvq8.OK


def _weights(lib, step, **kw):
    a = dict(q=FAKE, kn=FAKE, vn=FAKE, batch=1, nqh=8, nkv=8, hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE,
             num_blocks=4, table=FAKE, max_blocks=4, bs=256, lens=FAKE, sm=0.088, out=FAKE, wsum=FAKE, ws=FAKE,
             ws_bytes=0, status=None, stream=None)
    a.update(kw)
    if not step:
        a.pop("kn"), a.pop("vn")
    return getattr(lib, "kvq8_decode_step_weights" if step else "kvq8_decode_attn_weights")(*a.values())


@pytest.mark.parametrize("step", [False, True])
def test_weights_refusals(lib, step):
    need = kvq8.weights_workspace_bytes(1, 8, 8, 4)
    assert need >= kvq8.decode_workspace_bytes(1, 8, 8, 4) + 8 * 4 * 256 * 4 and need % 256 == 0
    assert kvq8.weights_workspace_bytes(1, 6, 2, 4) == 0                 # G = 3
    assert lib.kvq8_weights_workspace_bytes(1, 8, 8, 64, 4, 256) == 0
    assert lib.kvq8_weights_workspace_bytes(1, 8, 8, 128, 0, 256) == 0
    assert _weights(lib, step, hd=64) == kvq8.ERR_UNSUPPORTED
    assert _weights(lib, step, nqh=12) == kvq8.ERR_UNSUPPORTED
    assert _weights(lib, step, batch=-1) == kvq8.ERR_INVALID_ARG
    for name in ("q", "kp", "vp", "ks", "vs", "table", "lens", "out", "wsum"):
        assert _weights(lib, step, ws_bytes=need, **{name: None}) == kvq8.ERR_INVALID_ARG, name
        assert _weights(lib, step, ws_bytes=need, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    if step:
        assert _weights(lib, step, ws_bytes=need, vn=None) == kvq8.ERR_INVALID_ARG
        assert _weights(lib, step, ws_bytes=need, kn=FAKE + 8) == kvq8.ERR_INVALID_ARG
    assert _weights(lib, step, ws_bytes=need, sm=float("nan")) == kvq8.ERR_INVALID_ARG
    # the plain decode's workspace is too small: the scores need their room
    assert _weights(lib, step, ws_bytes=kvq8.decode_workspace_bytes(1, 8, 8, 4)) == kvq8.ERR_WORKSPACE
    assert _weights(lib, step, ws_bytes=need - 1) == kvq8.ERR_WORKSPACE
    assert _weights(lib, step, batch=0) == kvq8.OK


def _evict(lib, **kw):
    a = dict(batch=1, nkv=2, hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, wsum=FAKE, num_blocks=8, table=FAKE,
             max_blocks=4, bs=256, lens=FAKE, keep=300, first=4, recent=32, dst=FAKE, dst_blocks=2, kept=FAKE,
             new_lens=FAKE, status=None, stream=None)
    a.update(kw)
    return lib.kvq8_evict(*a.values())


def test_evict_refusals(lib):
    assert _evict(lib, hd=96) == kvq8.ERR_UNSUPPORTED
    assert _evict(lib, bs=64) == kvq8.ERR_UNSUPPORTED
    assert _evict(lib, batch=65536) == kvq8.ERR_UNSUPPORTED
    assert _evict(lib, max_blocks=2**22 + 1) == kvq8.ERR_UNSUPPORTED       # more than 2^30 positions
    assert _evict(lib, dst_blocks=2**22 + 1) == kvq8.ERR_UNSUPPORTED
    assert _evict(lib, batch=60000, nkv=60000, keep=2, first=0, recent=0) == kvq8.ERR_UNSUPPORTED   # more kept rows than 2^31
    for bad in (dict(keep=0, first=0, recent=0), dict(keep=-5), dict(first=-1), dict(recent=-1),
                dict(keep=35), dict(keep=300, first=301, recent=0), dict(first=2**31 - 1, recent=2**31 - 1),
                dict(keep=513), dict(dst_blocks=0), dict(nkv=0), dict(num_blocks=0), dict(max_blocks=0),
                dict(batch=-1)):
        assert _evict(lib, **bad) == kvq8.ERR_INVALID_ARG, bad
    for name in ("kp", "vp", "ks", "vs", "wsum", "table", "lens", "dst", "kept", "new_lens"):
        assert _evict(lib, **{name: None}) == kvq8.ERR_INVALID_ARG, name
        assert _evict(lib, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    assert _evict(lib, batch=0) == kvq8.OK


def _norm(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=kvq8.DTYPE_F32, qs=1024, kst=256, vst=256, batch=1, n_new=3, nqh=8,
             nkv=2, hd=128, qw=FAKE, kw=FAKE, eps=1e-6, rope=FAKE, n_pos=100, positions=FAKE, n_tokens=None,
             flags=0, start=FAKE, table=FAKE, max_blocks=4, bs=256, num_blocks=8, kp=FAKE, vp=FAKE, ks=FAKE,
             vs=FAKE, wsum=None, out=FAKE, status=None, stream=None)
    a.update(kw)
    return lib.kvq8_norm_rope_append(*a.values())


def test_norm_rope_refusals(lib):
    assert _norm(lib, hd=64) == kvq8.ERR_UNSUPPORTED
    assert _norm(lib, nqh=6) == kvq8.ERR_UNSUPPORTED
    assert _norm(lib, dtype=3) == kvq8.ERR_UNSUPPORTED
    assert _norm(lib, dtype=-1) == kvq8.ERR_UNSUPPORTED
    assert _norm(lib, batch=65536) == kvq8.ERR_UNSUPPORTED
    assert _norm(lib, batch=60000, n_new=60000) == kvq8.ERR_UNSUPPORTED
    for bad in (dict(flags=2), dict(qw=None), dict(kw=None), dict(eps=0.0), dict(eps=-1e-6), dict(eps=2.0),
                dict(eps=float("nan")), dict(n_pos=0), dict(n_new=-1), dict(batch=-1), dict(num_blocks=0),
                dict(qs=1020), dict(qs=1022), dict(kst=128), dict(vst=258), dict(qs=-1024),
                dict(dtype=kvq8.DTYPE_BF16, qs=1028)):
        assert _norm(lib, **bad) == kvq8.ERR_INVALID_ARG, bad
    for name in ("q", "k", "v", "rope", "start", "table", "kp", "vp", "ks", "vs", "out"):
        assert _norm(lib, **{name: None}) == kvq8.ERR_INVALID_ARG, name
        assert _norm(lib, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    for name in ("qw", "kw", "positions", "n_tokens", "wsum"):
        assert _norm(lib, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    assert _norm(lib, batch=0) == kvq8.OK
    assert _norm(lib, n_new=0) == kvq8.OK
    assert _norm(lib, qw=None, kw=None, eps=0.0, n_new=0) == kvq8.OK     # eps is not used without weights
    assert lib.kvq8_rope_table(FAKE, 10, 64, FAKE, None) == kvq8.ERR_UNSUPPORTED
    assert lib.kvq8_rope_table(FAKE, -1, 128, FAKE, None) == kvq8.ERR_INVALID_ARG
    assert lib.kvq8_rope_table(None, 10, 128, FAKE, None) == kvq8.ERR_INVALID_ARG
    assert lib.kvq8_rope_table(FAKE, 10, 128, FAKE + 4, None) == kvq8.ERR_INVALID_ARG
    assert lib.kvq8_rope_table(FAKE, 0, 128, FAKE, None) == kvq8.OK


def test_binding_refuses_host_tensors_and_strides():
    class Dev:   # a device tensor's face, for the checks alone
        def __init__(self, t, device=0):
            self.t, self.dtype, self.shape, self.device = t, t.dtype, t.shape, device

        def get_device(self):
            return self.device

        def __getattr__(self, name):
            return getattr(self.t, name)

    kvq8._torch()
    t, f32 = torch.zeros(2, 128), torch.float32
    cur, torch.cuda.current_device = torch.cuda.current_device, lambda: 0
    try:
        kvq8._need(("t", Dev(t), f32, (2, 128)), ("u", Dev(t[0]), f32, (128,)))
        for bad in (t, Dev(t, 1), Dev(t.half()), Dev(t.T), Dev(torch.zeros(2, 129)), Dev(torch.zeros(2, 256)[:, ::2])):
            with pytest.raises(ValueError, match="t: expected contiguous"):
                kvq8._need(("u", Dev(t[0]), f32, (128,)), ("t", bad, f32, (2, 128)))
    finally:
        torch.cuda.current_device = cur
    packed = torch.zeros(3, 5, 12 * 128)
    rows = packed[..., 256:1280].unflatten(-1, (8, 128))
    assert kvq8._token_stride("q", rows, 3, 5, 8) == 12 * 128
    assert kvq8._token_stride("q", rows[:1], 1, 5, 8) == 12 * 128
    assert kvq8._token_stride("q", rows[:, :1], 3, 1, 8) == 5 * 12 * 128
    assert kvq8._token_stride("q", rows[:1, :1], 1, 1, 8) == 8 * 128
    wide = torch.zeros(3, 5, 8, 256)
    for bad in (rows.transpose(1, 2).contiguous().transpose(1, 2), rows.transpose(0, 1)[:3], wide[..., ::2],
                wide[..., :128], torch.zeros(3, 6, 8, 128)[:, :5]):
        with pytest.raises(ValueError, match="side by side"):
            kvq8._token_stride("q", bad, *bad.shape[:3])
