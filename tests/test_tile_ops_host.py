"""Host-side checks of the prompt attention, the decode over shared prefixes and the
cache read back: every refusal returns before a launch, so this runs without a GPU."""
import os
import re

import pytest

from int8_quantized_kv_gb300 import build as kbuild
from int8_quantized_kv_gb300 import kvq8

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_quantized_kv_gb300", "csrc")
FAKE = 1 << 20   # a 256-aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq8.load()


def _prompt(lib, **kw):
    a = dict(q=FAKE, q_dtype=kvq8.DTYPE_F32, qs=1024, batch=1, n_new=3, nqh=8, nkv=2, hd=128, kp=FAKE, vp=FAKE, ks=FAKE,
             vs=FAKE, num_blocks=4, table=FAKE, max_blocks=4, bs=256, start=FAKE, n_tokens=None, sm=0.088, out=FAKE,
             out_dtype=kvq8.DTYPE_F32, os=1024, ws=FAKE, ws_bytes=0, status=None, stream=None)
    a.update(kw)
    return lib.kvq8_prompt_attn(*a.values())


def test_prompt_refusals(lib):
    need = kvq8.prompt_workspace_bytes(1, 3, 8, 2, 4)
    assert need > 0 and need % 256 == 0
    assert kvq8.prompt_workspace_bytes(1, 3, 6, 2, 4) == 0                # G = 3
    assert kvq8.prompt_workspace_bytes(1, -1, 8, 2, 4) == 0
    assert kvq8.prompt_workspace_bytes(60000, 60000, 8, 2, 4) == 0
    assert lib.kvq8_prompt_workspace_bytes(1, 3, 8, 2, 64, 4, 256) == 0
    for bad in (dict(hd=64), dict(bs=128), dict(nqh=6), dict(batch=65536), dict(max_blocks=(2**31 - 1) // 256 + 1),
                dict(q_dtype=3), dict(out_dtype=-1), dict(batch=60000, n_new=60000)):
        assert _prompt(lib, **bad) == kvq8.ERR_UNSUPPORTED, bad
    for bad in (dict(batch=-1), dict(n_new=-1), dict(num_blocks=0), dict(max_blocks=0), dict(sm=float("nan")),
                dict(sm=float("inf")), dict(qs=1020), dict(qs=1026), dict(os=896), dict(os=1025), dict(qs=-1024),
                dict(q_dtype=kvq8.DTYPE_BF16, qs=1028), dict(out_dtype=kvq8.DTYPE_F16, os=1028)):
        assert _prompt(lib, ws_bytes=need, **bad) == kvq8.ERR_INVALID_ARG, bad
    for name in ("q", "kp", "vp", "ks", "vs", "table", "start", "out"):
        assert _prompt(lib, ws_bytes=need, **{name: None}) == kvq8.ERR_INVALID_ARG, name
        assert _prompt(lib, ws_bytes=need, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    assert _prompt(lib, ws_bytes=need, n_tokens=FAKE + 2) == kvq8.ERR_INVALID_ARG
    assert _prompt(lib, ws_bytes=need - 1) == kvq8.ERR_WORKSPACE
    assert _prompt(lib, ws_bytes=need, ws=FAKE + 16) == kvq8.ERR_WORKSPACE
    assert _prompt(lib, ws_bytes=need, ws=None) == kvq8.ERR_WORKSPACE
    assert _prompt(lib, batch=0) == kvq8.OK
    assert _prompt(lib, n_new=0) == kvq8.OK


def _shared(lib, step, **kw):
    a = dict(q=FAKE, kn=FAKE, vn=FAKE, batch=4, nqh=8, nkv=2, hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE,
             num_blocks=4, table=FAKE, max_blocks=4, bs=256, lens=FAKE, groups=2, starts=FAKE, shared=FAKE, sm=0.088,
             out=FAKE, ws=FAKE, ws_bytes=0, status=None, stream=None)
    a.update(kw)
    if not step:
        a.pop("kn"), a.pop("vn")
    return getattr(lib, "kvq8_decode_step_shared" if step else "kvq8_decode_attn_shared")(*a.values())


@pytest.mark.parametrize("step", [False, True])
def test_shared_refusals(lib, step):
    need = kvq8.shared_workspace_bytes(4, 2, 8, 2, 4)
    assert need > kvq8.decode_workspace_bytes(4, 8, 2, 4) and need % 256 == 0
    assert kvq8.shared_workspace_bytes(4, 65536, 8, 2, 4) == 0
    assert kvq8.shared_workspace_bytes(4, -1, 8, 2, 4) == 0
    assert kvq8.shared_workspace_bytes(4, 2, 6, 2, 4) == 0
    for bad in (dict(hd=64), dict(bs=128), dict(nqh=24, nkv=8), dict(batch=65536), dict(groups=65536)):
        assert _shared(lib, step, **bad) == kvq8.ERR_UNSUPPORTED, bad
    for bad in (dict(batch=-1), dict(groups=-1), dict(groups=0), dict(batch=0, groups=-1),
                dict(sm=float("inf"))):
        assert _shared(lib, step, ws_bytes=need, **bad) == kvq8.ERR_INVALID_ARG, bad
    for name in ("q", "kp", "vp", "ks", "vs", "table", "lens", "starts", "shared", "out") + (("kn", "vn") if step else ()):
        assert _shared(lib, step, ws_bytes=need, **{name: None}) == kvq8.ERR_INVALID_ARG, name
        assert _shared(lib, step, ws_bytes=need, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    assert _shared(lib, step, ws_bytes=kvq8.decode_workspace_bytes(4, 8, 2, 4)) == kvq8.ERR_WORKSPACE
    assert _shared(lib, step, ws_bytes=need - 1) == kvq8.ERR_WORKSPACE
    assert _shared(lib, step, ws_bytes=need, ws=FAKE + 128) == kvq8.ERR_WORKSPACE
    assert _shared(lib, step, batch=0, groups=0) == kvq8.OK


def _read(lib, **kw):
    a = dict(batch=1, n_new=3, nkv=2, hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, num_blocks=4, table=FAKE, max_blocks=4,
             bs=256, start=FAKE, n_tokens=None, k=FAKE, v=FAKE, dtype=kvq8.DTYPE_F32, k_s=256, v_s=256, status=None,
             stream=None)
    a.update(kw)
    return lib.kvq8_read(*a.values())


def test_read_refusals(lib):
    for bad in (dict(hd=64), dict(bs=128), dict(batch=65536), dict(nkv=65536), dict(dtype=7),
                dict(max_blocks=(2**31 - 1) // 256 + 1)):
        assert _read(lib, **bad) == kvq8.ERR_UNSUPPORTED, bad
    for bad in (dict(batch=-1), dict(n_new=-1), dict(nkv=0), dict(num_blocks=0), dict(max_blocks=0), dict(k=None, v=None),
                dict(k_s=128), dict(v_s=258), dict(dtype=kvq8.DTYPE_BF16, v_s=260), dict(k_s=-256)):
        assert _read(lib, **bad) == kvq8.ERR_INVALID_ARG, bad
    for name in ("kp", "vp", "ks", "vs", "table", "start"):
        assert _read(lib, **{name: None}) == kvq8.ERR_INVALID_ARG, name
    for name in ("kp", "vp", "ks", "vs", "table", "start", "n_tokens", "k", "v"):
        assert _read(lib, **{name: FAKE + 2}) == kvq8.ERR_INVALID_ARG, name
    assert _read(lib, batch=0) == kvq8.OK
    assert _read(lib, n_new=0) == kvq8.OK


def test_the_tail_split_acquires_what_it_does_not_wait_for():
    # it starts without the wait that would order the plan's rows, lengths, tables and queries ahead of its loads, so it
    # acquires them itself, in every thread and ahead of the first load
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "decode_tail.cuh")).read())
    body = text[text.index("decode_tail_kernel(DecodeParams p) {"):text.index("launch_tail_g")]
    acquire = body.index("\n    acquire_gpu(p.windows);\n")
    loads = re.search(r"p\.(ctx_lens|windows|block_table|q|k_new|v_new|batch)\b(?!\);)", body)
    assert acquire < loads.start() < body.index("pdl_wait()")
    ptx = open(os.path.join(CSRC, "kvq8_ptx.cuh")).read()
    assert re.search(r"ld\.relaxed\.gpu\.global\.s32 [^;]*;\\n\\tfence\.acq_rel\.gpu;", ptx)


def test_read_takes_no_more_rows_than_one_launch_has_warps_for(lib):
    # 65535 * 65535 * 2^27 tasks at most; a count that passed 31 bits would make a small grid of it.  (Without a GPU what
    # passes the checks fails at its launch.)
    top = 2**31 - 1
    for bad in (dict(n_new=top, batch=256, nkv=1, k_s=128, v_s=128), dict(n_new=top, batch=65535, nkv=8, k_s=1024, v_s=1024),
                dict(n_new=2**30, batch=2048, nkv=2), dict(n_new=top, batch=65535, nkv=65535, k_s=2**23, v_s=2**23),
                dict(n_new=top - 29, batch=128, nkv=1, k_s=128, v_s=128)):
        assert _read(lib, **bad) == kvq8.ERR_UNSUPPORTED, bad


def test_kernels_that_trade_registers_have_the_count_that_they_trade(lib):
    # setmaxnreg draws on what the launch holds: a compiler that gives such a kernel another count fails the build, not
    # every large prompt at its launch
    said = open(os.path.join(kbuild.BUILD_DIR, "tiles.ptxas")).read()
    counts = re.findall(r"Compiling entry function '(\S*tile_kernelILb[01]ELi128E\S*)'.*?Used (\d+) registers", said, re.S)
    assert len(counts) == 3
    want = re.search(r"kLaunchRegs = (\d+)", open(os.path.join(CSRC, "tiles.cu")).read()).group(1)
    assert {n for _, n in counts} == {want} and [w for _, w in kbuild.TRADING] == [int(want)]
    kbuild.check_registers("tiles.cu", said)
    for other in (int(want) - 8, int(want) + 8):
        with pytest.raises(RuntimeError, match="registers per thread"):
            kbuild.check_registers("tiles.cu", said.replace(f"Used {want} registers", f"Used {other} registers"))
    kbuild.check_registers("other.cu", "ptxas info : Compiling entry function '_Z5plainv' for 'sm_103a'\nUsed 40 registers")
