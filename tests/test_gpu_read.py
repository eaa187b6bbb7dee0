"""The cache read back: every value is code * scale, exactly in fp32, rounded once
otherwise; positions, padding, strides, broken tables."""
import pytest
import torch

import tile_ref as ref
from int8_quantized_kv_gb300 import kvq8

pytestmark = pytest.mark.gpu
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _want(cache, table, b, h, t):
    """code * scale in fp32 (the same product in 64 bits, rounded: codes have 8 bits, so it fits 32 + 8 bits exactly)."""
    k, v = ref.rows64(cache, table[b], h, t)
    return k.float(), v.float()


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("nkv", [1, 3, 8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 64, 300])
def test_values(gpu_lib, kind, nkv, n):
    starts = [0, 1, 15, 16, 63, 200, 255, 256, 500]
    table, nb = ref.random_table(len(starts), (500 + n + 255) // 256, n)
    cache = ref.random_cache(nb, nkv, n, spread=8.0)
    ns = [n, n, max(n - 1, 0), n, 0, n + 50, 1, n, -2]
    k = torch.full((len(starts), n, nkv, 128), 7.0, dtype=KINDS[kind], device="cuda")
    v = torch.full_like(k, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kvq8.read_cache(cache, table, i32(starts), k, v, n_tokens=i32(ns), dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for b, (p, m) in enumerate(zip(starts, ns)):
        m = max(0, min(n, m))
        assert bool((k[b, m:] == 7).all()) and bool((v[b, m:] == 9).all())
        for h in range(nkv):
            wk, wv = _want(cache, table, b, h, torch.arange(p, p + m, device="cuda"))
            assert torch.equal(k[b, :m, h], wk.to(k.dtype)) and torch.equal(v[b, :m, h], wv.to(k.dtype))


def test_one_side_and_strides(gpu_lib):
    table, nb = ref.random_table(2, 3, 5)
    cache = ref.random_cache(nb, 2, 5)
    start = torch.tensor([100, 33], dtype=torch.int32, device="cuda")
    k, v = torch.empty((2, 400, 2, 128), device="cuda"), torch.empty((2, 400, 2, 128), device="cuda")
    kvq8.read_cache(cache, table, start, k, v)
    packed = torch.full((2, 400, 520), 5.0, device="cuda")
    kvq8.read_cache(cache, table, start, None, packed[..., 4:260].unflatten(-1, (2, 128)))
    kvq8.read_cache(cache, table, start, packed[..., 260:516].unflatten(-1, (2, 128)), None)
    torch.cuda.synchronize()
    assert torch.equal(packed[..., 4:260], v.flatten(2)) and torch.equal(packed[..., 260:516], k.flatten(2))
    assert bool((packed[..., :4] == 5).all()) and bool((packed[..., 516:] == 5).all())
    for bad in (dict(k_out=None, v_out=None), dict(v_out=v.half()), dict(k_out=k.double(), v_out=v.double()),
                dict(k_out=k.cpu()), dict(k_out=k[:, :5]), dict(start_pos=start.long())):
        with pytest.raises(ValueError):
            kvq8.read_cache(**{**dict(cache=cache, block_table=table, start_pos=start, k_out=k, v_out=v), **bad})


def test_what_is_outside_is_left_and_flagged(gpu_lib):
    table, nb = ref.random_table(4, 2, 6)
    cache = ref.random_cache(nb, 2, 6)
    table[1, 0], table[2, 1] = -1, nb
    starts = [-20, 250, 200, 500]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.full((4, 100, 2, 128), 7.0, device="cuda")
    v = torch.full_like(k, 7.0)
    kvq8.read_cache(cache, table, torch.tensor(starts, dtype=torch.int32, device="cuda"), k, v, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvq8.DEV_BAD_POSITION | kvq8.DEV_BAD_BLOCK_ID
    there = [range(20, 100), range(6, 100), range(0, 56), range(0, 12)]
    for b, p in enumerate(starts):
        gone = torch.ones(100, dtype=torch.bool)
        gone[list(there[b])] = False
        assert bool((k[b, gone.cuda()] == 7).all()) and bool((v[b, gone.cuda()] == 7).all())
        for h in range(2):
            t = torch.tensor([p + i for i in there[b]], device="cuda")
            wk, wv = _want(cache, table, b, h, t)
            assert torch.equal(k[b, list(there[b]), h], wk) and torch.equal(v[b, list(there[b]), h], wv)
    far = torch.tensor([2**31 - 50] * 4, dtype=torch.int32, device="cuda")
    status.zero_()
    kvq8.read_cache(cache, table, far, k, v, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvq8.DEV_BAD_POSITION


def test_append_and_read_back(gpu_lib):
    # the nearest multiple of a row's scale: half a step off at most, plus the roundings of v / scale and code * scale
    x = torch.randn((3, 77, 2, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    cache = kvq8.alloc_cache(6, 2)
    table = torch.tensor([[3, 0], [1, 5], [2, 4]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 200, 100], dtype=torch.int32, device="cuda")
    kvq8.quantize_append(x, -2 * x, start, table, cache)
    k, v = torch.empty_like(x), torch.empty_like(x)
    kvq8.read_cache(cache, table, start, k, v)
    torch.cuda.synchronize()
    step = x.abs().amax(-1, keepdim=True) / 127
    assert bool(((k - x).abs() <= step * (0.5 + 127 * 2.0 ** -22)).all())
    assert torch.equal(v, -2 * k)


def test_blocks_past_32_bits(gpu_lib):
    table, nb = ref.random_table(1, 3, 9)
    cache = ref.random_cache(nb, 8, 9)
    start = torch.tensor([70], dtype=torch.int32, device="cuda")
    spare = 2**32 // (8 * 256 * 128)
    big = kvq8.KVCache(*(torch.empty((spare + nb,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in cache))
    for x, y in zip(big, cache):
        x[spare:] = y
    got = [torch.empty((1, 600, 8, 128), device="cuda") for _ in range(4)]
    kvq8.read_cache(cache, table, start, got[0], got[1])
    kvq8.read_cache(big, table + spare, start, got[2], got[3])
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


def test_captured_and_replayed_with_other_positions(gpu_lib):
    table, nb = ref.random_table(2, 3, 11)
    cache = ref.random_cache(nb, 2, 11)
    start = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    ns = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
    k, v = torch.empty((2, 300, 2, 128), device="cuda"), torch.empty((2, 300, 2, 128), device="cuda")
    kvq8.read_cache(cache, table, start, k, v, n_tokens=ns)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq8.read_cache(cache, table, start, k, v, n_tokens=ns)
    for starts, counts in (([5, 468], [300, 300]), ([255, 16], [1, 0])):
        start.copy_(torch.tensor(starts))
        ns.copy_(torch.tensor(counts))
        k.fill_(7.0)
        v.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for b, (p, m) in enumerate(zip(starts, counts)):
            assert bool((k[b, m:] == 7).all()) and bool((v[b, m:] == 9).all())
            for h in range(2):
                wk, wv = _want(cache, table, b, h, torch.arange(p, p + m, device="cuda"))
                assert torch.equal(k[b, :m, h], wk) and torch.equal(v[b, :m, h], wv)
