"""Prompt attention, the steps over a shared prefix and the cache read back in a run, as a
server has them: a prompt in two parts, several samples continued from it, drafted tokens
verified, the rows read back; against the 64-bit form over the same cache, eagerly and captured."""
import pytest
import torch

import tile_ref as ref
from int8_quantized_kv_gb300 import kvq8

pytestmark = pytest.mark.gpu

NQH, NKV, SAMPLES, STEPS, DRAFT = 8, 2, 3, 4, 3
PROMPT = (300, 77)                       # parts of the prompt
MB = 3


def test_prompt_samples_and_drafts(gpu_lib):
    g = torch.Generator("cuda").manual_seed(11)
    n = sum(PROMPT)
    total = n + STEPS + DRAFT
    x = torch.randn((SAMPLES, total, NQH + 2 * NKV, 128), generator=g, device="cuda").bfloat16()
    x[:, :n] = x[0, :n]                  # the prompt is the samples' own
    one = torch.ones(128, device="cuda")
    rope = kvq8.rope_table(1e6 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64), 1024)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = kvq8.alloc_cache(1 + SAMPLES * (MB - 1) + 1, NKV, "cuda")
    for t in cache:
        t.zero_()
    # sample 0 has the prompt's blocks; the others list its whole block and have their own from there on
    table = torch.tensor([[0] + [1 + b * (MB - 1) + j for j in range(MB - 1)] for b in range(SAMPLES)],
                         dtype=torch.int32, device="cuda")
    status = i32(0)
    q = torch.empty((1, n, NQH, 128), device="cuda")
    out = torch.empty((1, n, NQH, 128), device="cuda")
    wp = kvq8.alloc_prompt_workspace(SAMPLES, n, NQH, NKV, MB)
    wd = kvq8.alloc_shared_workspace(SAMPLES, 1, NQH, NKV, MB)
    starts, prefix = i32(0, SAMPLES), i32(n)
    begins = [i32(0), i32(PROMPT[0])]
    lens = [i32(*[n + i + 1] * SAMPLES) for i in range(STEPS)]
    steps_q, steps_out = (torch.empty((STEPS, SAMPLES, NQH, 128), device="cuda") for _ in range(2))
    q_draft, out_draft = (torch.empty((SAMPLES, DRAFT, NQH, 128), device="cuda") for _ in range(2))
    draft_at = i32(*[n + STEPS] * SAMPLES)
    k_all, v_all = (torch.empty((SAMPLES, total, NKV, 128), device="cuda") for _ in range(2))
    at0 = i32(*[0] * SAMPLES)

    def heads(t):
        return [h.contiguous() for h in (t[..., :NQH, :], t[..., NQH:NQH + NKV, :], t[..., NQH + NKV:, :])]

    def run():
        for begin, i, m in zip(begins, (0, PROMPT[0]), PROMPT):
            kvq8.norm_rope_append(*heads(x[:1, i:i + m]), one, one, 1e-6, rope, begin, table[:1], cache, q[:, i:i + m],
                                  dev_status=status)
            kvq8.prompt_attn(q[:, i:i + m], cache, table[:1], begin, out[:, i:i + m], wp, dev_status=status)
        for b in range(1, SAMPLES):      # the block that the prompt ends in, for each sample
            for t in cache:
                t[1 + b * (MB - 1)] = t[1]
        for i in range(STEPS):
            args = (cache, table, lens[i], starts, prefix, steps_out[i], wd)
            _, k, v = heads(x[:, n + i])
            if i % 2:                    # the step appends the rows as they are
                steps_q[i].copy_(x[:, n + i, :NQH])
                kvq8.decode_step_shared(steps_q[i], k.float(), v.float(), *args, dev_status=status)
            else:
                kvq8.norm_rope_append(*heads(x[:, n + i:n + i + 1]), one, one, 1e-6, rope, lens[i] - 1, table, cache,
                                      steps_q[i][:, None], dev_status=status)
                kvq8.decode_attn_shared(steps_q[i], *args, dev_status=status)
        kvq8.norm_rope_append(*heads(x[:, n + STEPS:]), one, one, 1e-6, rope, draft_at, table, cache, q_draft,
                              dev_status=status)
        kvq8.prompt_attn(q_draft, cache, table, draft_at, out_draft, wp, dev_status=status)
        kvq8.read_cache(cache, table, at0, k_all, v_all, dev_status=status)

    def check():
        assert status.item() == 0
        G = NQH // NKV
        for b in range(SAMPLES):
            for h in range(NKV):
                k, v = ref.rows64(cache, table[b], h, torch.arange(total, device="cuda"))
                assert torch.equal(k_all[b, :, h], k.float()) and torch.equal(v_all[b, :, h], v.float())

                def same(rows, got, first, what):
                    """rows, got [m][NQH][128]: query tokens from position first on."""
                    lims = (first + 1 + torch.arange(len(rows), device="cuda")).repeat_interleave(G)
                    pick = lambda t: t[:, h * G:(h + 1) * G].reshape(-1, 128)  # noqa: E731
                    want, tol = ref.attend(pick(rows), k, v, lims)
                    ref.check(pick(got), want, tol, f"{what} of sample {b}, head {h}")
                if b == 0:
                    same(q[0], out[0], 0, "prompt")
                for i in range(STEPS):
                    same(steps_q[i, b:b + 1], steps_out[i, b:b + 1], n + i, f"step {i}")
                same(q_draft[b], out_draft[b], n + STEPS, "draft")

    run()
    torch.cuda.synchronize()
    check()
    first = [t.clone() for t in (out, steps_out, out_draft, k_all, v_all, *cache)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in (out, steps_out, out_draft, k_all, v_all, *cache):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check()
    for a, b in zip(first, (out, steps_out, out_draft, k_all, v_all, *cache)):
        assert torch.equal(a, b)
