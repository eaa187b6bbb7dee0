"""The order of programmatic launches, read from the kernels' sources: a kernel
that lets the next one of its stream start before it has waited for the one
ahead of it would let a decode step with the cache declared ready
(KVQ8_STEP_CACHE_READY) read the cache before it is written.  Such a race
rarely shows in a run, so the rule is checked here, without a GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_quantized_kv_gb300", "csrc")
# decode_combine_kernel releases first where it follows its own split (kEarly): everything ahead of that split is
# done by then.  The 4-bit split releases its merge by its end, so it is done when that starts.
EARLY = {"decode_combine_kernel", "decode_combine_fixed_kernel"}


def _kernels():
    """name -> body (comments stripped) of every kernel."""
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__ void\s*(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\))?\s*(\w+)\([^)]*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            found[m.group(1)] = text[m.end():i]
    return found


KERNELS = _kernels()
RELEASING = sorted(n for n, b in KERNELS.items() if "pdl_launch_dependents()" in b)


def test_kernels_are_found():
    assert {"decode_split_kernel", "weights_merge_kernel", "evict_select_kernel", "evict_copy_kernel",
            "norm_rope_append_kernel", "quantize_append_kernel"} | EARLY <= set(RELEASING)


@pytest.mark.parametrize("name", [n for n in RELEASING if n not in EARLY])
def test_waits_before_it_releases(name):
    body = KERNELS[name]
    assert 0 <= body.find("pdl_wait()") < body.find("pdl_launch_dependents()")


def test_split_of_a_ready_step_waits_in_every_thread():
    # its producer starts without a wait; it waits before the stages that the step ahead may write and, in any case,
    # before the CTA's release, which counts with the first thread that gets there
    body = KERNELS["decode_split_kernel"]
    producer = body[body.index("if (warp == kConsumerWarps)"):body.index("for (int k = max(0, kbase - Lay::kStages)")]
    assert producer.count("pdl_wait()") == 2
    assert re.search(r"pdl_wait\(\);\s*if \(lane == 0\) \{\s*$", producer)
    consumers = body[body.index("for (int k = max(0, kbase - Lay::kStages)"):]
    assert consumers.index("pdl_wait()") < consumers.index("while (remaining > 0")


def test_a_merge_called_on_its_own_releases_late():
    # anything may lie between kvq8_decode_split and kvq8_decode_combine
    text = open(os.path.join(CSRC, "abi.cu")).read()
    combine = text[text.index("kvq8_status kvq8_decode_combine("):text.index("kvq8_status kvq8_decode_attn(")]
    assert "p.release_early = 0;" in combine
