"""Source check: a kernel that issues tcgen05 MMAs waits for those in flight before it
frees its tensor memory, also where a bounded wait ran out (a late MMA would write into
columns that another CTA may have by then). No input makes a wait run out, so the order
of the calls stands in for a run."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_ffn_fp32_gb300", "csrc")


def kernels():
    """name: body of every kernel that frees tensor memory."""
    found = {}
    for file in sorted(os.listdir(CSRC)):
        if not file.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
        for part in text.split("__global__")[1:]:
            at = part.index("{")
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(part[end], 0)
                end += 1
                if depth == 0:
                    break
            body = part[at:end]
            if "tmem_dealloc" in body:
                found[f"{file}:{re.search(r'(\w+_kernel)', part).group(1)}"] = body
    return found


def test_the_kernels_are_found():
    names = " ".join(kernels())
    for word in ("adapter_shrink_tc_kernel", "adapter_expand_tc_kernel", "tc_grouped_gemm_kernel", "nt_gemm_kernel"):
        assert word in names


@pytest.mark.parametrize("name", sorted(kernels()))
def test_mmas_are_waited_for_before_their_memory_is_freed(name):
    body = kernels()[name]
    drain = max(body.rfind("bounded_drain("), body.rfind(" drain("))
    assert body.rfind("tc_mma") < drain < body.rfind("tmem_dealloc")


def test_stages_are_not_refilled_after_a_wait_that_ran_out():
    """The adapters' copies into what MMAs read stand behind `alive`."""
    for name, body in kernels().items():
        if not name.startswith("adapter_tc.cu"):
            continue
        calls = [line for line in body.splitlines() if re.search(r"(?<!\.)\b(load|load_b)\(", line)]
        assert len(calls) >= 2
        assert all("alive" in line for line in calls), calls
