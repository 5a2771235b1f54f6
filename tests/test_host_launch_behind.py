"""Every kernel that is launched behind another one while that one still runs, whichever helper launches it and wherever it
is: it waits for its predecessor before it reads what that one writes, and promises nothing about it.  The two that
read something earlier, and the one that lets its successor start early, are held to the reasons why they may."""
import glob
import os
import re

import pytest

import shared_prompt_exact_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")
WAIT, EARLY = "cudaGridDependencySynchronize();", "cudaTriggerProgrammaticLaunchCompletion();"
KERNELS = {"append_kernel", "read_kernel", "decode_kernel", "prompt_kernel", "join_kernel", "rope_weight_kernel",
           "policy_finish_kernel"}


def _text(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def _sources():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
    return {os.path.basename(f): _text(os.path.basename(f)) for f in files if os.path.basename(f) != "launch.cuh"}


def _kernels():
    """{name: (parameters, body)}"""
    found = {}
    for name, text in _sources().items():
        for kernel in re.findall(r"launch_behind(?:_shared)?\(\s*(\w+)", text):
            m = re.search(r"__global__[^;{]*?\b" + kernel + r"\s*\(([^{]*)\)\s*\{(.*?)\n\}", text, re.S)
            assert m, (name, kernel)
            found[kernel] = m.group(1), m.group(2)
    return found


def test_all_of_them_are_known():
    assert set(_kernels()) == KERNELS
    # nobody asks for such a launch past the helpers
    assert not [n for n, t in _sources().items() if "ProgrammaticStreamSerialization" in t]


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_it_waits_and_promises_nothing(name):
    parameters, body = _kernels()[name]
    assert WAIT in body
    assert not re.search(r"const[^,]*\*\s*__restrict__", parameters)
    assert "__ldg" not in body and ".nc" not in body


def test_only_the_prompts_kernel_lets_its_successor_start_early():
    assert [n for n, t in _sources().items() if "cudaTriggerProgrammaticLaunchCompletion" in t] == ["prompt.cu"]
    body = _kernels()["prompt_kernel"][1]
    # once, behind its own wait and a barrier of the block: what the prompts' kernel waited for is complete then
    assert body.count(EARLY) == 1 and body.count(WAIT) == 1
    assert body.index(WAIT) < body.index("__syncthreads();", body.index(WAIT)) < body.index(EARLY)
    # its successor is the walk, and the walk's is the join
    order = re.search(r"cudaError_t launch_decode\(.*?\n\}", _text("decode.cu"), re.S).group(0)
    assert order.index("launch_prompt(") < order.index("walk<false>(") < order.index("join<64>(")


def test_the_walk_waits_at_its_start_or_its_end():
    body = _kernels()["decode_kernel"][1].rstrip()
    # at its start, but behind the prompts' kernel, which has waited for the same before this one could start; and at
    # its end, so that who waits for the walk finds both kernels' results
    assert body.count(WAIT) == 2 and body.endswith("if (warp == 0) " + WAIT)
    start = body.index("if (!A.big) " + WAIT)
    assert start < body.index("deal_sources<") and "A.lens" not in body[:start] and "A.q " not in body[:start]
    # the partial results, which the prompts' kernel writes too, are written here and never read
    assert not re.search(r"=\s*ws\.partial\[", body) and "ws.o[" not in body


def test_the_join_reads_lengths_alone_before_its_wait():
    body = _kernels()["join_kernel"][1]
    before = body[:body.index(WAIT)]
    assert body.count(WAIT) == 1 and "ws.partial" not in before and "ws.o" not in before
    assert re.findall(r"\b(response_len|prompt_len)\(", before) == ["response_len", "prompt_len"]
    assert not re.search(r"A\.(q|kv|table|prompt_table|out|lse)\b", before)
