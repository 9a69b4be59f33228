"""Tensor-memory accesses of the cache attention's kernels follow a fence (CPU).

A thread that learns from an mbarrier (waited for or tested) that the tensor
core is done may touch tensor memory only after tcgen05.fence::after_thread_sync:
the barrier alone does not order its tcgen05 instructions behind the product's.
Whether a GPU shows a missing fence depends on timing, so the order is read
off the source: between an access and the wait before it in the same role
there has to be the fence.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "target_model_verify_gb300", "csrc")
ROLE = re.compile(r"// -{10,}")                                   # a role's heading: its own order
WAIT = re.compile(r"\b(warp_wait|mbar_test|mbar_wait<true>|wait_drain)\(")
FENCE = re.compile(r"\btc_fence_after\(\)")
ACCESS = re.compile(r"\b(tmem_load|tmem_store|mma_ss<[^>]*>|mma_ts<[^>]*>)\(")


def _unfenced(text):
    """(accesses, line numbers of those with a wait after the last fence) of a kernel's text."""
    seen, bad, waited = 0, [], False
    for no, line in enumerate(text.splitlines(), 1):
        code = line.split("//")[0]
        if ROLE.search(line):
            waited = False
        marks = sorted([(m.start(), "wait") for m in WAIT.finditer(code)] +
                       [(m.start(), "fence") for m in FENCE.finditer(code)] +
                       [(m.start(), "access") for m in ACCESS.finditer(code)])
        for _, what in marks:
            if what == "access":
                seen += 1
                if waited:
                    bad.append(no)
            else:
                waited = what == "wait"
    return seen, bad


@pytest.mark.parametrize("name,kernel", [("cache_attention.cuh", "cache_attn_kernel("),
                                         ("cache_attention_keys.cuh", "cache_attn_keys_kernel(")])
def test_tensor_memory_is_touched_behind_a_fence(name, kernel):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = f.read()
    seen, bad = _unfenced(text[text.index(kernel):])
    assert seen >= 6
    assert not bad, bad


def test_the_reading_itself():
    fine = "warp_wait(a);\ntc_fence_after();\ntmem_load(x);\ntmem_store(x);\n"
    assert _unfenced(fine) == (2, [])
    assert _unfenced(fine + "if (mbar_test(b))\n  tmem_store(x);\n") == (3, [6])
    assert _unfenced("warp_wait(a);\n// ----------- other role --\ntmem_store(x);\n") == (1, [])
