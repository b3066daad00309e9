"""Kernels launched with programmatic dependence may start while the work before
them on the stream is still running: each has to wait for it before it touches
global memory.  Checked in the source text."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "looped_transformer_self_b200",
                    "csrc")


def _sources():
    text = "\n".join(open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))))
    return re.sub(r"//[^\n]*", "", text)


def _body(text, name):
    """The kernel's text between its braces."""
    at = re.search(r"__global__[^;{]*?\b%s\(" % name, text)
    assert at, f"{name}: no definition found"
    i = text.index("{", at.end())
    depth, j = 1, i + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
    return text[i:j]


def _launched(text):
    names = set(re.findall(r"launch_pdl\((k_\w+)", text))
    return sorted(names | {"k_verify"})  # a launch of its own, with a cluster


def test_the_launches_are_found():
    names = _launched(_sources())
    assert {"k_attn_tc", "k_attn_prompt_simt", "k_attn_prompt_join", "k_attn_prefix_simt", "k_attn_prefix_mma",
            "k_attn_prefix_merge", "k_verify"} <= set(names)


# What reads or writes global memory in these kernels: loads and stores through the argument
# struct's pointers, the offsets' readers, TMA, and the error word.
TOUCHES = [r"__ldg\(", r"off_range\(", r"prompt_tile\(", r"\.start\(", r"tma_load", r"cp_async16\(", r"simt_fetch",
           r"\ba\.(q|k|v|o|p|u_acc|u_draw|tok|n_acc|part|part_ml|row_tab|tile_tab|cache|tail|prefix|draft|off)\b\s*[\[+)]",
           r"\)a\.(q|k|v|o|cache)\b"]


@pytest.mark.parametrize("name", _launched(_sources()))
def test_kernel_waits_before_it_touches_global_memory(name):
    body = _body(_sources(), name)
    at = body.find("pdl_wait();")
    assert at >= 0, f"{name} is launched beside its predecessor and never waits for it"
    for pattern in TOUCHES:
        hit = re.search(pattern, body[:at])
        assert hit is None, f"{name}: {hit.group(0)!r} before the wait"


SERVING = ["attn_common.cuh", "attn_prefix.cuh", "attn_prefix_mma.cuh", "attn_tc.cuh", "attn_tc_kernel.cuh",
           "prompt_tile.cuh", "capi_attn_prefix.cu", "capi_attn_prompt.cu", "capi_verify.cu"]


@pytest.mark.parametrize("name", SERVING)
def test_inputs_are_not_read_as_constant_memory(name):
    """__ldg (ld.global.nc) asks for memory that nothing writes while the kernel lives.  These kernels start
    while the work that writes their inputs still runs, and such a load may also move in front of the wait."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for word in ("__ldg(", "ld.global.nc", "__restrict__"):
        assert word not in text, word


@pytest.mark.parametrize("name", _launched(_sources()))
def test_tensor_memory_is_held_before_the_next_kernel_may_start(name):
    """A next kernel that took tensor memory first and then waited for this one, which waits for the memory,
    would never end."""
    body = _body(_sources(), name)
    at = body.find("pdl_trigger();")
    assert at < 0 or "tcgen05.alloc" not in body[at:]


@pytest.mark.parametrize("name", _launched(_sources()))
def test_no_early_return_without_the_wait(name):
    """A CTA that reports an error or leaves before the wait would let what follows start too early."""
    body = _body(_sources(), name)
    assert "set_err(" not in body[:body.find("pdl_wait();")]
