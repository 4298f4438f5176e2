"""Whole warps act together in the kernels' sources: what no run can show safely.

A wait with a limit that each lane of a warp takes for itself may end differently in
each; unless the warp agrees on the outcome, some lanes leave and the others wait for
them at the next warp-wide instruction without a limit.  The tests read the kernels'
sources, so that the fault needs no GPU.
"""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gptq_qqq_calibration_gb300", "csrc")


def code_of(name):
    """The file without comments and with its strings kept."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body_of(code, kernel):
    """The body of `kernel`, from its first brace to the one that closes it."""
    at = code.index("{", code.index(kernel + "("))
    depth = 0
    for i in range(at, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[at:i + 1]
    raise AssertionError("unbalanced braces")


def statements(body):
    """(statement, the headers of the blocks around it) of a body, in order."""
    found, around, start, parens = [], [], 1, 0
    for i in range(1, len(body) - 1):
        c = body[i]
        parens += {"(": 1, ")": -1}.get(c, 0)
        # (a lambda's body inside an argument list is part of its statement)
        if parens == 0 and c in "{};":
            text = " ".join(body[start:i].split())
            if c == "{":
                around.append(text)
            else:
                if text:
                    found.append((text, tuple(around)))
                if c == "}" and around:
                    around.pop()
            start = i + 1
    return found


ONE_LANE = re.compile(r"lane == 0|elect_one\(\)|threadIdx\.x == 0|leader")


@pytest.mark.parametrize("text,bad", [
    ("{ if (warp == 0 && lane == 0) { if (!wait(x)) { ok = 1; } } }", 0),
    ("{ for (;;) { if (!wait(x)) { ok = 1; break; } } }", 1),
    ("{ bool come = wait(x); read(); come = wait(y) && come; ok = warp_came(come); }", 0),
    ("{ bool come = wait(x); if (!come) break; ok = warp_came(come); }", 1),
    ("{ ok = warp_came(wait(x)); if (elect_one()) { if (!wait(y)) z(); } }", 0)])
def test_reader(text, bad):
    assert len(lone_waits(text, "wait")) == bad


VOTE = re.compile(r"warp_came\(|epi_barrier_any\(|epilogue_t<")  # (epilogue_t votes itself)


def lone_waits(body, wait):
    """Waits that lanes of a warp take one by one, without agreeing on the outcome: neither
    in a branch of one lane, nor in a vote, nor kept in a variable that is next seen in one."""
    lines, headers = [], set()
    for text, around in statements(body):
        for k, h in enumerate(around):  # a block's header is a statement of its own
            if (h, around[:k]) not in headers:
                headers.add((h, around[:k]))
                lines.append((h, around[:k]))
        if text:
            lines.append((text, around))
    bad = []
    for i, (text, around) in enumerate(lines):
        if wait + "(" not in text or VOTE.search(text) or any(ONE_LANE.search(a) for a in around):
            continue
        kept = re.search(r"\b(\w+) = [^=]*" + wait + r"\(", text)
        if kept:
            name = kept.group(1)
            uses = [t for t, _ in lines[i + 1:] if re.search(r"\b%s\b" % name, t) and not re.search(r"\b%s = [^=]*%s\(" % (name, wait), t)]
            if uses and re.search(r"warp_came\(%s\)" % name, uses[0]):
                continue
        bad.append(text)
    return bad


def test_integer_layer_waits_are_agreed_on():
    body = body_of(code_of("int8_linear.cu"), "int8_pair_kernel")
    assert body.count("mbar_wait_soon(") >= 5
    assert lone_waits(body, "mbar_wait_soon") == []


def test_barriers_tested_by_other_lanes_are_ordered():
    """Lanes test barriers for each other: what they saw is passed on by a warp barrier, as votes
    order no memory."""
    body = body_of(code_of("int8_linear.cu"), "int8_pair_kernel")
    order = [text for text, _ in statements(body)]
    shared = [i for i, text in enumerate(order) if "mbar_test(" in text]
    assert len(shared) == 1
    assert "__ballot_sync(" in order[shared[0]] and order[shared[0] + 1] == "__syncwarp()"


WARP_WIDE = re.compile(r"bar\.sync|bar\.red|cluster_sync_all\(\)|tmem_dealloc|tmem_alloc")
TOGETHER = re.compile(r"__syncwarp\(\)|__syncthreads\(\)|cluster_sync_all\(\)")


def loose_barriers(body):
    """Warp-wide barriers and tensor-memory calls with no point in front where the warp's lanes meet."""
    order = [text for text, _ in statements(body)]
    bad = []
    for i, text in enumerate(order):
        if not WARP_WIDE.search(text):
            continue
        before = [t for t in order[:i] if t and not re.match(r"tc_fence_|tmem_|uint32_t any$", t)]
        if not before or not TOGETHER.search(before[-1]):
            bad.append(text)
    return bad


@pytest.mark.parametrize("text,bad", [
    ("{ __syncwarp(); asm(\"bar.sync 1, 128;\"); }", 0),
    ("{ if (leader) { issue(); } asm(\"bar.sync 1, 128;\"); }", 1),
    ("{ __syncthreads(); if (x) { while (late()) nap(); } tc_fence_before(); cluster_sync_all(); }", 1),
    ("{ __syncwarp(); tc_fence_before(); cluster_sync_all(); if (warp == 1) { tc_fence_after(); tmem_dealloc(t); } }", 0)])
def test_barrier_reader(text, bad):
    assert len(loose_barriers(text)) == bad


def test_integer_layer_warps_meet_before_barriers():
    code = code_of("int8_linear.cu")
    for name in ("epi_barrier_any", "int8_pair_kernel"):
        assert loose_barriers(body_of(code, name)) == [], name


def test_feed_forward_warps_meet_before_barriers():
    code = code_of("gated_ff.cu")
    for name in ("epi_barrier", "epi_barrier_any", "void sync", "gated_ff_kernel", "gated_ff_few_kernel"):
        body = body_of(code, name)
        assert WARP_WIDE.search(body), name
        assert loose_barriers(body) == [], name


@pytest.mark.parametrize("name,kernels,wait", [
    ("gated_ff.cu", ["gated_ff_kernel", "gated_ff_few_kernel"], r"mbar_wait"),
    ("syrk_common.cuh", ["epilogue_t"], "wait_full"), ("syrk_bf16.cu", ["syrk_bf16_kernel"], "mbar_wait"),
    ("syrk_bf16_2sm.cu", ["syrk_bf16_2sm_kernel"], "mbar_wait"),
    ("syrk_f32.cu", ["syrk_f32_kernel"], "mbar_wait"), ("gemm_tf32.cu", ["gemm_tf32_kernel"], "mbar_wait"),
    ("local_gram.cu", ["local_gram_kernel"], "mbar_wait")])
def test_other_kernels_waits_are_agreed_on(name, kernels, wait):
    code = code_of(name)
    for kernel in kernels:
        body = body_of(code, kernel).replace("mbar_wait_cluster(", "mbar_wait(")
        assert wait + "(" in body
        assert lone_waits(body, wait) == [], kernel


def test_cluster_barrier_brings_warps_together():
    order = [text for text, _ in statements(body_of(code_of("ptx.cuh"), "void cluster_sync_all"))]
    assert order[0] == "__syncwarp()" and "barrier.cluster.arrive" in order[1]
