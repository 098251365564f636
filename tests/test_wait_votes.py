"""Bounded waits in the windowed attention's sources.  A warp that issues
together (shuffles, ballots, __syncwarp) has to decide together whether a wait
ran out: lanes that went on alone would wait for the others without a bound.
That is read off the sources, since a wait that runs out cannot be arranged in
a healthy kernel: a lane's own decision (guarded_wait) stands inside a vote or
in a block that one lane runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "trainable_block_sparse_compressed_b200", "csrc")


def enclosing_blocks(src, at):
    """Headers (the text before each brace) of the blocks open at offset `at`."""
    stack = []
    for m in re.finditer(r"[{}]", src[:at]):
        if m.group() == "{":
            start = max(src.rfind(c, 0, m.start()) for c in ";{}")
            stack.append(src[start + 1:m.start()])
        elif stack:
            stack.pop()
    return stack


def lone_decisions(src):
    src = re.sub(r"//[^\n]*", "", src)
    bad = []
    for m in re.finditer(r"\bguarded_wait\(", src):
        voted = re.search(r"__all_sync\([^;]*$", src[:m.start()]) is not None
        one_lane = any(re.search(r"if \((lane|threadIdx\.x) == 0\)\s*$", h)
                       for h in enclosing_blocks(src, m.start()))
        if not voted and not one_lane:
            bad.append(src[src.rfind("\n", 0, m.start()) + 1:src.find("\n", m.start())].strip())
    return bad


@pytest.mark.parametrize("name", ["window_attn.cu", "window_bwd.cu"])
def test_whole_warps_decide_their_waits_together(name):
    with open(os.path.join(CSRC, name)) as f:
        assert lone_decisions(f.read()) == []


def test_the_reading_tells_the_forms_apart():
    assert lone_decisions("if (w) { ok = guarded_wait(b); }") != []
    assert lone_decisions("if (w) { if (lane == 0) { for (;;) { ok = guarded_wait(b); } } }") == []
    assert lone_decisions("ok = __all_sync(m, ok && guarded_wait(b));") == []
    assert lone_decisions("if (lane == 0) { x(); } ok = guarded_wait(b);") != []


@pytest.mark.gpu
@pytest.mark.parametrize("ns", [0, -5, 1, 999_999])
def test_no_wait_limit_is_shorter_than_copies_in_flight_take(cuda_lib, ns):
    """The limit holds for a kernel's own copies too, which it waits for before
    it returns its shared memory: a limit below 1 ms counts as 1 ms, and real
    work does not run into it."""
    import torch
    from test_window_attn import make, run
    api = cuda_lib
    Q, K, V = make(1, 600, 8, 2, seed=1)
    want = run(api, Q, K, V, 100, 4)
    api.set_wait_limit(ns)
    try:
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        api.selftest_timeout()
        b.record()
        assert api.get_status() == api.STATUS_TIMEOUT
        assert a.elapsed_time(b) >= 0.99
        got = run(api, Q, K, V, 100, 4)
    finally:
        api.set_wait_limit(2_000_000_000)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
