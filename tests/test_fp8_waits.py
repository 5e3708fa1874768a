"""The waits of fp8_gemm.cu, read from its source.

A wait is bounded by a timer that each lane reads by itself, so where one runs out the lanes of a warp
may disagree. Running out cannot be provoked without a fault in the kernel, so the rule that keeps
the end of such a kernel defined is checked in the text: a lane leaves a loop on its own finding
only where it works alone (under `if (lane == 0)`), or where nothing in the loop is the whole warp's
(warp 2, whose lanes copy scales); else the warp votes first.
"""
import os
import re

SOURCE = os.path.join(os.path.dirname(__file__), "..", "int4_quantized_b200", "csrc", "fp8_gemm.cu")


def text():
    with open(SOURCE) as f:
        return re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), f.read())


def opened_before(s, at):
    """The heads (text before each `{`) of the blocks that hold position `at`, outermost first."""
    heads, last = [], 0
    for m in re.finditer(r"[{};]", s[:at]):
        if m.group() == "{":
            heads.append(s[last:m.start()].strip())
        elif m.group() == "}":
            heads.pop()
        last = m.end()
    return heads


def test_a_warp_leaves_a_loop_together():
    s = text()
    jumps = [m.start() for m in re.finditer(r"if \(timed_out\) break;|timed_out = true;\s*break;", s)]
    assert len(jumps) >= 6
    for at in jumps:
        heads = opened_before(s, at)
        if any(re.fullmatch(r"if \(lane == 0\)", h) for h in heads):
            continue
        if any(re.fullmatch(r"(else )?if \(warp == 2\)", h) for h in heads):
            body = s[s.rfind("warp == 2", 0, at):s.index("cp.async.wait_all", at)]
            assert not re.search(r"_sync\(|__sync|elect_one|tmem_|cluster_|\.aligned|named_barrier", body)
            continue
        decided = s[s.rfind("mbar_wait(", 0, at) - 80:at]
        assert re.search(r"__(any|all)_sync\(0xffffffffu", decided), f"line {s.count(chr(10), 0, at) + 1}: lanes leave by themselves"


def test_every_wait_is_bounded():
    # nothing waits on a barrier but by mbar_wait
    s = text()
    assert not re.search(r"mbarrier\.(try_wait|test_wait)|mbar_try_wait|while \(true\)|for \(;;\)", s)


def test_blocks_of_a_pair_wait_for_the_arrivals_they_get():
    # the tensor core's arrivals go to the barriers of both blocks of a pair: each waits for its last
    # ones before it may end (and its shared memory become another block's)
    s = text()
    wide = s[s.index("fp8_wide(const Fp8Args"):s.index("bool encode_codes_map")]
    assert re.search(r"mbar_wait\(\(PAIR \? empty : full\) \+ i,", wide)
    first, second = wide[wide.index("} else if (warp == 1 && rank == 0) {"):].split("} else if (warp == 1) {", 1)
    assert "mbar_wait(done, 0)" in first and "mbar_wait(done, 0)" in second.split("}", 1)[0]
