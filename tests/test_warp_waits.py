"""The tensor-core kernels' bounded waits, by reading their sources: no GPU.

A wait gives up by a clock and a flag that each lane reads for itself, so lanes of one warp may answer differently
where a limit runs out as a phase completes. Warps whose lanes go on together (tcgen05.ld, __syncwarp, elect.sync) need
one answer. (No launch shows it: a lost phase completes for no lane.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_row_online_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_the_warps_wait_asks_all_lanes():
    body = re.search(r"bool warp_wait\([^)]*\) \{([^}]*)\}", source("hl_tc.cuh")).group(1)
    assert re.search(r"return __all_sync\(0xffffffffu, wait_phase\(", body)


def test_the_8_bit_products_warps_wait_together():
    text = source("hl_fp8_gemm.cu")
    assert text.count("warp_wait(") >= 3
    # a lane's own answer, where it is taken, decides nothing before all lanes have heard it
    own = [m.start() for m in re.finditer(r"(?<!\w)wait_phase\(", text)]
    assert len(own) == text.count("const bool there = wait_phase(") <= 1
    for at in own:
        end = text.index("__all_sync(0xffffffffu, there)", at)
        between = text[text.index(";", at):end]
        assert not re.search(r"there|break|return|continue|go\b(?! = $)", between)


def test_the_bf16_products_epilogue_waits_together():
    text = source("lmhead_tc.cu")
    kernel = text[text.index("lmhead_gemm_kernel("):]
    single = kernel[kernel.index("if (lane == 0) {"):kernel.index("const int q = warp & 3;")]  # the roles of one lane
    whole = kernel[kernel.index("const int q = warp & 3;"):]
    assert single.count("wait_phase(") == 3
    assert whole.count("wait_phase(") == len(re.findall(r"__all_sync\(0xffffffffu, wait_phase\(", whole)) == 1
