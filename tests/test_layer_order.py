"""Orders in the layer kernels that nothing but their source shows: what a race or a missing wait would
spoil only now and then on a GPU."""
import os
import re

import heterogeneous_adapters_sgmv_b200 as L

CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")


def part(name, start, end):
    """The source between two marks, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    src = src[src.index(start):]
    return re.sub(r"//[^\n]*", "", src[:src.index(end)])


def test_gemm_issuer_reads_a_stage_before_it_gives_it_back():
    """The commit on a stage's `empty` barrier lets the producer write the stage's record (`last`, `lo`,
    `hi`) for its next use, so the issuer has to have read all of it before."""
    src = part("layer_gemm.cu", "---- MMA issuer", "---- epilogue")
    loop = src[src.index("bool last"):]
    reads = [m.start() for m in re.finditer(r"ctl\.(?:last|lo|hi)\[", loop)]
    assert len(reads) == 3
    # each branch (base product, adapters) commits once; lo and hi are read in the second only
    base, adapters = [m.start() for m in re.finditer(r"umma_commit_pair\(empty0", loop)]
    assert loop.index("ctl.last[") < base
    assert loop.index("ctl.lo[") < adapters and loop.index("ctl.hi[") < adapters


def test_weight_pass_waits_before_it_reads_anything():
    """Without a shrink in front (`early` is 0) the producer's wait for the stream's earlier work comes before
    its first load, of W as of x: W may have been written by the kernel before."""
    src = part("layer_stream.cu", "---- producer", "---- MMA issuer")
    assert src.count("pdl_wait()") == 1 and src.index("pdl_wait()") < src.index("tma_load_2d(")
    before = src[:src.index("pdl_wait()")]
    # what stands before it asks L2, and changes nothing
    assert "if (!p.early)" in before and before.count("&p.tm_w") == before.count("tma_prefetch_2d(") == 1
