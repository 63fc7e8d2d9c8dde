"""What the kernels of the 4-bit operators hand from one block or kernel to
another, read from their sources (no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_matrix_multiplication_sm_gb300", "csrc")


def sources():
    files = sorted(glob.glob(os.path.join(CSRC, "mx4_*")))
    assert files
    for path in files:
        with open(path) as f:
            yield os.path.basename(path), f.read()


def test_arrivals_on_another_blocks_barrier_have_cluster_scope():
    """Without a scope PTX takes the block's own, which orders nothing between two blocks."""
    found = 0
    for name, text in sources():
        for arrival in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster", text):
            found += 1
            assert re.search(r"\.(release|relaxed)\.cluster\.shared::cluster", arrival), (name, arrival)
    assert found


def test_relaxed_arrivals_come_after_a_fence():
    for name, text in sources():
        if "mbar_arrive_cluster(" not in text or name == "mx4_ptx.h":
            continue
        lines = text.split("\n")
        for i, line in enumerate(lines):
            if "mbar_arrive_cluster(" in line:
                before = "\n".join(lines[max(0, i - 5):i])
                assert "tc_fence_before()" in before or "release_smem()" in before, (name, i + 1)


def test_operands_are_not_read_as_read_only():
    """A kernel starts while the one before it still writes its operands
    (programmatic dependent launch): loads for what nothing writes while the
    kernel runs may not be used for them, and may move above the wait."""
    for name, text in sources():
        code = re.sub(r"//.*", "", text)
        for what in ("__ldg", "ld.global.nc", "__restrict__"):
            assert what not in code, (name, what)


def test_kernels_that_take_all_tensor_memory_have_an_sm_to_themselves():
    """Their wait for it has no limit, and blocks of a cluster wait for each
    other: two clusters on the same SMs could each hold what the other needs.
    An SM has 228 KB of shared memory, 1 KB of it taken for each block."""
    kb = 1024
    text = dict(sources())
    limit = int(re.search(r"SMEM_LIMIT = (\d+) \* 1024;", text["mx4_weights_tmem.cu"])[1]) * kb
    assert re.search(r"ONE_BLOCK = SMEM_LIMIT / 2 \+ 1024;", text["mx4_weights_tmem.cu"])
    assert re.search(r"smem_bytes<FMT>\(p\.rows\) > ONE_BLOCK \? smem_bytes<FMT>\(p\.rows\) : ONE_BLOCK;", text["mx4_weights_tmem.cu"])
    assert 2 * (limit // 2 + kb + kb) > 228 * kb
    # The others' stages alone, in bytes.
    for name, stage in (("mx4_gemm.cu", 2 * 128 * 128), ("mx4_weights.cu", 2 * 128 * 128)):
        stages = int(re.search(r"constexpr int STAGES = (\d+);", text[name])[1])
        assert 2 * (stages * stage + kb) > 228 * kb, name
