"""What the header of the 4-bit operators promises, against their sources (no GPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def read(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def test_the_header_says_when_gemm_w4_takes_scratch():
    """An A off 16 bytes is copied wherever the kernel for few rows, which reads
    it as it is, does not take the product."""
    csrc = ("tiled_matrix_multiplication_sm_gb300", "csrc")
    few = re.search(r"mx4_few_rows\(int M, int N, int K\) \{ return M <= (\d+) \|\| \(M <= MX4_FEW_ROWS && "
                    r"\(long\)N \* K < 1L << (\d+)\); \}", read(*csrc, "mx4_internal.h"))
    most = re.search(r"MX4_FEW_ROWS = (\d+);", read(*csrc, "mx4_internal.h"))
    cols = re.search(r"if \(mx4_few_rows\(M, N, K\) && K < 1 << (\d+)\)", read(*csrc, "mx4_weights.cu"))
    says = re.search(r"where M > (\d+),\s+where M > (\d+) and N K >= 2\^(\d+), and where K >= 2\^(\d+)",
                     re.sub(r"\n \* ", " ", read("include", "tgemm_mx4.h")))
    assert says, "the header's rule"
    assert says.groups() == (most[1], few[1], few[2], cols[1])
