"""The block-scale decode kernel's code stays small enough for the SM's instruction caches
(its sixteen warps run six roles; see tests/test_code_size.py for what code size costs these
kernels). With two merge sites and unrolled index loops it was 91 KB (2 query heads per kv
head) and 105 KB (4), and 1 to 2% slower. Budgets are the current sizes plus ~15%."""
from tests.test_code_size import _check, _code_sizes


def test_blockscale_decode_kernel_code_fits(tmp_path):
    sizes = _code_sizes(tmp_path, "decode_blockscale.cu", r"decode_blockscale_kernelILi(\d+)E")
    _check(sizes, {("1",): 74 * 1024, ("2",): 80 * 1024, ("4",): 90 * 1024, ("8",): 108 * 1024},
           "decode_blockscale_kernel")
