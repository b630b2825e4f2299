"""Cases run against the debug build of the library (``RMSNORM_LIBRARY=<debug .so> python -m
tests.serving_debug_cases``): products whose blocks of a cluster share K, with one warp of one block
that acts as if a wait had given up. Its sums lack blocks of K, so no block of the cluster may
store: the output stays as it was, bit 0 of the device error word is set, and the next
product is right.
"""
import sys

import torch

from rmsnorm_fwd_bwd_gb300 import binding as B
from tests.test_serving_gpu import check_product, product_inputs

# few rows and 128 x 128 tiles, by TMA and by the loaders of rows off 16 bytes
CASES = [(8, 512, 2048), (50, 300, 1024), (9, 512, 2051), (100, 300, 4096), (200, 130, 4099)]


def main() -> int:
    assert B.LIB_PATH.endswith("librmsnorm_debug.so"), B.LIB_PATH
    B.rmsnorm_device_error(clear=True)
    wrong = []
    for M, N, K in CASES:
        a, lda, b, ldb, sa, sb = product_inputs(M, N, K, 128, 61)

        def product():
            y = torch.full((M, N + 1), 7.0, device="cuda")
            assert B.rmsnorm_quant_matmul(a, lda, sa, sa.shape[1], b, ldb, sb, sb.shape[1], None, y, N + 1, M, N, K, "float32",
                                          128) == 0
            return y
        for rank in (0, 1):
            assert B.rmsnorm_selftest_matmul_gives_up(rank) == 0
            y = product()
            word = B.rmsnorm_device_error(clear=True)
            if word != 1 or not (y == 7.0).all():
                wrong.append((M, N, K, rank, word, int((y != 7.0).sum())))
            assert B.rmsnorm_selftest_matmul_gives_up(-1) == 0
            check_product(a, b, sa, sb, "float32", 128, product())
            assert B.rmsnorm_device_error(clear=True) == 0
    print(f"products that gave up: {len(wrong)} of {2 * len(CASES)} stored something or reported nothing: {wrong}")
    return 1 if wrong else 0


if __name__ == "__main__":
    sys.exit(main())
