"""Where the operators of a pass over several new tokens begin to refuse sizes (no
GPU needed: a refusal comes before the first CUDA call, which fails here)."""
import pytest
import torch

from test_chunk_ops_host import INVALID, OK, UNSUPPORTED, lib, matmul  # noqa: F401

CUDA = 3  # what a call that is not refused ends with where there is no GPU
MOST_K = (1 << 31) - 272  # the last multiple of 16 whose blocks' ends are 32-bit


@pytest.mark.parametrize("k", [MOST_K + 16, MOST_K + 32, MOST_K + 128, (1 << 31) - 16])
def test_products_whose_blocks_of_k_would_pass_32_bits(lib, k):  # noqa: F811
    for m, n in ((1, 1), (5, 7), (0, 7)):
        assert matmul(lib, m=m, n=n, k=k) == UNSUPPORTED


def test_the_longest_product(lib):  # noqa: F811
    assert matmul(lib, m=0, k=MOST_K) == OK
    assert matmul(lib, k=MOST_K + 8) == INVALID
    if not torch.cuda.is_available():
        assert matmul(lib, k=MOST_K) == CUDA
