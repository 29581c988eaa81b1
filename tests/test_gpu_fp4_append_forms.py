"""The FP4 append on both sides of each change of its form: a token to a warp up
to 4,096 tokens, then runs of two, three and more."""
import pytest

import test_gpu_fp4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [4095, 4096, 4097, 6080, 6081, 12160, 12161, 18241])
def test_append_forms(cuda_lib, n):
    """Every byte of every row, with tokens out of range among them."""
    test_gpu_fp4.test_append_many_tokens(cuda_lib, n)
