"""The norm's gradient at every rank count up to nine in fp32 and bf16, on rows of whole waves, of lanes, and wider than a
wave's slots, with more rows than the resident workgroups take at once and fewer: the next row is read ahead at some counts
and not at others."""
import pytest

from test_gpu_block import BF16, F32
from test_gpu_block_paths import check_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", range(1, 10))
@pytest.mark.parametrize("rows,hidden,dt,save8,in_place", [
    (600, 2048, F32, False, False), (1500, 4096, F32, True, True), (4500, 200, F32, True, False), (2600, 120, F32, False, True),
    (600, 2048, BF16, True, True), (300, 8200, F32, False, False)])
def test_norm_bwd(n, rows, hidden, dt, save8, in_place):
    check_bwd(n, rows, hidden, dt, True, save8, 0, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,rows,hidden,dt", [
    (1, 256, 200, BF16), (7, 256, 520, BF16), (7, 255, 520, F32), (8, 244, 1024, BF16), (8, 245, 1024, BF16), (8, 122, 1024, F32),
    (8, 123, 1024, F32), (16, 129, 300, BF16), (16, 130, 300, BF16), (40, 53, 4096, BF16), (64, 33, 200, BF16), (64, 34, 200, BF16),
    (64, 16, 8192, F32), (64, 17, 8192, F32)])
def test_one_launch_and_two(n, rows, hidden, dt, in_place):
    """Both sides of the number of reads up to which the gradient is one launch."""
    check_bwd(n, rows, hidden, dt, True, True, 0, in_place)
