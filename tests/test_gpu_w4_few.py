"""Products with 4-bit weights on both sides of each limit by which few rows of x take one kernel or the other:
x held whole or in chunks (two, or more than the three that are under way at a time), eight rows and nine, all of the weight's
rows at once or not, one row of a long reduction. The definition and its bounds are those of the other sizes."""
import pytest

from tests.test_gpu_w4 import built, check_linear, experts  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,group", (("int4", 128), ("fp4", 32)))
@pytest.mark.parametrize("k", (2048, 4128, 7168, 16384))
@pytest.mark.parametrize("rows", (1, 2, 3, 8, 9, 15, 16))
def test_experts_with_long_rows(rows, k, kind, group):
    k -= k % group
    experts([rows, 0, 1, max(1, rows - 1)], rows, k, 40, "none", kind, group)
    experts([rows], rows, k, 24, "swiglu", kind, group)


@pytest.mark.parametrize("rows", (1, 2, 8, 9, 14, 15, 16))
@pytest.mark.parametrize("k,n", [(2048, 4096), (2048, 2048), (2176, 2440), (4096, 4872), (512, 7304)])
def test_a_weight_of_one_round_or_two(rows, k, n):
    check_linear(rows, k, n, "relu", "int4", 128, True, True)


@pytest.mark.parametrize("k", (7168, 7296, 8192, 16384, 32768))
def test_one_long_row(k):
    check_linear(1, k, 200, "silu", "fp4", 128, True, True)


@pytest.mark.parametrize("rows", (8, 9))
def test_many_small_weights(rows):
    experts([rows, 0, 3, 1] * 100, rows, 128, 48, "swiglu", "int4", 64)
