"""Layer norm and its backward of odd rows whose last warp has no whole 16-byte vector of the tensor to itself: on the
last row its few columns lie in the tensor's last vector, which is cut short, and nothing of them can be copied in bulk."""

import pytest

from tests.test_gpu_layer_norm import _backward, _forward

pytestmark = pytest.mark.gpu

# One to seven columns (float32: one to three) past a whole number of warps' segments, in the last vector of one or
# several rows; the last of each type has a whole vector after all.
CASES = [("bf16", 1, 5121), ("bf16", 3, 5121), ("f16", 2, 5123), ("f16", 1, 5127), ("bf16", 1, 6401), ("bf16", 1, 7681),
         ("f16", 2, 15361), ("bf16", 5, 5129),
         ("f32", 1, 5121), ("f32", 3, 5121), ("f32", 1, 5123), ("f32", 1, 6401), ("f32", 3, 6401), ("f32", 2, 5125)]


@pytest.mark.parametrize("dt,R,C", CASES)
@pytest.mark.parametrize("resid", [True, False])
def test_layer_norm(dt, R, C, resid):
    _forward(R, C, dt, 0.3, resid)


@pytest.mark.parametrize("dt,R,C", CASES)
@pytest.mark.parametrize("resid", [True, False])
def test_layer_norm_backward(dt, R, C, resid):
    _backward(R, C, dt, 0.3, resid)


def test_more_rows_than_warps_at_once():
    """The row without a copy comes after others in the same stages."""
    _forward(1001, 5121, "bf16", 0.0, True)
    _backward(1001, 5121, "bf16", 0.0, True)
