"""The combination's backward for row lengths on both sides of every split of a row over warps."""

import pytest

from tests import test_gpu_experts as experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", [256, 257, 264, 500, 512, 520, 600, 768, 776, 1024, 1025, 1281, 1288, 1536, 1800, 2304, 2560, 2568, 5120,
                               5121, 8192])
def test_combine_and_its_backward(dt, C):
    experts.test_combine_and_its_backward(dt, 45, 3, C)
