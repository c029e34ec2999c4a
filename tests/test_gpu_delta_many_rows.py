"""The delta rule token by token in calls of many rows, whose workgroups take 64 rows of a state instead of 16: from 256 (up to
64 keys), 512 (128) and 1,024 (256) of the small ones on."""
import pytest

import test_gpu_delta as delta

pytestmark = pytest.mark.gpu

ROWS = [(70, 4, 2, 128, 32), (67, 4, 2, 100, 40), (70, 8, 4, 256, 32), (35, 4, 4, 200, 130), (90, 3, 1, 64, 17)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, heads, groups, kd, vd", ROWS)
def test_steps(rows, heads, groups, kd, vd, dtype):
    assert rows * heads * -(-vd // 16) > (256 if kd <= 64 else 512 if kd <= 128 else 1024)
    delta.test_steps(rows, heads, groups, kd, vd, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, heads, groups, kd, vd", ROWS)
def test_short_prompts(rows, heads, groups, kd, vd, dtype):
    delta.test_equal_prompts_without_a_state(rows, 7, heads, groups, kd, vd, dtype)
