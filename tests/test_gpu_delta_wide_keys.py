"""Prompts with more than 128 keys in calls of few workgroups, one on a CU."""
import pytest

import test_gpu_delta as delta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [delta.LENGTHS, delta.LONG], ids=["both paths", "blocks alone"])
@pytest.mark.parametrize("heads, groups, kd, vd", [(1, 1, 256, 40), (2, 1, 200, 32), (4, 2, 256, 16)])
def test_ragged_prompts(heads, groups, kd, vd, lengths, dtype):
    """One to several blocks of tokens, carried states, rows behind the last sequence: 27 to 36 workgroups."""
    delta.test_ragged_prompts(heads, groups, kd, vd, lengths, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs, each, heads, groups, kd, vd", [(9, 31, 2, 1, 256, 32), (9, 32, 2, 2, 200, 32), (9, 33, 2, 1, 200, 32), (70, 24, 8, 4, 256, 32), (1, 200, 2, 1, 256, 256), (2, 300, 1, 1, 256, 40), (1, 257, 2, 1, 200, 32), (1, 64, 4, 4, 256, 16)])
def test_equal_prompts(seqs, each, heads, groups, kd, vd, dtype):
    delta.test_equal_prompts_without_a_state(seqs, each, heads, groups, kd, vd, dtype)
