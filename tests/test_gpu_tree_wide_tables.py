"""Attention of trees over tables as wide as a model's context whatever the texts'
lengths: both sides of the rules that choose the kernels.  Inputs, the 64-bit form and
the tolerance are those of test_gpu_tree_attention."""
import pytest

from gpt_transformer_forward_gb300 import binding as ab

from draft_reference import trees
from gpu_helpers import need_gpu, no_device_error
from test_gpu_tree_attention import check, make, ragged

pytestmark = pytest.mark.gpu
TYPES16, IDS16 = [ab.GPT2_BF16, ab.GPT2_FP16], ["bf16", "fp16"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def wide(precision, B, N, NH, most, capacity, bs=16, seed=1, hs=64):
    """Texts of 0 to `most` positions in a table of `capacity`."""
    pos = ragged(B, most, seed)
    row = (most + N - 1) // bs + 1
    c = make(precision, N, NH, hs, pos, bs, trees(B, N, seed=seed), seed=seed, spare=capacity // bs - row)
    assert c["table"].shape[1] * bs == capacity
    return c


@pytest.mark.parametrize("precision", TYPES16, ids=IDS16)
@pytest.mark.parametrize("B,NH,capacity,most", [
    (26, 12, 1024, 60), (26, 12, 1024, 500), (26, 12, 1040, 60), (25, 12, 1024, 60), (25, 12, 768, 300),
    (13, 12, 768, 700), (12, 12, 1024, 300), (8, 38, 1024, 960), (1, 12, 1024, 960), (101, 3, 1024, 90),
])
@pytest.mark.parametrize("N", [33, 64])
def test_wide_trees_in_a_models_context(precision, B, NH, capacity, most, N):
    """On both sides of two pairs an SM and one, and of 768 and 1024 positions."""
    check(wide(precision, B, N, NH, most, capacity, seed=B + N))
    no_device_error()
