"""The comparisons that the GPU tests of the log probabilities use notice what they are there for."""
import pytest
import torch

import row_ops_ref as ref


def test_a_swapped_top_list_is_noticed():
    x = ref.make_logits(4, 500, torch.float32, seed=2)
    x[2, [7, 90]] = 50.0  # two tied tokens at the head of a row
    want = ref.logprobs(x, None, 5, 1.0)["top_ids"]
    assert want[2, :2].tolist() == [7, 90]
    ref.tops_equal(want.int(), want)
    for row, a, b in ((0, 0, 1), (3, 3, 4), (2, 0, 1)):
        swapped = want.int()
        swapped[row, [a, b]] = swapped[row, [b, a]]
        with pytest.raises(AssertionError):
            ref.tops_equal(swapped, want)
    lost = want.int()
    lost[1, 4] = -1
    for wrong in (lost, want.int()[:, :4], want):  # a missing token, a shorter list, another type
        with pytest.raises(AssertionError):
            ref.tops_equal(wrong, want)
