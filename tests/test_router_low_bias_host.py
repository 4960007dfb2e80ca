"""The choice under a bias of FP32's lowest value, by hand."""
import numpy as np
import pytest

from oracle import router as R

LOW = np.finfo(np.float32).min


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_sums_of_lowest_values(score):
    z, b = np.zeros((1, 8)), np.full(8, LOW, np.float32)
    assert R.choose(z, 4, score, b, 4, 2).tolist() == [[0, 1, 2, 3]]
    assert R.choose(z, 3, score, b, 4, 2).tolist() == [[0, 1, 2]]
    b[:2] = -np.inf  # a group with nothing is no equal of one whose sum is -inf
    assert R.choose(z, 4, score, b, 4, 2).tolist() == [[2, 3, 4, 5]]
    assert R.choose(z, 2, score, b, 4, 1).tolist() == [[2, 3]]
    b[4] = -np.inf   # expert 5 alone: a finite value
    assert R.choose(z, 2, score, b, 4, 1).tolist() == [[5, -1]]
    assert R.choose(z, 4, score, b, 4, 2).tolist() == [[2, 3, 5, -1]]
    assert R.choose(z, 4, score, np.full(8, -np.inf, np.float32), 4, 2).tolist() == [[-1] * 4]
