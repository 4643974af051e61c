"""What the layer in parts answers at its edges, as far as it can be told without a GPU."""
import numpy as np

from oracle import parts


def test_the_oracle_drops_values_that_are_not_finite():
    x = np.zeros((1, 256))
    x[0, :3], x[0, 128:131] = [np.inf, 1.0, 3.0], [1.0, -np.inf, 3.0]
    d = np.ones((1, 128))
    d[0, 2] = np.inf
    with np.errstate(invalid="ignore"):
        got, mag = parts.act_backward(x, d, clamp=2.0)
    assert np.array_equal(got[0, [0, 1, 2, 128, 129, 130]], np.zeros(6)) and np.isfinite(mag[0, :3]).all()
