"""Draft verification on the GPU at the ends of its arguments' ranges, against float64 on the CPU."""
import math

import pytest
import torch

from test_gpu_verify import _compare, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tau", [1e30, 1e36, 1e38])
@pytest.mark.parametrize("V", [50, 9000])
def test_the_highest_temperatures(tau, V):
    """Logits of the temperature's size, some forbidden: every finite one weighs something."""
    t, d, x, u = _inputs(8, 3, V, seed=3, spread=1.0)
    t, d = (t * tau).clamp(-3.4e38, 3.4e38), (d * tau).clamp(-3.4e38, 3.4e38)
    t[:, :, 3:20] = -math.inf
    d[:, :, 5:30] = -math.inf
    tau = float(torch.tensor(tau, dtype=torch.float32))
    _compare(t, d, x, tau, u)
    _compare(t, None, x, tau, u)
