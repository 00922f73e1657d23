"""Draft verification on the GPU at the ends of its arguments' ranges, against float64 on the CPU."""
import math

import pytest
import torch

from test_gpu_verify import _compare, _inputs, _run

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


@pytest.mark.parametrize("with_draft", [True, False])
def test_a_test_on_its_border_is_refused_whatever_the_logits_size(with_draft):
    """p(x) = 1/2 exactly and u q(x) = 1/2: not below. The rows' sums are rounded with their largest
    logit's product, which must not tell on one side only."""
    n = 400
    t = torch.full((n, 2, 8), -math.inf)
    t[:, :, :2] = torch.linspace(1e5, 2.8e6, n)[:, None, None]
    d = torch.full((n, 1, 8), -math.inf)
    d[:, 0, 0] = torch.linspace(2.8e6, 1e5, n)
    x = torch.zeros((n, 1), dtype=torch.long)
    u = torch.full((n, 2), 0.5)
    out, counts = _run(t, d if with_draft else None, x, 1.0, u)
    assert (counts == 1).all() and (out[:, 0] == 1).all()
    u[:, 0] = 0.5 - 2.0 ** -25  # the number below: accepted
    out, counts = _run(t, d if with_draft else None, x, 1.0, u)
    assert (counts == 2).all() and (out[:, 0] == 0).all()


@pytest.mark.parametrize("with_draft", [True, False])
def test_logits_further_apart_than_the_type_reaches(with_draft):
    """Logits of both signs near the type's ends, at a temperature where the lower ones weigh a tenth
    of the upper ones: their difference is no finite number in 32 bits."""
    n, V = 64, 40
    g = torch.Generator().manual_seed(1)
    t = torch.where(torch.rand((n, 2, V), generator=g) < 0.5, 3.3e38, -3.3e38)
    t[:, :, 0] = 3.3e38
    d = torch.where(torch.rand((n, 1, V), generator=g) < 0.5, 3.2e38, -3.1e38)
    x = torch.randint(0, V, (n, 1), generator=g)
    u = torch.rand((n, 2), generator=g) * (1.0 if with_draft else 0.06)
    tau = float(torch.tensor(3e38, dtype=torch.float32))
    _compare(t, d if with_draft else None, x, tau, u)
