"""The convolution's SiLU and its slope over their whole range, float32."""
import pytest
import torch

import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu


def test_silu_over_its_range():
    """A filter that passes its input on: y = silu(x) from -85 to 85.  The exponential, the
    reciprocal, 1 + e and two products round: 2^-20 of y wherever x lies.  The slope
    s + p s (1 - s): three more steps, by the size of each term."""
    x = torch.linspace(-85, 85, 64 * 40000, device="cuda").view(1, 1, 40000, 64)
    w = torch.zeros(1, 64, 2, device="cuda")
    w[..., 1] = 1
    p = x.double()
    s = torch.sigmoid(p)
    y = sdm.conv_forward(x, w)
    assert float(((y.double() - p * s).abs() / (p * s).abs().clamp_min(1e-30)).max()) <= 2.0 ** -20
    dx = sdm.conv_backward(x, w, torch.ones_like(x))["x"].double()
    c = torch.sigmoid(-p)
    bound = 2.0 ** -20.5 * s + 2.0 ** -19.5 * p.abs() * s * c
    assert float(((dx - (s + p * s * c)).abs() / bound).max()) <= 1
