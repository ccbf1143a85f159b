"""Slow pairs: the sine of a small angle to its own precision.

With x_b = 0, y_b = x_a sin t.  The angle is rounded as two words (1.5 2^-24 of it at
most, and as much of its sine where the angle is small), sincospi is within one
unit (2 2^-24), the product with x_a is rounded once: below 6 2^-24 of y_b.  The
frequency itself is held to 2^-65 turns: at 1e-6 radians, 1.6e-7 turns, below 2^-42 of
it."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import sca  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D", [64, 66])     # vectors of 16 bytes; single elements
def test_sines_of_small_angles(sca, layout, D):
    f = [10.0 ** (-2 - 4 * i / (D // 2)) for i in range(D // 2)]       # 1e-2 to 1e-6 radians a position
    angles = sca.RotaryAngles(D, layout=layout, frequencies=f)
    pos = torch.tensor([1, -1, 3, -7, 20], dtype=torch.int32)
    i = np.arange(D // 2)
    a, b = (i, i + D // 2) if layout == "half" else (2 * i, 2 * i + 1)
    x = torch.zeros(1, 1, len(pos), D)
    x[..., a] = torch.rand(1, 1, len(pos), D // 2, generator=torch.Generator().manual_seed(1)) + 0.5
    y, _ = sca.RotaryPositions(1, 1, len(pos), D, angles, dtype=torch.float32).forward(x.cuda(), x.cuda(), positions=pos.cuda())
    want = x[0, 0][:, a].double().numpy() * np.sin(pos.double().numpy()[:, None] * np.array(f))
    got = y[0, 0][:, b].double().cpu().numpy()
    assert (np.abs(got - want) <= 6 * 2.0 ** -24 * np.abs(want)).all(), (np.abs(got / want - 1)).max()
