"""The rotation's cosines and sines on their own, against exact angles: positions up to 2^31 - 1."""

import math
from fractions import Fraction

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P

pytestmark = pytest.mark.gpu

#: 1 / 2 pi to 40 digits: off by 1e-41 of a turn per position and unit of frequency
INV = Fraction("0.1591549430918953357688837633725143620345")


def exact(positions, freq):
    """cos and sin [positions, pairs] in float64 of angles whose whole turns are taken out exactly."""
    turns = [int(Fraction(f) * INV * 2 ** 160) for f in freq]
    half = 1 << 159
    angle = [[2 * math.pi * (((p * t + half) % (1 << 160)) - half) / 2 ** 160 for t in turns] for p in positions]
    return torch.tensor(angle, dtype=torch.float64).cos(), torch.tensor(angle, dtype=torch.float64).sin()


def bounds(c, s):
    """Of a computed cosine c (of a sine s, the other way round): sincospi is within 1 ulp, of a value that
    lies up to 6.0e-6 (2^-20 of a turn) beside c; the correction rounds once more; the angle is cut at 2^-32 of
    a turn and its frequency is off by 3 2^-64 turns a position, 2^31 of them: 5/2 2^-32 2 pi; the
    correction's second order is 2^-41 (pi 2^-19, squared, half)."""
    return 2.0 ** -23 * (c.abs() + 6.0e-6) + 2.0 ** -24 * c.abs() + 2.5 * 2.0 ** -32 * 2 * math.pi * s.abs() + 2.0 ** -35


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,theta", [(128, 1e4), (64, 1e6)])
def test_cosines_and_sines(layout, dim, theta):
    g = torch.Generator().manual_seed(dim)
    pos = torch.randint(0, 2 ** 31 - 1, (1500,), generator=g)
    pos[:4] = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 31 - 2])
    pos[4:500] %= 1 << 20
    rope = P.PagedRope(dim, theta, layout)
    x = torch.zeros(len(pos), 1, dim, device="cuda")
    one, two = (slice(0, dim // 2), slice(dim // 2, dim)) if layout == "half" else (slice(0, dim, 2), slice(1, dim, 2))
    x[..., one] = 1.0                                      # (1, 0) turns to (cos, sin)
    y = torch.empty_like(x)
    P.paged_norm_rope(pos.int().cuda(), rope, q=x, q_out=y)
    y = y[:, 0].double().cpu()
    c, s = exact(pos.tolist(), rope.inv_freq)
    for got, want, other in ((y[:, one], c, s), (y[:, two], s, c)):
        off = (got - want).abs() / bounds(want, other)
        assert (off <= 1).all(), (float(off.max()), (off > 1).nonzero()[:3].tolist())
