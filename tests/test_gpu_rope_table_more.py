"""qnre_rope_table at its edges: frequencies of a few 2^-64 of a turn, and the default magnitude of stretched tables."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


@pytest.mark.parametrize("units", [0.6, 1.9, 2.4, 7.75, 1000.5])
def test_slowest_frequencies_are_rounded(units):
    """A position's share of a turn is held in units of 2^-64, rounded: p 2^-65 of a turn.  Sines this small show it (the value's own
    roundings: 2^-22 of it)."""
    first, n, rot = (1 << 31) - 50, 50, 16
    factor = 2.0 ** 64 / (2 * math.pi * units)        # so that pair 0, whose frequency is 1 / factor, turns by so many units
    out = torch.empty((n, rot), device="cuda")
    _qb().qnre_rope_table(out, first=first, scaling="linear", factor=factor)
    p = torch.arange(first, first + n, dtype=torch.float64)
    want = torch.sin(2 * math.pi * units * 2.0 ** -64 * p)
    err = (out[:, rot // 2].cpu().double() - want).abs()
    assert (err <= 2 * math.pi * p * 2.0 ** -65 + 2.0 ** -22 * want).all()


@pytest.mark.parametrize("factor,want", [(0.25, 1.0), (1.0, 1.0), (4.0, 0.1 * math.log(4.0) + 1.0)])
def test_default_magnitude_grows_with_stretched_tables_alone(factor, want):
    out = torch.empty((1, 64), device="cuda")
    _qb().qnre_rope_table(out, scaling="yarn", factor=factor, original=4096.0)
    assert (out[0, :32].cpu() - want).abs().max() <= 2.0 ** -23 and not out[0, 32:].any()
