"""The error bounds of attention over the key/value cache, on the CPU: they hold for operands as the kernels take them, and
fail for operands of fewer bits or taken to another row's value scales."""
import numpy as np
import pytest
import torch

from kv_bounds import bounded, far, in_16_bits
from kv_spread_cases import case, filled
from kv_util import DT, Batch, rows


def sides(kind, fmt, D, dt, gap, parts, by_row):
    cache, batch, q, scale = case(kind, fmt, D, dt, [1, 30], gap)
    y, bound = bounded(cache, batch, q.double().numpy(), scale, 0, DT[dt][1])
    return far(in_16_bits(cache, batch, q.double().numpy(), scale, 0, DT[dt][1], parts, by_row), y, bound)


@pytest.mark.parametrize("kind,gap", [("heavy", 20), ("behind", 20), ("sinks", 26), ("ladder", 20)])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_bounds_hold_by_row(fmt, D, kind, gap):
    assert sides(kind, fmt, D, "f16", gap, 2, True) <= 1
    assert sides(kind, fmt, D, "bf16", gap, 1, True) <= 1


@pytest.mark.parametrize("fmt", ["i8", "u4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_part_is_told_from_two(fmt, D):
    assert sides("behind", fmt, D, "f16", 20, 2, True) <= 1 < sides("behind", fmt, D, "f16", 20, 1, True)


@pytest.mark.parametrize("fmt", ["i8", "u4"])
@pytest.mark.parametrize("kind,gap,dt", [("heavy", 20, "f16"), ("heavy", 28, "bf16"), ("behind", 20, "f16"),
                                         ("behind", 32, "bf16"), ("sinks", 40, "bf16")])
def test_another_rows_scales_are_told_from_its_own(fmt, kind, gap, dt):
    assert sides(kind, fmt, 64, dt, gap, 2 if dt == "f16" else 1, False) > 1


@pytest.mark.parametrize("fmt", ["i8", "u4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_part_is_told_from_two_over_ordinary_rows(fmt, D):
    """Queries of both signs, weights much alike: what the test of the kernels takes."""
    rng = np.random.default_rng(D)
    cache = filled(rng, fmt, 14, 64, 1, D, torch.float16)
    batch = Batch(cache, [60, 20], [500, 100], rng)
    q = rows(rng, batch.rows, 2, D, torch.float16)
    y, bound = bounded(cache, batch, q.double().numpy(), 0.004, 0, torch.float16)
    one, two = (far(in_16_bits(cache, batch, q.double().numpy(), 0.004, 0, torch.float16, parts), y, bound) for parts in (1, 2))
    assert two <= 1 < one
