"""Attention over caches whose value scales are far apart, in both kernels and in pieces, within a bound that counts every
token by its own weight and value scale: tokens that count for nothing, and those that other rows see, cost no bits."""
import numpy as np
import pytest

import bit_weight_only_pack_amd as lb
from kv_bounds import bounded
from kv_spread_cases import case, largest
from kv_util import DT, assert_within, attend

pytestmark = pytest.mark.gpu


def check(cache, batch, q, scale, dt, what):
    dtype, D = DT[dt][1], cache.D
    batch.device()
    y = attend(cache.handle(cache.device()), batch, q.cuda(), q.shape[1] * D, q.shape[1], dt, scale, 0, batch.rows, D, fill=7.0)
    want, bound = bounded(cache, batch, q.double().numpy(), scale, 0, dtype)
    assert_within(y, want, bound, what)


@pytest.mark.parametrize("kind,gaps", [("heavy", (8, 14, 20, 28, 40, 60)), ("behind", (8, 14, 20, 26, 40)),
                                       ("sinks", (8, 14, 20, 26, 40, 60)), ("ladder", (0, 4, 9, 16, 24))])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_spread(fmt, D, dt, kind, gaps):
    for gap in gaps:
        if dt == "f16" and gap > 26 and kind in ("behind", "sinks"):
            continue                                                  # past what fp16 holds of inputs or of results
        for n in ([1, 2], [9, 15], [1, 30], [70, 40]):
            cache, batch, q, scale = case(kind, fmt, D, dt, n, gap)
            check(cache, batch, q, scale, dt, "2^%d, rows %s" % (gap, n))


@pytest.mark.parametrize("kind,gap", [("heavy", 30), ("behind", 20), ("sinks", 24), ("ladder", 20)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_spread_in_pieces(fmt, dt, kind, gap):
    for n in ([1, 2], [70, 130]):
        cache, batch, q, scale = case(kind, fmt, 64, dt, n, gap, long=True)
        batch.device()
        assert lb.lowbit_kv_attention_workspace_bytes(cache.handle(256), batch.handle(), 4) > 0
        check(cache, batch, q, scale, dt, str(n))


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("offset", [False, True])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_values_up_to_the_largest(fmt, D, offset, long):
    """Weighted means of finite values are finite, whatever many tokens' sums would be."""
    for n in ([1, 2], [70, 130]):
        cache, batch, q, scale = largest(fmt, D, n, long, offset)
        check(cache, batch, q, scale, "bf16", str(n))


# queries, keys and scale times 2^these: scores of ordinary size
@pytest.mark.parametrize("dt,q_by,k_by,by", [("bf16", -120, 118, 2), ("bf16", -126, 121, 5), ("bf16", -100, 0, 100),
                                             ("bf16", 110, -105, -5), ("bf16", -60, 120, -60), ("bf16", -128, 120, 8),
                                             ("f16", 3, 122, -125), ("f16", 0, 100, -100), ("f16", -3, -97, 100)])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_scores_of_small_and_large_factors(fmt, dt, q_by, k_by, by):
    """Queries, keys and scales far from 1, whose product is not."""
    for n in ([1, 2], [9, 15], [70, 40]):
        cache, batch, q, scale = case("ladder", fmt, 64, dt, n, 0)
        for which in range(cache.arrays // 2):
            cache.meta(0, which)[:] = np.ldexp(cache.meta(0, which), k_by)
        q = (q.double() * 2.0 ** q_by).to(q.dtype)
        check(cache, batch, q, float(np.float32(np.ldexp(scale, by))), dt, str(n))
