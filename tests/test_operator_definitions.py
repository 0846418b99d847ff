"""CPU: the fp64 definitions behind the operator tests against closed forms and torch, and the rotary table
(a host function of the library) against its definition."""
import math

import numpy as np
import pytest
import torch

from oracle import operators as R


def test_round8_matches_every_e4m3_value_and_midpoint():
    vals = np.arange(0, 127, dtype=np.uint8)             # 0 .. 448, the format's non-negative numbers in order
    num = torch.from_numpy(vals).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round8(num, "e4m3"), num)
    mid = (num[:-1] + num[1:]) / 2
    even = np.where(vals[:-1] % 2 == 0, num[:-1], num[1:])
    assert np.array_equal(R.round8(mid, "e4m3"), even)   # ties to even
    assert np.array_equal(R.round8(mid * (1 - 1e-9), "e4m3"), num[:-1])
    assert np.array_equal(R.round8(-mid * (1 + 1e-9), "e4m3"), -num[1:])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_block_scale_is_the_smallest_power_of_two_that_fits(fmt):
    q = R.QMAX[fmt]
    for e in (-99, -20, 0, 7, 100):
        assert R.block_scale(q * 2.0 ** e, fmt) == 2.0 ** e
        assert R.block_scale(q * 2.0 ** e * (1 + 1e-12), fmt) == 2.0 ** (e + 1)
    assert R.block_scale(0.0, fmt) == 2.0 ** -100 and R.block_scale(1e-40, fmt) == 2.0 ** -100
    assert math.isnan(R.block_scale(math.inf, fmt)) and math.isnan(R.block_scale(math.nan, fmt))


def test_growing_block_keeps_int8_values_within_one_step():
    rng = np.random.default_rng(3)
    for _ in range(50):
        block, x = R.Block(8, "int8"), rng.normal(size=(16, 8)) * np.exp(rng.normal(size=(16, 1)) * 2)
        for t in range(16):
            block.write(t, x[t:t + 1])
        assert np.abs(block.values() - x).max() <= block.scale        # 1/2 (1 + 1/2 + 1/4 + ...) steps


def test_rope_preserves_norms_and_relative_positions():
    rng = np.random.default_rng(1)
    turns = R.rope_turns(16)
    q, k = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    for layout in ("half", "interleaved"):
        a = R.rope(q, [70], turns, layout)
        assert np.allclose(np.linalg.norm(a), np.linalg.norm(q), rtol=1e-12)
        d = [float((R.rope(q, [p + 5], turns, layout) * R.rope(k, [p], turns, layout)).sum()) for p in (0, 9, 1000)]
        assert np.allclose(d, d[0], rtol=1e-9)
    assert np.allclose(R.rope(q, [0], turns), q)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=128), dict(rotary_dim=2, base=500000.0), dict(rotary_dim=64, scaling="linear", factor=4.0),
    dict(rotary_dim=128, scaling="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
    dict(rotary_dim=96, scaling="bands", factor=40.0, original_len=4096.0, low=1.0, high=32.0),
    dict(rotary_dim=6, scaling="bands", factor=1.0, original_len=1.0, low=0.0, high=1e-3),
])
def test_rope_table_matches_its_definition(kw):
    import long_context_layer_b200 as L
    kinds = {"plain": L.DELTA_ROPE_PLAIN, "linear": L.DELTA_ROPE_LINEAR, "bands": L.DELTA_ROPE_BANDS}
    p = L.DeltaRopeParams(kw["rotary_dim"], kinds[kw.get("scaling", "plain")], kw.get("base", 10000.0),
                          kw.get("factor", 1.0), kw.get("original_len", 0.0), kw.get("low", 0.0), kw.get("high", 1.0))
    got, ref = np.array(L.rope_table(p)), R.rope_turns(**kw)
    assert got.shape == ref.shape
    # pow, a division by 2 pi and at most five more operations in double on either side
    assert np.all(np.abs(got - ref) <= 32 * 2.0 ** -53 * np.abs(ref) * max(1.0, kw.get("factor", 1.0)))


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=-2), dict(scaling=3), dict(base=1.0), dict(base=math.inf),
    dict(base=math.nan), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan), dict(scaling=2, original_len=0.0),
    dict(scaling=2, low_turns=4.0, high_turns=4.0), dict(scaling=2, low_turns=-1.0), dict(scaling=2, high_turns=math.inf),
])
def test_rope_table_refusals(bad):
    import long_context_layer_b200 as L
    kw = dict(rotary_dim=64, scaling=0, base=10000.0, factor=2.0, original_len=4096.0, low_turns=1.0, high_turns=32.0)
    kw.update(bad)
    with pytest.raises(L.DeltaError):
        L.rope_table(L.DeltaRopeParams(*kw.values()))


def test_visible_tokens():
    assert R.visible(10, 3, 2) == [0, 1, 7, 8, 9]
    assert R.visible(4, 3, 2) == [0, 1, 2, 3]
    assert R.visible(5, 0, 0) == [] and R.visible(0, 4, 4) == []
    assert R.visible(5, 100, 0) == list(range(5))
