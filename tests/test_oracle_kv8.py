"""Pins of the 8-bit cache oracle (CPU): the library cast, the definition's
inequalities, and the error of a value against its unrounded one."""
import numpy as np
import pytest
import torch

from oracle import kv8 as O8
from query_aware_sparse_decode_b200 import tb as TB


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rounding_equals_the_library_cast(fmt):
    rng = np.random.default_rng(3)
    y = np.concatenate([rng.normal(size=4000) * 50, np.linspace(-2, 2, 4097) / 64, [448, -448, 0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    y = np.float32(np.clip(y, -O8.LARGEST[fmt], O8.LARGEST[fmt]))
    if fmt == "e4m3":
        want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    else:
        want = torch.from_numpy(y).round().double().numpy()
    assert np.array_equal(O8.round_code(y, fmt), want)
    # every value of the format is its own rounding
    codes = np.arange(256, dtype=np.uint8)
    vals = torch.from_numpy(codes).view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).double().numpy()
    vals = vals[np.isfinite(vals) & (np.abs(vals) <= O8.LARGEST[fmt])]
    assert np.array_equal(O8.round_code(vals, fmt), vals)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_exponent_is_the_smallest_that_fits(fmt):
    big = O8.LARGEST[fmt]
    for top in (1e-3, 1.0, big, np.nextafter(big, 1e9), big * 2, 2.9e38, 447.0, 126.5):
        e = O8.exponent(np.array([top, -top / 3]), fmt)
        assert top <= big * 2.0 ** e and (top > big * 2.0 ** (e - 1))
    # the largest finite values saturate at F 2^e, which fp32 and bf16 hold
    top = float(np.finfo(np.float32).max)
    assert O8.exponent(np.array([top]), fmt) == O8.E_MAX[fmt] and np.isfinite(np.float32(big * 2.0 ** O8.E_MAX[fmt]))
    val, _ = O8.quantise(np.full((16, 4), top), fmt)
    assert np.all(val == big * 2.0 ** O8.E_MAX[fmt])
    assert O8.exponent(np.zeros(4), fmt) == O8.E_MIN
    assert O8.exponent(np.array([1e-38, 0]), fmt) == O8.E_MIN
    assert O8.exponent(np.array([np.inf, np.nan, 1.0]), fmt) == O8.exponent(np.array([1.0]), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_one_write_is_within_half_a_step_and_growth_within_one(fmt):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(48, 64)) * np.exp(rng.normal(size=(48, 1)))

    def step(e, v):
        if fmt == "int8":
            return np.full_like(v, 2.0 ** e)
        k = np.floor(np.log2(np.maximum(np.abs(v) / 2.0 ** e, 2.0 ** -6)))
        return 2.0 ** (k - 3) * 2.0 ** e
    val, ex = O8.quantise(x, fmt)
    per_row = np.repeat(ex, 16)[:, None].astype(np.float64)
    assert np.all(np.abs(val - x) <= 0.5 * step(per_row, x) * (1 + 1e-12))
    one, e1 = np.zeros((48, 64)), np.full(3, O8.E_MIN)
    for t in range(48):
        one, e1 = O8.append(one, e1, t, x[t:t + 1], fmt)
    assert np.array_equal(e1, ex)          # the same scales however the rows came
    assert np.all(np.abs(one - x) <= step(per_row, x) * (1 + 1e-12))


def test_cache_helper_and_null_context():
    cfg = TB.make_config(1, 2, 8, 2, 64, 16, 1, 512, "bf16", 30, 4, 16)
    k, v, ks, vs = TB.kv8_cache(cfg, "e4m3", device="cpu")
    assert k.shape == v.shape == (2, 2, 512, 64) and k.dtype == torch.float8_e4m3fn
    assert ks.shape == vs.shape == (2, 2, 32) and ks.dtype == torch.float32
    assert TB.kv8_cache(cfg, "int8", device="cpu")[0].dtype == torch.int8
    with pytest.raises(ValueError):
        TB.kv8_cache(cfg, "e5m2", device="cpu")
    L = TB.lib()
    assert L.tb_bind_layer_kv8(None, 0, 1, None, None, None, None, None, None) == 1
    assert L.tb_bind_layer_kv8_paged(None, 0, 1, None, None, None, None, 1, None, 64, 1, None, None) == 1
    assert L.tb_append_kv_rows(None, 0, None, None, None, None, None, None) == 1
    assert L.tb_read_kv(None, 0, 0, 1, None, None, None) == 1
