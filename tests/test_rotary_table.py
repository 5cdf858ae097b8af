"""Rotary tables on the CPU: every frequency of the banded scaling, and what has no table."""
import math

import numpy as np
import pytest

from speculative_decoding_specdec_gb300.engine import rotary_table


@pytest.mark.parametrize("rot,base,factor,original,fast,slow", [
    (128, 1e6, 4.0, 32768, 32.0, 1.0), (64, 1e4, 8.0, 2048, 32.0, 1.0)])
def test_bands_ramp_with_the_turns_within_the_trained_length(rot, base, factor, original, fast, slow):
    """gamma(r) = (r - slow) / (fast - slow), cut to [0, 1], of r = original / wavelength keeps that
    part of a frequency and divides the rest by the factor."""
    got = rotary_table(40, rot, base=base, scaling="bands", factor=factor, original=original,
                       beta_fast=fast, beta_slow=slow, device="cpu").double().numpy()
    amp, inside = 0.1 * math.log(factor) + 1, 0
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        r = original / (2 * math.pi / f)
        g = min(1.0, max(0.0, (r - slow) / (fast - slow)))
        inside += 0 < g < 1
        f = g * f + (1 - g) * f / factor
        np.testing.assert_allclose(got[:, i, 0], amp * np.cos(np.arange(40) * f), atol=2e-7)
        np.testing.assert_allclose(got[:, i, 1], amp * np.sin(np.arange(40) * f), atol=2e-7)
    assert inside > 0


@pytest.mark.parametrize("bad", [
    dict(scaling="bands", original=64, beta_fast=1.0, beta_slow=1.0),    # no ramp between
    dict(scaling="bands", original=64, beta_fast=1.0, beta_slow=32.0),
    dict(scaling="base", rot_dim=2),                                     # one frequency, always 1
    dict(scaling="bands", original=64, beta_fast=float("nan"))])
def test_settings_without_a_table_are_refused(bad):
    with pytest.raises(ValueError):
        rotary_table(**({"positions": 4, "rot_dim": 8, "factor": 4.0, "device": "cpu"} | bad))
