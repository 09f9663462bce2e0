"""Planted mistakes in the 8-bit-moment oracle: each must fail one of its pins (CPU only)."""
import numpy as np
import pytest

import oracle
import test_oracle_state8 as pins
from oracle import state8

ENCODE, WORDS, DECODE = state8.encode, state8.words, state8.decode


def _pins():
    yield pins.test_decode_matches_torch_for_every_code_and_scale
    for power in (-130, 0, 100):
        yield lambda power=power: pins.test_nearest_codes_match_torchs_conversion(power)
    yield pins.test_codes_survive_a_round_trip
    for value in (1.03, 0.37, 3.3e-3):
        yield lambda value=value: pins.test_stochastic_rounding_is_unbiased_over_all_draws(value)
    yield pins.test_zeros_positive_minimum_and_non_finite_blocks
    yield pins.test_words_match_a_pure_python_count
    yield lambda: pins.test_words_are_uniform_and_uncorrelated(0.3)
    yield pins.test_step_on_exact_states_equals_the_32_bit_step
    yield pins.test_windows_round_as_the_whole


def _some_pin_fails():
    for pin in _pins():
        try:
            pin()
        except AssertionError:
            return True
    return False


def _raise_codes(x, second, draw=None):
    codes, scales = ENCODE(x, second, draw)
    return np.where((codes & 0x7F) < 0x70, codes + 1, codes).astype(np.uint8), scales


def _scale_up(x, second, draw=None):
    codes, scales = ENCODE(x, second, draw)
    return codes, np.where((scales > 0) & (scales < 250), scales + 1, scales).astype(np.uint8)


def _plain_step(*args, seed=0, first_element=0, **kw):
    """Windows numbered from zero instead of their place."""
    return STEP(*args, seed=seed, first_element=0, **kw)


STEP = state8.adamw8_step
MISTAKES = {
    "nearest in place of stochastic": ("encode", lambda x, second, draw=None: ENCODE(x, second)),
    "the draw unused (cut)": ("encode", lambda x, second, draw=None: ENCODE(
        x, second, None if draw is None else np.zeros_like(draw))),
    "a code too high": ("encode", _raise_codes),
    "a scale too high": ("encode", _scale_up),
    "no least code for a positive second moment": ("encode", lambda x, second, draw=None: ENCODE(x, False, draw)),
    "the sign dropped": ("encode", lambda x, second, draw=None: ENCODE(np.abs(x), second, draw)),
    "non-finite blocks kept": ("encode", lambda x, second, draw=None: ENCODE(np.nan_to_num(x), second, draw)),
    "words of a constant step": ("words", lambda n, first, seed, step: WORDS(n, first, seed, 1)),
    "words of a constant seed": ("words", lambda n, first, seed, step: WORDS(n, first, 0, step)),
    "one word per group": ("words", lambda n, first, seed, step: WORDS(n // 8 * 8 + 8, first, seed, step)[
        np.arange(n) // 8 * 8]),
    "words without the place": ("words", lambda n, first, seed, step: WORDS(n, 0, seed, step)),
    "decode a power too high": ("decode", lambda codes, scales: DECODE(codes, scales) * np.float32(2)),
    "decode without NaN blocks": ("decode", lambda codes, scales: np.nan_to_num(DECODE(codes, scales))),
    "windows numbered from zero": ("adamw8_step", _plain_step),
}


@pytest.mark.parametrize("mistake", sorted(MISTAKES))
def test_each_mistake_fails_a_pin(mistake, monkeypatch):
    name, wrong = MISTAKES[mistake]
    monkeypatch.setattr(state8, name, wrong)
    if name == "adamw8_step":
        monkeypatch.setattr(oracle, "adamw8_step", wrong)
    assert _some_pin_fails(), mistake


def test_the_oracle_passes_the_same_pins():
    assert not _some_pin_fails()
