"""The 8-bit steps' random words over distance: each window of 2^28 elements has
a key of its own, and the draws of elements far apart are independent."""
import numpy as np
import pytest

import oracle
from oracle import state8

WORDS = state8.words
M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def _word(e, seed, step):
    """One word from the definition, in Python integers."""
    w, q, j = e >> 28, (e & (1 << 28) - 1) >> 3, e & 7
    z = (seed + step * 0x6A09E667F3BCC909 + w * 0xA54FF53A5F1D36F1) & M64
    z = (z ^ z >> 32) * 0xBB67AE8584CAA73B & M64
    z = (z ^ z >> 29) * 0x3C6EF372FE94F82B & M64
    z ^= z >> 32
    a = ((q ^ (z & M32)) * 0xA54FF53B) & M32
    a ^= a >> 16
    a = ((a + (z >> 32)) * 0x510E527F) & M32
    a ^= a >> 15
    b = a * 0x9B05688D & M32
    b = (b ^ b >> 16) | 1
    return (a + j * b) & M32


@pytest.mark.parametrize("first", [0, (1 << 28) - 140, (1 << 28), (5 << 28) - 3, (1 << 36) + 12_345, (1 << 62) - 150])
def test_words_of_the_definition(first):
    for seed, step in ((0, 1), ((1 << 64) - 1, 7), (3, 1 << 40)):
        got = state8.element_words(300, first, seed, step)
        assert got.tolist() == [_word(first + i, seed, step) for i in range(300)]


def test_the_first_window_has_the_step_stream():
    """Elements below 2^28 keep the words of one stream per step."""
    for first in (0, 128, (1 << 28) - 256):
        assert np.array_equal(state8.element_words(256, first, 9, 4), state8.words(256, first, 9, 4))


def _events(w, p=0.3):
    cut = (1 - p) * 2 ** 20
    return np.stack([w >> 12, w & 0xFFFFF]) >= cut, round(p * 2 ** 20) / 2 ** 20


@pytest.mark.parametrize("k", range(3, 41))
def test_far_elements_round_independently(k):
    """The joint rate of rounding up at e and e + 2^k, over 2^15 elements of a step: within 5 standard deviations
    of the product of the rates, in both draws and three steps."""
    n = 1 << 15
    for step in (1, 2, 77):
        (a, q), (b, _) = (_events(state8.element_words(n, first, 99, step)) for first in (0, 1 << k))
        bound = 5 * np.sqrt(q * q / n * (1 + 4 * q))
        assert (abs((a & b).mean(axis=1) - q * q) < bound).all(), (step, (a & b).mean(axis=1))


def test_one_far_pair_differs_by_no_constant():
    """One pair of elements 2^k apart over 1,024 steps: its draws' correlation within 5 standard deviations
    (5 / 32), and the difference modulo 1 in no 64th more often than 16 + 6 * 4 times (a Poisson count of mean 16
    passes 40 with a probability of 1e-7)."""
    steps = 1024
    for e in (0, 12_345 * 8 + 3):
        for k in (28, 29, 30, 31, 32, 33, 34, 35, 36, 40):
            w = np.array([[state8.element_words(1, at, 5, t)[0] for at in (e, e + (1 << k))]
                          for t in range(1, steps + 1)]).astype(np.int64)
            for draw in (w >> 12, w & 0xFFFFF):
                x, y = draw.T
                assert abs(np.corrcoef(x, y)[0, 1]) < 5 / np.sqrt(steps), (e, k)
                assert np.bincount(((x - y) % (1 << 20)) >> 14, minlength=64).max() <= 40, (e, k)


def test_a_step_across_a_border_rounds_as_its_two_parts():
    rng = np.random.default_rng(1)
    n, cut = 128 * 6 + 17, 128 * 2
    first = (1 << 28) - cut
    p = rng.standard_normal(n).astype(np.float32)
    g = oracle.f32_to_bf16(rng.standard_normal(n).astype(np.float32))
    m, ms = state8.encode(rng.standard_normal(n).astype(np.float32), False)
    v, vs = state8.encode(np.abs(rng.standard_normal(n)).astype(np.float32), True)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    whole = oracle.adamw8_step(p, m, ms, v, vs, g, 9, seed=8, first_element=first, **hp)
    for a, b in ((0, cut), (cut, n)):
        part = oracle.adamw8_step(p[a:b], m[a:b], ms[a // 128:-(-b // 128)], v[a:b], vs[a // 128:-(-b // 128)], g[a:b],
                                  9, seed=8, first_element=first + a, **hp)
        for x, y, s in zip(whole, part, (1, 1, 128, 1, 128, 1)):
            assert np.array_equal(x[a // s:-(-b // s)], y)


STATISTICAL = {
    "one key for all elements": lambda n, first, seed, step: WORDS(n, first, seed, step),
    "windows with one key": lambda n, first, seed, step: WORDS(n, first % (1 << 28), seed, step),
}
MISTAKES = dict(STATISTICAL, **{
    "keys other than the definition's": lambda n, first, seed, step: WORDS(
        n, first % (1 << 28), (seed + (first >> 28)) & M64, step)})


def _fails(pin):
    try:
        pin()
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("mistake", sorted(MISTAKES))
def test_each_mistake_fails_its_pins(mistake, monkeypatch):
    monkeypatch.setattr(state8, "element_words", MISTAKES[mistake])
    assert _fails(lambda: test_words_of_the_definition(1 << 28))
    if mistake in STATISTICAL:
        assert _fails(test_one_far_pair_differs_by_no_constant)
        assert any(_fails(lambda k=k: test_far_elements_round_independently(k)) for k in (28, 31, 33, 35))
