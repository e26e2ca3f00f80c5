"""Which form of the dense layer with bias takes a size (host only)."""
import random

import pytest

import block_causal_attention_wave_b200 as wave
from dense_forms import FORMS, LONG, PAIRS, SMS, TILES, TOKENS, form_of


def test_the_sizes_reach_their_forms():
    lib = wave.load()
    for table in (FORMS, {f: [s] for f, s in LONG.items()}):
        for form, sizes in table.items():
            assert [form_of(lib, *s) for s in sizes] == [form] * len(sizes), (form, sizes)


def test_every_form_that_a_size_takes_is_listed():
    """Sizes spread over the logarithm of M, K and N: no form but those of the list."""
    lib, rng = wave.load(), random.Random(1)
    seen = set()
    for _ in range(60000):
        M, K, N = (int(2 ** rng.uniform(0, 13)) for _ in range(3))
        seen.add(form_of(lib, M, 8 * K, 8 * N))
    assert {f for f in seen if f[0] != TOKENS} <= set(FORMS)
    assert {f for f in seen if f[0] == TOKENS} == {(TOKENS, 8, 8), (TOKENS, 8, 16), (TOKENS, 16, 8)}


@pytest.mark.parametrize("sms", [1, 20, 74, 132, SMS])
def test_a_form_fits_its_size(sms):
    """On any number of SMs K is cut into no more parts than it has slices of 128, and a
    cluster has at most eight CTAs."""
    lib, rng = wave.load(), random.Random(2)
    for _ in range(5000):
        M, K, N = int(2 ** rng.uniform(0, 20)), 8 * int(2 ** rng.uniform(0, 13)), 8 * int(2 ** rng.uniform(0, 13))
        kind, cols, parts = form_of(lib, M, K, N, sms)
        if kind == TOKENS:
            assert M <= 16 and (cols, parts) in ((8, 8), (8, 16), (16, 8)) and (parts == 8 or M <= 8)
        else:
            assert 1 <= parts <= (8 if kind == TILES else 4) and parts <= (K + 127) // 128
            assert cols in ((64, 128) if kind == TILES else (192, 256)), kind
            assert kind in (TILES, PAIRS)
