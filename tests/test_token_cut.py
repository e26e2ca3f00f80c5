"""How token attention cuts its lists over a GPU's SMs (host only)."""
import ctypes

import pytest

import block_causal_attention_wave_b200 as wave


def _cut(sms, lists, longest):
    out = (ctypes.c_int32 * 2)()
    wave.load().wavei_token_cut(ctypes.c_int32(sms), ctypes.c_int64(lists), ctypes.c_int32(longest), out)
    return out[0], out[1]


@pytest.mark.parametrize("lists,longest,cut", [(24, 5, (5, 1)), (12, 259, (8, 1)), (1, 1517, (8, 15)), (3, 400, (8, 5)),
                                               (148, 7, (1, 1)), (1, 1, (1, 1)), (1, 0, (1, 1))])
def test_on_148_sms(lists, longest, cut):
    assert _cut(148, lists, longest) == cut


@pytest.mark.parametrize("sms", [8, 16, 37, 74, 110, 132, 148])
def test_few_lists_fill_the_sms_once(sms):
    """Fewer than eight long lists are cut into as many clusters of eight as the GPU holds
    at a time, not into those of a larger GPU, which would run in a second wave."""
    for lists in range(1, 8):
        for longest in (128, 700, 5000):
            cluster, parts = _cut(sms, lists, longest)
            held = max(1, 15 * sms // 148)
            assert cluster == 8 and parts >= 1 and parts <= max(1, longest // 64)
            assert parts == 1 or lists * parts <= held


@pytest.mark.parametrize("sms", [37, 74, 148])
def test_one_wave_where_one_suffices(sms):
    """As many lists as SMs: a CTA each."""
    assert _cut(sms, sms, 64) == (1, 1)
    assert _cut(sms, sms // 2, 64)[0] <= 2
