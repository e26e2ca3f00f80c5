"""A node whose history is longer than the cache: refused at once, without a list of
as many entries as its chunk's number."""
import resource

import pytest

import block_causal_attention_wave_b200 as wave

FAR = 2 ** 31 - 1


@pytest.mark.parametrize("policy", ["clean", "same", "progressive"])
def test_far_chunk_is_refused_at_once(policy):
    kv = wave.KVCache(1, 64, 128, 2, pool_bytes=1 << 20)
    for c in range(FAR - 3, FAR):
        for level in range(3):
            kv.alloc(c, level)
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    with pytest.raises(wave.WaveError) as e:
        kv.gather_table([(FAR, 1)], policy)
    assert e.value.code == -2
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 1 << 18  # KB
    with_window = wave.KVCache(1, 64, 128, 2, window=2, pool_bytes=1 << 20)
    for c in range(FAR - 2, FAR + 1):
        for level in range(3):
            with_window.alloc(c, level)
    assert [len(r) for r in with_window.gather_table([(FAR, 1)], policy)] == [3]


def test_the_missing_entry_is_named():
    kv = wave.KVCache(1, 64, 128, 1, pool_bytes=1 << 20)
    for c in range(1, 4):
        kv.alloc(c, 1)
    for node, missing in (((3, 1), "(0, 1)"), ((9, 1), "(0, 1)"), ((4, 1), "(0, 1)")):
        with pytest.raises(wave.WaveError) as e:
            kv.gather_table([node], "same")
        assert e.value.code == -2 and missing in str(e.value)
    kv.alloc(0, 1)
    with pytest.raises(wave.WaveError) as e:
        kv.gather_table([(9, 1)], "same")
    assert "(4, 1)" in str(e.value)
