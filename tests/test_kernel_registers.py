"""A kernel's register count: a query that fails is reported and not kept."""
import ctypes

import block_causal_attention_wave_b200 as wave


def test_a_failed_query_is_not_kept():
    lib = wave.load()
    known, regs = ctypes.c_int32(0), ctypes.c_int32(-1)
    not_a_kernel = ctypes.cast(lib.wave_strerror, ctypes.c_void_p)
    for _ in range(2):
        assert lib.wavei_kernel_registers(not_a_kernel, ctypes.byref(known), ctypes.byref(regs)) == -4
        assert known.value == 0 and b"cudaFuncGetAttributes" in lib.wave_last_error_detail()
    known.value = 128  # what a query has found is not asked for again
    assert lib.wavei_kernel_registers(not_a_kernel, ctypes.byref(known), ctypes.byref(regs)) == 0
    assert regs.value == 128
