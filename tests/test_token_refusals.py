"""What the single-token calls refuse: every bad argument at the C boundary, on
the CPU (tests/c/token_check.cpp), and the tensors that the binding refuses."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "block_causal_attention_wave_b200")


def _check(tmp_path, gpu):
    if not os.path.exists(os.path.join(LIBDIR, "libwave.so")):
        pytest.skip("libwave.so not built")
    exe = tmp_path / "token_check"
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cmd = ["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(LIBDIR, "csrc"), "-I", cuda_inc,
           os.path.join(ROOT, "tests", "c", "token_check.cpp"),
           "-L", LIBDIR, "-lwave", f"-Wl,-rpath,{LIBDIR}", "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe), "1" if gpu else "0"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("ok ") >= 100


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_refusals_without_a_gpu(tmp_path):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; the gpu-marked variant covers this")
    _check(tmp_path, gpu=False)


@pytest.mark.gpu
def test_refusals_with_a_gpu(tmp_path):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device in this process")
    _check(tmp_path, gpu=True)


def test_host_only_handles_refuse():
    import torch
    import block_causal_attention_wave_b200 as wave
    kv = wave.KVCache(2, 64, 200, 2, pool_bytes=1 << 20)
    t = torch.zeros(2, 128, dtype=torch.bfloat16)
    for call in (lambda: kv.linear_bias(t, t, t), lambda: kv.rotary(None, t.view(2, 2, 64)),
                 lambda: kv.write_tokens([(0, 1)], [0], t, t), lambda: kv.token_attn([], "same", t, t),
                 lambda: kv.token_attn_workspace([(0, 1)], "same")):
        with pytest.raises(wave.WaveError) as e:
            call()
        assert e.value.code == -1


@pytest.mark.gpu
def test_binding_refuses_tensors_a_kernel_would_misread(cuda_lib):
    import torch
    wave = cuda_lib
    H, d = 2, 64
    pool = torch.zeros(4096 + 4 * wave.KVCache.page_bytes(H, d), dtype=torch.uint8, device="cuda")
    kv = wave.KVCache(H, d, 100, 1, pool=pool)
    kv.alloc(0, 1)
    z = lambda *s, dtype=torch.bfloat16, device="cuda": torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
    q, pos = z(3, H, d), z(3, 3, dtype=torch.int32)
    bad = [
        lambda: kv.linear_bias(z(3, 64, dtype=torch.float16), z(8, 64), z(3, 8)),
        lambda: kv.linear_bias(z(3, 64, device="cpu"), z(8, 64), z(3, 8)),
        lambda: kv.linear_bias(z(3, 64), z(8, 72), z(3, 8)),
        lambda: kv.linear_bias(z(3, 64), z(8, 64), z(2, 8)),
        lambda: kv.linear_bias(z(3, 64), z(8, 128)[:, :64], z(3, 8)),
        lambda: kv.linear_bias(z(64, 3).t(), z(8, 64), z(3, 8)),
        lambda: kv.linear_bias(z(3, 64), z(8, 64), z(3, 8), bias=z(7)),
        lambda: kv.linear_bias(z(3, 64), z(8, 64), z(3, 8), R=z(3, 16)),
        lambda: kv.rotary(z(3, 3, dtype=torch.int64), q),
        lambda: kv.rotary(z(2, 3, dtype=torch.int32), q),
        lambda: kv.rotary(z(3, 4, dtype=torch.int32)[:, :3], q),
        lambda: kv.rotary(pos, z(3, H, 32)),
        lambda: kv.rotary(pos, q, z(2, H, d)),
        lambda: kv.rotary(pos, z(3, d, H).transpose(1, 2)),
        lambda: kv.write_tokens([(0, 1)], [0], z(2, H, d), z(1, H, d)),
        lambda: kv.write_tokens([(0, 1)], [0, 1], z(1, H, d), z(1, H, d)),
        lambda: kv.write_tokens([(0, 1)], [0], z(1, H, d, dtype=torch.float32), z(1, H, d)),
        lambda: kv.token_attn([(0, 1)], "same", q, z(1, H, d)),
        lambda: kv.token_attn([(0, 1)], "same", z(1, H, d), z(1, H, d), lse=z(1, H)),
        lambda: kv.token_attn([(0, 1)], "same", z(1, H, d), z(1, H, d), own_tokens=[1, 2]),
        lambda: kv.token_attn([(0, 1)], "same", z(1, H, d), z(1, H, d), workspace=z(999, device="cpu")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    kv.status()
