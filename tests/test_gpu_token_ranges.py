"""The single-token operators at the ends of their ranges: the largest tables, offsets
past 32 bits, runs long enough for each kernel's own form of them, and first calls
made inside a capture.

Tolerances as in test_gpu_token.py, against 64-bit results; pages bit for bit.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import block as oblock
from oracle import quant
from oracle import token as otok
from test_gpu_token import FORMATS, U, _World, _bf, _cache, _dev, _pages, _within
from wave_testlib import torch_to_f64

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- rotation
def _rotated(x, pos, layout, ladder, inverse):
    """64 bits, on the GPU: x [rows][heads][d] turned by pos [rows][3]."""
    import torch
    d = x.shape[-1]
    axis, freq = otok.frequencies(d, oblock.rope_groups(d), 10000.0, ladder)
    angle = pos.double()[:, torch.from_numpy(axis).cuda()] * torch.from_numpy(freq).cuda()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if inverse else 1)
    x = x.double()
    if layout == "halves":
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _check_rotated(got, x, ref, what):
    tol = U * ref.abs() + 2.0 ** -20 * 2 * x.double().abs().amax(-1, keepdim=True)
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, the first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("rows,qh,kh", [(3001, 5, 3), (20011, 12, 12), (2500, 24, 24), (9000, 1, 2), (70001, 1, 1),
                                        (37, 64, 8)])
def test_rotary_long(cuda_lib, d, layout, rows, qh, kh):
    """Rows enough that a thread takes several heads, in whole batches and less, across the
    border of Q and K; read from a packed projection, out of place and in place."""
    import torch
    kv = _cache(cuda_lib, d=d)
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    packed = torch.randn(rows, (qh + 2 * kh) * d, generator=gen, device="cuda").bfloat16()
    Q = packed[:, :qh * d].unflatten(1, (qh, d))
    K = packed[:, qh * d:(qh + kh) * d].unflatten(1, (kh, d))
    pos = torch.randint(0, 300, (rows, 3), generator=gen, device="cuda", dtype=torch.int32)
    ref = [_rotated(x, pos, layout, "ladder", True) for x in (Q, K)]
    Qo, Ko = (torch.full((rows + 2, x.shape[1], d), 7.0, dtype=torch.bfloat16, device="cuda") for x in (Q, K))
    kv.rotary(pos, Q, K, Qo[1:-1], Ko[1:-1], layout=layout, ladder="ladder", inverse=True)
    for got, x, want in ((Qo, Q, ref[0]), (Ko, K, ref[1])):
        _check_rotated(got[1:-1], x, want, f"{rows} rows, {qh} + {kh} heads")
        assert (got[0] == 7).all() and (got[-1] == 7).all()
    before = packed.clone()
    kv.rotary(pos, Q, K, layout=layout, ladder="ladder", inverse=True)
    assert torch.equal(Q, Qo[1:-1]) and torch.equal(K, Ko[1:-1])
    assert torch.equal(packed[:, (qh + kh) * d:], before[:, (qh + kh) * d:])


def test_rotary_rows_far_apart(cuda_lib):
    """Row strides that pass 2^32 elements from the first row to the last."""
    import torch
    rows, d, ld = 3, 64, 8 * (1 << 28) + 8
    kv = _cache(cuda_lib, d=d)
    big = torch.empty(2 * ld + 2 * d, dtype=torch.bfloat16, device="cuda")
    Q = torch.as_strided(big, (rows, 1, d), (ld, d, 1))
    K = torch.as_strided(big, (rows, 1, d), (ld, d, 1), d)
    x = torch.randn(2, rows, 1, d, device="cuda").bfloat16()
    Q.copy_(x[0])
    K.copy_(x[1])
    pos = torch.tensor([[1, 2, 3], [4, 5, 6], [7, 8, 9]], dtype=torch.int32, device="cuda")
    kv.rotary(pos, Q, K)
    _check_rotated(Q, x[0], _rotated(x[0], pos, "interleaved", "axis", False), "Q")
    _check_rotated(K, x[1], _rotated(x[1], pos, "interleaved", "axis", False), "K")


# -------------------------------------------------------------- dense layer
@pytest.mark.parametrize("M,K,N", [(70000, 16, 65536), (70000, 72, 32776), (65600, 65536, 8), (1, 65536, 65536),
                                   (16, 65536, 32776), (40, 65536, 65536)])
def test_linear_past_32_bits(cuda_lib, M, K, N):
    """Outputs, activations and weights of more than 2^31 elements: rows all along the
    layer against 64 bits."""
    import torch
    kv = _cache(cuda_lib)
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    A = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    W = torch.empty(N, K, dtype=torch.bfloat16, device="cuda").normal_(0, K ** -0.5, generator=gen)
    bias = torch.empty(N, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    kv.linear_bias(A, W, Y, bias=bias)
    kv.status()
    assert not torch.isnan(Y).any()
    at = torch.linspace(0, M - 1, min(M, 64), device="cuda").long()
    cols = torch.unique(torch.linspace(0, N - 1, min(N, 2048), device="cuda").long())
    a, w = A[at].double(), W[cols].double()
    ref = a @ w.T + bias[cols].double()
    size = a.abs() @ w.abs().T + bias[cols].double().abs()
    bad = ~((Y[at][:, cols].double() - ref).abs() <= U * ref.abs() + (2 * K + 16) * 2.0 ** -23 * size)
    assert not bad.any(), f"{int(bad.sum())} off, the first at {bad.nonzero()[0].tolist()}"


# ------------------------------------------------------------- token writes
@FORMATS
@pytest.mark.parametrize("entries,tokens,heads", [(12, 300, 2), (3, 4680, 12), (64, 130, 1), (2, 9000, 3)])
def test_write_long(cuda_lib, fp8, entries, tokens, heads):
    """More entries or pages than the small tables hold, and tiles enough for the long
    writes' kernel: from the middle of a page, in two pieces, of a packed projection."""
    import torch
    d, per = 64 if tokens == 300 else 128, -(-tokens // 128)
    kv = _cache(cuda_lib, heads, d, tokens, 1, pages=entries * per, fp8=fp8, fill=0xFF)
    rng = np.random.default_rng(entries)
    x = oblock.bf16_round(rng.standard_normal((2, entries, tokens, heads, d)) *
                          np.exp(rng.standard_normal((2, entries, tokens, 1, 1))))
    nodes = [(c, 1) for c in range(entries)]
    for n in nodes:
        kv.alloc(*n)
    cut = [1 + (37 * c) % (tokens - 1) for c in range(entries)]
    for first, count in (([0] * entries, cut), (cut, [tokens - n for n in cut])):
        rows = [np.concatenate([x[i, c, f:f + n] for c, (f, n) in enumerate(zip(first, count))]) for i in range(2)]
        packed = _dev(np.stack([np.zeros_like(rows[0]), *rows], 1))
        kv.write_tokens(nodes, first, packed[:, 1], packed[:, 2], count)
    kv.status()
    for c, n in enumerate(nodes):
        if fp8:
            codes, scales = _pages(kv, n)
            for i in range(2):
                ent = otok.Fp8Entry(tokens, heads, d)
                ent.write(0, x[i, c, :cut[c]])
                ent.write(cut[c], x[i, c, cut[c]:])
                assert np.array_equal(scales[i], ent.scales), n
                assert np.array_equal(quant.e4m3_decode(codes[i]), quant.e4m3_decode(ent.codes)), n
        else:
            want = np.zeros((2, per * 128, heads, d), dtype=np.uint16)
            want[:, :tokens] = (x[:, c].astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
            want = want.reshape(2, per, 128, heads, d).transpose(0, 1, 3, 2, 4)
            assert np.array_equal(_pages(kv, n), want), n


# ---------------------------------------------------------- token attention
def test_token_attn_full_table(cuda_lib):
    """As many pages as a call takes, right; one more, refused."""
    import torch
    most = 5120
    w = _World(cuda_lib, 1, 64, 128 * 20, 1, pages=most + 20, seed=31)
    k, v = (_bf(w.rng, 128 * 20, 1, 64) for _ in range(2))
    K, V = _dev(k), _dev(v)
    for c in range(most // 20 + 1):
        w.kv.append(c, 1, K, V)
        w.entries[c, 1] = (k, v)
    last = most // 20
    w.check([(last - 1, 1)], "same", what="5120 pages")
    w.check([(last, 1)], "same", own=[0], what="5120 pages and no own token")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cuda_lib.WaveError) as e:
        w.kv.token_attn([(last, 1)], "same", q, q.clone(), own_tokens=[1])
    assert e.value.code == -7


@FORMATS
def test_token_attn_most_queries(cuda_lib, fp8):
    """64 queries with a row stride each, every count around a page's edges, all groups of rows."""
    w = _World(cuda_lib, 2, 128, 300, 1, prefix=3, fp8=fp8, seed=32)
    for c in range(2):
        w.add(c, 1)
    own = [(5 * i + 100) % 301 for i in range(64)]
    for group in (1, 3, 8):
        w.check([(1, 1)] * 64, "same", own=own, group=group, strided=True, what=f"group {group}")


def test_token_attn_rows_far_apart(cuda_lib):
    """Queries and results whose strides pass 2^32 elements."""
    import torch
    w = _World(cuda_lib, 1, 64, 100, 1, seed=33)
    w.add(0, 1)
    ld = 8 * (1 << 28) + 8
    big = torch.empty(2 * ld + 128, dtype=torch.bfloat16, device="cuda")
    Q = torch.as_strided(big, (3, 1, 64), (ld, 64, 1))
    O = torch.as_strided(big, (3, 1, 64), (ld, 64, 1), 64)
    q = _bf(w.rng, 3, 1, 64)
    Q.copy_(_dev(q))
    nodes, own = [(0, 1)] * 3, [100, 64, 7]
    w.kv.token_attn(nodes, "same", Q, O, own_tokens=own)
    w.kv.status()
    for i, n in enumerate(own):
        o, _, a = otok.token_attention(q[i], *(x[:n] for x in w.entries[0, 1]))
        _within(torch_to_f64(O)[i], o, U * np.abs(o) + 2.0 ** -12 * a, f"row {i}")


# ------------------------------------------------------------- first calls
_FIRST = """
import sys
import torch
import block_causal_attention_wave_b200 as wave
fp8 = sys.argv[1] == "fp8"
H, d, T = 2, 128, 300
fmt = wave.KV_FP8_E4M3 if fp8 else wave.KV_BF16
pool = torch.zeros(4096 + 20 * (wave.KVCache.page_bytes(H, d, fmt) + 64) + 512, dtype=torch.uint8, device="cuda")
kv = wave.KVCache(H, d, T, 1, pool=pool, kv_format=fmt)
kv.alloc(0, 1)
gen = torch.Generator(device="cuda").manual_seed(1)
X = torch.randn(T, 256, generator=gen, device="cuda").bfloat16()
W = (torch.randn(256, 256, generator=gen, device="cuda") / 16).bfloat16()
Y, O, L = torch.empty_like(X), torch.empty(1, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(X[:1])
pos = torch.arange(3 * T, dtype=torch.int32, device="cuda").view(T, 3)
ws = torch.empty(max(1, kv.token_attn_workspace([(0, 1)], "same")), dtype=torch.uint8, device="cuda")
def step():
    kv.linear_bias(X, W, Y)
    kv.rotary(pos, Y.view(T, H, d))
    kv.write_tokens([(0, 1)], [0], Y.view(T, H, d), X.view(T, H, d), [T])
    kv.token_attn([(0, 1)], "same", Y[:1].view(1, H, d), O, workspace=ws)
    kv.linear_bias(O.view(1, 256), W, L)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = Y.clone(), O.clone(), L.clone()
Y.zero_(), O.zero_(), L.zero_()
step()
kv.status()
assert all(torch.equal(a, b) for a, b in zip(got, (Y, O, L))) and torch.isfinite(L).all() and L.any()
print("captured")
"""


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_first_calls_inside_a_capture(cuda_lib, fmt):
    """A process whose first calls of the operators are captured ones."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST, fmt], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_write_fp8_of_nan_and_infinity(cuda_lib):
    """A NaN is kept and leaves the scale to the others; an infinity takes its page and
    head with it until it is rewritten, and no other page or head."""
    import torch
    H, d, T = 2, 64, 200
    kv = _cache(cuda_lib, H, d, T, 1, pages=2, fp8=True, fill=0xFF)
    kv.alloc(0, 1)
    x = torch.randn(T, H, d, device="cuda").bfloat16()

    def read():
        codes, scales = _pages(kv, (0, 1))
        with np.errstate(invalid="ignore"):
            v = quant.e4m3_decode(codes) * scales[..., None, None].astype(np.float64)
        return v.transpose(0, 1, 3, 2, 4).reshape(2, -1, H, d)[:, :T], scales   # [K, V][token][head][d]
    kv.write_tokens([(0, 1)], [0], x, x, [T])
    before, scales = read()
    y = x[:1].clone()
    y[0, 0, 5] = float("nan")
    kv.write_tokens([(0, 1)], [0], y, x[:1])
    got, again = read()
    assert np.isnan(got[0, 0, 0, 5]) and np.isnan(got).sum() == 1
    got[0, 0, 0, 5] = before[0, 0, 0, 5]
    assert np.array_equal(scales, again) and np.array_equal(got, before)
    y[0, 0, 5] = float("inf")
    kv.write_tokens([(0, 1)], [0], y, x[:1])
    got, _ = read()
    gone = np.zeros(got.shape, dtype=bool)
    gone[0, :128, 0] = True
    assert np.isnan(got[gone]).all() and np.array_equal(got[~gone], before[~gone])
    kv.write_tokens([(0, 1)], [0], x[:1], x[:1])
    got, _ = read()
    gone[0, 0] = False
    assert (got[gone] == 0).all() and np.array_equal(got[0, 128:], before[0, 128:])
    assert (np.abs(got[0, 0] - torch_to_f64(x[0])) <= 2.0 ** -4 * np.abs(torch_to_f64(x[0])) + 2.0 ** -16).all()   # half steps; s < 2^-6


def test_token_attn_far_chunk(cuda_lib):
    """A query of a chunk whose history the cache cannot hold is refused at once; a
    window makes it an ordinary one."""
    import resource
    import torch
    far = 2 ** 31 - 1
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    w = _World(cuda_lib, 1, 64, 100, 1, seed=41)
    w.add(far, 1)
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    for call in (lambda: w.kv.token_attn([(far, 1)], "same", q, q.clone()),
                 lambda: w.kv.token_attn_workspace([(far, 1)], "same")):
        with pytest.raises(cuda_lib.WaveError) as e:
            call()
        assert e.value.code == -2
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 1 << 18  # KB
    w = _World(cuda_lib, 1, 64, 100, 1, window=1, seed=42)
    w.add(far, 1)
    w.add(far - 1, 1)
    w.check([(far, 1)], "same", what="far chunk")
