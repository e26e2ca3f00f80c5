"""GPU parity of the single-token operators against the float64 oracle: the
dense layer with bias, rotary embedding at given positions, token writes and
the attention of single tokens, at the sizes and masks where they can go wrong.

Tolerances, per element, from the arithmetic (u = 2^-8, half a bf16 step):
* bf16 results: u |ref| for the one rounding;
* dense layer: + (2 K + 16) 2^-23 (sum |a||w| + |b| + |r|), K fp32 additions
  that may truncate, and 2^-14 |ref| for the special-function unit;
* rotary: + 2^-20 (|a| + |b|): angle good to 2^-22, two products and a sum;
* attention: + (w + 2^-12) A with A the weighted mean of |V|: each weight is
  off by w (its rounding: 2^-8 as bf16, 2^-11 as f16) and by the score's fp32
  error and the exponential's, below 2^-12 for these scores;
* lse: 2^-20 (1 + |lse|) + d 2^-23 max_k sum |q||k| / sqrt(d).
Pages are compared bit for bit.
"""
import numpy as np
import pytest

import wave_inputs as wi
from oracle import block as oblock
from oracle import quant
from oracle import token as otok

from wave_testlib import bits_to_torch, torch_to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _bf(rng, *shape, scale=1.0):
    """bf16 values as float64."""
    return oblock.bf16_round(rng.standard_normal(shape) * scale)


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().bfloat16()


def _dev64(x):
    """bf16 values by their bits (subnormals too, which a conversion may flush)."""
    import torch
    bits = (np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()


def _strided(x, pad, fill=float("nan")):
    """The same values as columns of a wider tensor (the rest is `fill`)."""
    import torch
    t = _dev(x)
    wide = torch.full((t.shape[0], t[0].numel() + pad), fill, dtype=t.dtype, device="cuda")
    view = wide[:, :t[0].numel()]
    view.copy_(t.view(t.shape[0], -1))
    return view.view(t.shape) if t.dim() == 2 else view.unflatten(1, t.shape[1:])


def _cache(wave, heads=1, d=64, tokens=1, levels=1, window=0, prefix=0, pages=1, fp8=False, fill=None):
    import torch
    fmt = wave.KV_FP8_E4M3 if fp8 else wave.KV_BF16
    per = wave.KVCache.page_bytes(heads, d, fmt) + (2 * heads * 4 if fp8 else 0)
    pool = torch.empty(4096 + pages * per + 512, dtype=torch.uint8, device="cuda")
    if fill is not None:
        pool.fill_(fill)
    return wave.KVCache(heads, d, tokens, levels, window, prefix, pool=pool, kv_format=fmt)


def _within(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.abs(got - ref)[bad].max():.3e} where {tol[bad].min():.3e} is allowed, "
                           f"first at {tuple(np.argwhere(bad)[0])}")


# ------------------------------------------------------------- dense layer
def _linear_case(wave, kv, rng, M, K, N, act, bias, resid, pad=0, in_place=False):
    import torch
    a, w = _bf(rng, M, K), _bf(rng, N, K, scale=K ** -0.5)
    b = _bf(rng, N) if bias else None
    r = _bf(rng, M, N) if resid else None
    A = _strided(a, pad) if pad else _dev(a)
    R = (_strided(r, pad) if pad else _dev(r)) if resid else None
    if in_place:
        Y = R
    else:
        wide = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        Y = wide[:, :N]
    kv.linear_bias(A, _dev(w), Y, bias=_dev(b) if bias else None, R=R, act=act)
    kv.status()
    ref = otok.linear_bias(a, w, b, r, act)
    size = np.abs(a) @ np.abs(w).T + (np.abs(b) if bias else 0) + (np.abs(r) if resid else 0)
    _within(torch_to_f64(Y), ref, (U + 2.0 ** -14) * np.abs(ref) + (2 * K + 16) * 2.0 ** -23 * size,
            f"linear {M} x {K} x {N} {act}")
    if pad and not in_place:
        assert (wide[:, N:] == 7.0).all()


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("K,N", [(8, 8), (64, 256), (72, 136), (200, 264), (1000, 520)])
def test_linear_sizes(cuda_lib, M, K, N):
    kv = _cache(cuda_lib)
    _linear_case(cuda_lib, kv, np.random.default_rng(M * 1000 + N), M, K, N, "none", True, True)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("bias,resid", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M", [3, 150])
def test_linear_epilogues(cuda_lib, act, bias, resid, M):
    kv = _cache(cuda_lib)
    _linear_case(cuda_lib, kv, np.random.default_rng(11), M, 136, 392, act, bias, resid)


@pytest.mark.parametrize("M", [1, 5, 70, 260])
def test_linear_strides_and_in_place(cuda_lib, M):
    kv = _cache(cuda_lib)
    for in_place in (False, True):
        _linear_case(cuda_lib, kv, np.random.default_rng(12), M, 320, 264, "silu", True, True, pad=24,
                     in_place=in_place)


@pytest.mark.parametrize("M,K,N", [(1, 8960, 1536), (4, 1536, 8960), (100, 4096, 1536), (984, 1536, 1536)])
def test_linear_block_sizes(cuda_lib, M, K, N):
    kv = _cache(cuda_lib)
    _linear_case(cuda_lib, kv, np.random.default_rng(13), M, K, N, "gelu_tanh", True, True)


@pytest.mark.parametrize("M,K,N", [(8, 1536, 5000), (3, 2048, 4736), (5, 4096, 2368), (5, 4096, 2376), (9, 1536, 3552),
                                   (16, 1000, 3560), (16, 4096, 7104), (16, 4104, 520), (9, 264, 7112), (12, 8960, 1536)])
def test_linear_few_rows_by_waves(cuda_lib, M, K, N):
    """Both sides of each limit between the forms for up to 16 rows."""
    _linear_case(cuda_lib, _cache(cuda_lib), np.random.default_rng(6), M, K, N, "silu", True, True, pad=16)


def test_linear_no_rows(cuda_lib):
    import torch
    kv = _cache(cuda_lib)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    kv.linear_bias(e, torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda"),
                   torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"))
    kv.status()


def test_linear_extremes(cuda_lib):
    """Infinities and NaN stay in their own rows; activations at their ends."""
    import torch
    kv = _cache(cuda_lib)
    for M in (6, 140):
        a = np.zeros((M, 64))
        a[:, 0] = 1.0
        a[0, 0], a[1, 0], a[2, 0], a[3, 0] = np.inf, np.nan, 300.0, -300.0
        w = np.zeros((16, 64))
        w[:, 0] = 1.0
        for act in ("none", "gelu_tanh", "gelu_erf", "silu"):
            Y = torch.empty(M, 16, dtype=torch.bfloat16, device="cuda")
            kv.linear_bias(_dev(a), _dev(w), Y, act=act)
            y = torch_to_f64(Y)
            assert np.isnan(y[1]).all() and np.isfinite(y[2:]).all(), act
            # inf times the zero columns of w is NaN in exact arithmetic too
            assert (y[2] == 300).all() and (y[3] == (-300.0 if act == "none" else 0.0)).all(), act


@pytest.mark.parametrize("M", [3, 140, 2400])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
def test_linear_infinities(cuda_lib, act, M):
    """Every activation's limit: +inf stays; -inf is NaN (-inf times zero) but for none."""
    import torch
    kv = _cache(cuda_lib)
    a, w = np.full((M, 8), 1.0), np.full((1536 if M > 200 else 16, 8), 1.0)
    a[0] = a[M - 1] = np.inf
    a[1] = -np.inf
    Y = torch.empty(M, w.shape[0], dtype=torch.bfloat16, device="cuda")
    kv.linear_bias(_dev(a), _dev(w), Y, act=act)
    y = torch_to_f64(Y)
    assert np.isposinf(y[[0, M - 1]]).all()
    assert np.isneginf(y[1]).all() if act == "none" else np.isnan(y[1]).all()
    assert np.isfinite(y[2:M - 1]).all()


# ------------------------------------------------------------------ rotary
def _rotary_tol(x, ref):
    size = np.abs(x).max(-1, keepdims=True) * 2
    return U * np.abs(ref) + 2.0 ** -20 * size


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("ladder", ["axis", "ladder"])
@pytest.mark.parametrize("rows,qh,kh", [(1, 1, 1), (3, 4, 2), (130, 3, 3), (77, 24, 24)])
def test_rotary(cuda_lib, d, layout, ladder, rows, qh, kh):
    import torch
    kv = _cache(cuda_lib, d=d)
    rng = np.random.default_rng(rows + d)
    q, k = _bf(rng, rows, qh, d), _bf(rng, rows, kh, d)
    pos = rng.integers(0, 200, (rows, 3))
    P = torch.from_numpy(pos.astype(np.int32)).cuda()
    pairs = oblock.rope_groups(d)
    Q, K = _strided(q, 8 * 5), _strided(k, 8)
    for inverse in (False, True):
        Qo, Ko = torch.empty_like(_dev(q)), torch.empty_like(_dev(k))
        kv.rotary(P, Q, K, Qo, Ko, layout=layout, ladder=ladder, inverse=inverse)
        for got, x in ((Qo, q), (Ko, k)):
            ref = otok.rotary(x, pos, pairs, layout=layout, ladder=ladder, inverse=inverse)
            _within(torch_to_f64(got), ref, _rotary_tol(x, ref), f"rotary {layout} {ladder}")
    Qi = Q.clone()   # in place, Q alone
    kv.rotary(P, Qi, layout=layout, ladder=ladder)
    assert torch.equal(Qi, kv.rotary(P, Q, None, torch.empty_like(Qi), layout=layout, ladder=ladder))


@pytest.mark.parametrize("pairs", [(32, 0, 0), (0, 0, 0), (0, 7, 0), (1, 1, 1), (5, 20, 2)])
def test_rotary_sections(cuda_lib, pairs):
    """Axes of any size; pairs past them are copied bit for bit, infinities too."""
    import torch
    kv = _cache(cuda_lib)
    rng = np.random.default_rng(21)
    x = _bf(rng, 9, 2, 64)
    pos = rng.integers(-1000, 1000, (9, 3))
    P = torch.from_numpy(pos.astype(np.int32)).cuda()
    for layout in ("interleaved", "halves"):
        y = x.copy()
        left = np.arange(sum(pairs), 32)
        at = np.r_[2 * left, 2 * left + 1] if layout == "interleaved" else np.r_[left, left + 32]
        y[0][:, at] = np.inf
        out = torch.empty(9, 2, 64, dtype=torch.bfloat16, device="cuda")
        kv.rotary(P, _dev(y), None, out, pairs=pairs, layout=layout, base=500.0)
        got = torch_to_f64(out)
        assert np.array_equal(got[..., at], y[..., at])
        ref = otok.rotary(x, pos, pairs, 500.0, layout)
        rest = np.setdiff1d(np.arange(64), at)
        _within(got[..., rest], ref[..., rest], _rotary_tol(x, ref)[..., rest], f"pairs {pairs}")


def test_rotary_far_positions(cuda_lib):
    """Any int32 position: the angle is reduced without loss. Reference angles in
    exact rational turns (numpy longdouble of pos * freq modulo 2 pi is not enough
    for base^0 pairs only, whose frequency is 1)."""
    import torch
    from fractions import Fraction
    import math
    kv = _cache(cuda_lib)
    vals = [0, 1, -1, 10 ** 6, 123456789, 2 ** 31 - 1, -2 ** 31]
    pos = np.zeros((len(vals), 3), dtype=np.int64)
    pos[:, 1] = vals
    # base 16, 4 pairs per axis: frequencies 1, 1/2, 1/4, 1/8 exactly
    x = np.zeros((len(vals), 1, 64))
    x[..., 0::2] = 1.0
    out = torch.empty(len(vals), 1, 64, dtype=torch.bfloat16, device="cuda")
    kv.rotary(torch.from_numpy(pos.astype(np.int32)).cuda(), _dev(x), None, out, pairs=(0, 4, 0), base=16.0)
    got = torch_to_f64(out)[:, 0]
    pi2 = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615")
    for i, v in enumerate(vals):
        for p in range(4):
            t = float(Fraction(v, 2 ** p) % pi2)
            assert abs(got[i, 2 * p] - math.cos(t)) <= U + 2.0 ** -20, (v, p)
            assert abs(got[i, 2 * p + 1] - math.sin(t)) <= U + 2.0 ** -20, (v, p)


# ------------------------------------------------------------- token writes
def _pages(kv, entry):
    """K and V pages of an entry: bf16 bits [2][pages][H][128][d], or FP8 codes and scales."""
    pb, off, _ = kv.layout()
    ids = kv.entry_pages(*entry)
    host = kv.pool.cpu().numpy()
    fp8 = kv.kv_format == 1
    shape = (2, kv.heads, 128, kv.head_dim)
    pages = np.stack([host[off + p * pb:off + (p + 1) * pb].view(np.uint8 if fp8 else np.uint16).reshape(shape)
                      for p in ids], 1)
    if not fp8:
        return pages
    at = kv.scale_offset()
    table = host[at:at + (max(ids) + 1) * 2 * kv.heads * 4].view(np.float32).reshape(-1, 2, kv.heads)
    return pages, table[ids].transpose(1, 0, 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,cuts", [(1, [1]), (5, [1, 4]), (300, [1, 127, 1, 100, 71]),
                                         (300, [300]), (256, [128, 128]), (130, [0, 129, 1])])
def test_write_in_pieces_is_an_append(cuda_lib, d, tokens, cuts):
    import torch
    H = 3
    kv = _cache(cuda_lib, H, d, tokens, 1, pages=20, fill=0xFF)  # NaN wherever nothing was written
    x = _dev(np.random.default_rng(31).standard_normal((tokens, 3, H, d)))
    kv.append(9, 0, x[:, 1].contiguous(), x[:, 2].contiguous())
    kv.alloc(0, 1)
    kv.alloc(1, 1)
    at = 0
    for n in cuts:
        part = x[at:at + n]
        if n == 1:   # one token of one entry, and a run into another in the same call
            kv.write_tokens([(0, 1), (1, 1)], [at, at], torch.cat([part[:, 1]] * 2),
                            torch.cat([part[:, 2]] * 2))
        else:        # read from the packed projection
            kv.write_tokens([(0, 1)], [at], part[:, 1], part[:, 2], [n])
            kv.write_tokens([(1, 1)], [at], part[:, 1], part[:, 2], [n])
        at += n
    want = _pages(kv, (9, 0))
    assert np.array_equal(_pages(kv, (0, 1)), want) and np.array_equal(_pages(kv, (1, 1)), want)
    # a rewrite touches its own rows only
    y = _dev(np.random.default_rng(32).standard_normal((1, H, d)))
    kv.write_tokens([(0, 1)], [tokens - 1], y, y)
    got = _pages(kv, (0, 1))
    page, row = (tokens - 1) // 128, (tokens - 1) % 128
    bits = y.view(torch.int16).cpu().numpy().view(np.uint16)[0]
    assert np.array_equal(got[0, page, :, row], bits) and np.array_equal(got[1, page, :, row], bits)
    got[:, page, :, row] = want[:, page, :, row]
    assert np.array_equal(got, want) and np.array_equal(_pages(kv, (1, 1)), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,cuts", [(1, [1]), (6, [1] * 6), (300, [1, 3, 124, 1, 100, 71]), (300, [300])])
def test_write_fp8_bits(cuda_lib, d, tokens, cuts):
    H = 2
    rng = np.random.default_rng(33)
    kv = _cache(cuda_lib, H, d, tokens, 1, pages=12, fp8=True, fill=0x7F)
    kv.alloc(0, 0)
    kv.alloc(1, 0)
    x = oblock.bf16_round(rng.standard_normal((2, tokens, H, d)) * np.exp(rng.standard_normal((2, tokens, 1, 1))))
    x[0, 0] = 0.0           # a zero first token of K
    x[1, :, 1] = 0.0        # a head of V that stays zero
    ents = [otok.Fp8Entry(tokens, H, d) for _ in range(2)]
    at = 0
    for n in cuts:
        for i in range(2):
            ents[i].write(at, x[i, at:at + n])
        kv.write_tokens([(1, 0)], [at], _dev(x[0, at:at + n]), _dev(x[1, at:at + n]), [n])
        at += n
    codes, scales = _pages(kv, (1, 0))
    for i in range(2):
        assert np.array_equal(scales[i], ents[i].scales)
        assert np.array_equal(quant.e4m3_decode(codes[i]), quant.e4m3_decode(ents[i].codes))
    # an appended entry counts as written whole: its tokens can be replaced
    kv.append(1, 1, _dev(x[0]), _dev(x[1]))
    big = 50 * x[:, :1] + 1.0
    for i, ent in enumerate(ents):
        ent.__init__(tokens, H, d)
        ent.write(0, x[i])
        ent.write(0, oblock.bf16_round(big[i]))
    kv.write_tokens([(1, 1)], [0], _dev(oblock.bf16_round(big[0])), _dev(oblock.bf16_round(big[1])))
    codes, scales = _pages(kv, (1, 1))
    for i in range(2):
        assert np.array_equal(scales[i], ents[i].scales)
        assert np.array_equal(quant.e4m3_decode(codes[i]), quant.e4m3_decode(ents[i].codes))


def test_write_fp8_every_quotient(cuda_lib):
    """Codes of values that lie on and next to rounding borders: all 128 bf16
    mantissas over 12 binades, both signs, against a page maximum each from all
    mantissas, and scales near the ends of float32."""
    H, d = 2, 128
    rng = np.random.default_rng(34)
    mant = 1.0 + np.arange(128) / 128.0
    for k in range(0, 40):
        top = mant[(37 * k) % 128] * 2.0 ** rng.integers(-3, 4)
        if k >= 34:
            top = (2.0 ** -118, 2.0 ** -125, 2.0 ** -133 * 3, 2.0 ** 110, 2.0 ** 127, 2.0 ** -104 * 1.5)[k - 34]
        x = np.zeros((100, H, d))
        vals = mant[None, :] * 2.0 ** -np.arange(0, 100)[:, None] * top
        x[:] = np.where(rng.random((100, 1, d)) < 0.5, -1, 1) * np.minimum(vals, top)[:, None, :]
        x[0, :, 0] = top
        x = oblock.bf16_round(x)
        kv = _cache(cuda_lib, H, d, 100, 1, pages=1, fp8=True)
        kv.alloc(0, 1)
        kv.write_tokens([(0, 1)], [0], _dev64(x), _dev64(x), [100])
        ent = otok.Fp8Entry(100, H, d)
        ent.write(0, x)
        codes, scales = _pages(kv, (0, 1))
        for i in range(2):
            assert np.array_equal(scales[i], ent.scales), top
            assert np.array_equal(codes[i][:, :, :100], ent.codes[:, :, :100]), top


# ---------------------------------------------------------- token attention
class _World:
    """A cache with written entries and the values that attention reads."""

    def __init__(self, wave, heads, d, tokens, levels, window=0, prefix=0, fp8=False, pages=64, seed=0,
                 scale=1.0):
        self.kv = _cache(wave, heads, d, tokens, levels, window, prefix, pages, fp8, fill=0xFF)
        self.rng = np.random.default_rng(seed)
        self.window, self.heads, self.d, self.tokens, self.fp8 = window, heads, d, tokens, fp8
        self.scale = scale
        self.entries, self.prefix = {}, None
        if prefix:
            self.prefix = self.add(-1, 0, prefix)

    def add(self, c, l, n=None):
        n = self.tokens if n is None else n
        k, v = (_bf(self.rng, n, self.heads, self.d, scale=self.scale) for _ in range(2))
        self.kv.append(c, l, _dev(k), _dev(v))
        if self.fp8:
            k, v = (self._stored(x) for x in (k, v))
        self.entries[c, l] = (k, v)
        return k, v

    def _stored(self, x):
        ent = otok.Fp8Entry(x.shape[0], self.heads, self.d)
        ent.write(0, x)
        return ent.values(x.shape[0])

    def check(self, nodes, policy="progressive", own=None, group=1, strided=False, what=""):
        import torch
        n, hq = len(nodes), self.heads * group
        q = _bf(self.rng, n, hq, self.d)
        Q = _strided(q, 40) if strided else _dev(q)
        wide = torch.full((n, hq * self.d + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        O = wide[:, :hq * self.d].unflatten(1, (hq, self.d))
        lse = torch.full((n, hq), float("nan"), device="cuda")
        need = self.kv.token_attn_workspace(nodes, policy, own, q_heads=hq)
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        self.kv.token_attn(nodes, policy, Q, O, own_tokens=own, lse=lse, workspace=ws)
        self.kv.status()
        assert (wide[:, hq * self.d:] == 7.0).all()
        first = O.clone()
        self.kv.token_attn(nodes, policy, Q, O, own_tokens=own, workspace=ws)  # again, without lse
        assert torch.equal(O, first), "the same call gives other bytes"
        got, glse = torch_to_f64(O), lse.double().cpu().numpy()
        w = 2.0 ** -11 if self.fp8 else 2.0 ** -8
        for i, node in enumerate(nodes):
            k, v = otok.node_tokens(node, policy, self.window, self.entries, self.prefix,
                                    None if own is None else own[i])
            k, v = (x.reshape(-1, self.heads, self.d) if x.size == 0 else x for x in (k, v))
            o, l, a = otok.token_attention(q[i], k, v)
            _within(got[i], o, U * np.abs(o) + (w + 2.0 ** -12) * a + 1e-30, f"{what} query {i} {node}")
            if k.shape[0] == 0:
                assert np.isneginf(glse[i]).all() and not got[i].any()
                continue
            big = max((np.abs(k[:, x // group]) @ np.abs(q[i, x])).max() for x in range(hq))
            tol = 2.0 ** -20 * (1 + np.abs(l)) + self.d * 2.0 ** -23 * big / self.d ** 0.5
            _within(glse[i], l, tol, f"{what} lse {i}")
        return got


FORMATS = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


@FORMATS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 128, 129, 300])
def test_token_attn_own_counts(cuda_lib, fp8, d, tokens):
    w = _World(cuda_lib, 2, d, tokens, 1, fp8=fp8, seed=tokens)
    w.add(0, 1)
    for own in sorted({0, 1, 2, 8, 9, tokens // 2, max(0, tokens - 1), tokens} & set(range(tokens + 1))):
        w.check([(0, 1)], own=[own], what=f"own {own} of {tokens}")
    w.check([(0, 1)])


@FORMATS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 16])
def test_token_attn_round(cuda_lib, fp8, d, group):
    """A round's nodes share history; own counts differ, one is nothing."""
    w = _World(cuda_lib, 3, d, 200, 3, prefix=77, fp8=fp8, seed=group)
    for c in range(4):
        w.add(c, 0)
    for i in range(3):
        w.add(4 + i, i + 1)
    nodes = [(4, 1), (5, 2), (6, 3)]
    w.check(nodes, own=[200, 77, 0], group=group, strided=True, what="round")
    w.check(nodes[::-1], group=group, what="reversed, whole")


@FORMATS
def test_token_attn_same_node_many_times(cuda_lib, fp8):
    """Several tokens of one entry, each seeing up to itself: more than 16 rows."""
    w = _World(cuda_lib, 2, 128, 150, 1, window=2, fp8=fp8, seed=5)
    for c in range(3):
        w.add(c, 0)
    w.add(3, 1)
    own = list(range(120, 150))
    w.check([(3, 1)] * 30, own=own, what="tokens of one entry")
    w.check([(3, 1)] * 20, own=[150] * 20, group=4, what="equal tokens")


@pytest.mark.parametrize("policy", ["clean", "same", "progressive"])
def test_token_attn_policies(cuda_lib, policy):
    w = _World(cuda_lib, 2, 64, 130, 2, window=3, prefix=5, seed=6)
    for c in range(5):
        for l in range(3):
            w.add(c, l)
    w.check([(4, 2), (4, 1), (0, 0), (2, 2)], policy, own=[130, 1, 0, 129])


def test_token_attn_empty(cuda_lib):
    """Queries that see nothing, alone, among others, and a call of none."""
    import torch
    w = _World(cuda_lib, 2, 64, 140, 1, seed=7)
    w.check([(0, 1)], own=[0])                       # no entry exists yet
    w.check([(0, 1), (0, 0)], own=[0, 0], group=16)  # two groups, both empty
    w.add(0, 1)
    w.check([(0, 1), (0, 1), (0, 1)], own=[0, 5, 0], group=16)  # groups: empty, not, empty
    w.check([(0, 1), (0, 1)], own=[0, 140])
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    w.kv.token_attn([], "clean", e, e)


@FORMATS
def test_token_attn_long_list(cuda_lib, fp8):
    """Enough pages that every SM has a part and lists are cut anywhere; more than
    one table size; pages out of order."""
    w = _World(cuda_lib, 5, 128, 640, 1, prefix=33, fp8=fp8, pages=400, seed=8)
    for c in range(30):
        w.add(c, 1)
    for c in range(0, 30, 2):       # holes, filled in another order
        w.kv.release(c, 1)
    for c in list(range(28, -1, -2)):
        w.add(c, 1)
    w.check([(29, 1)], "same", own=[639], what="one query")
    w.check([(29, 1), (20, 1), (29, 1)], "same", own=[1, 640, 500], group=2, what="three queries")


def test_token_attn_large_tables(cuda_lib):
    """More than 512 list items in one call (the larger table)."""
    w = _World(cuda_lib, 1, 64, 128, 1, pages=700, seed=9)
    for c in range(600):
        w.add(c, 1)
    w.check([(599, 1)], "same", what="600 pages")
    w.check([(599, 1)] * 2, "same", own=[128, 3], group=16, what="two groups")


@FORMATS
def test_token_attn_garbage_behind_the_mask(cuda_lib, fp8):
    """NaN and infinities in tokens that a query does not see reach nothing:
    tokens past its count, pages that only other queries see."""
    import torch
    H, d, T = 2, 128, 200
    w = _World(cuda_lib, H, d, T, 2, fp8=fp8, seed=10)
    for c in range(2):
        w.add(c, 0)
    w.add(2, 1)
    w.add(3, 2)
    # node (2, 1) sees its first 100 tokens; the others hold NaN and infinities
    bad = torch.full((100, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    if not fp8:
        bad[::2] = float("inf")
        w.kv.write_tokens([(2, 1)], [100], bad, bad, [100])
    else:
        page = w.kv.entry_pages(2, 1)
        pb, off, _ = w.kv.layout()
        codes = w.kv.pool[off:].view(torch.uint8)
        for p, row in ((page[0], 100), (page[1], 0)):
            tile = codes[p * pb:(p + 1) * pb].view(2 * H, 128, d)
            tile[:, row:] = 0x7F
    w.check([(2, 1)], own=[100], what="past the count")
    w.check([(2, 1), (2, 1)], own=[100, 37], what="two counts")
    # beside a query that does see them (its own result is NaN): (3, 2) reads (2, 1)
    q = _bf(w.rng, 2, H, d)
    O = torch.empty(2, H, d, dtype=torch.bfloat16, device="cuda")
    nodes, own = [(2, 1), (3, 2)], [100, 200]
    ws = torch.empty(max(1, w.kv.token_attn_workspace(nodes, "progressive", own)), dtype=torch.uint8, device="cuda")
    w.kv.token_attn(nodes, "progressive", _dev(q), O, own_tokens=own, workspace=ws)
    k, v = otok.node_tokens((2, 1), "progressive", 0, w.entries, None, 100)
    o, _, a = otok.token_attention(q[0], k, v)
    got = torch_to_f64(O)
    _within(got[0], o, U * np.abs(o) + (2.0 ** -8 + 2.0 ** -12) * a, "beside NaN")
    assert np.isnan(got[1]).all()


@FORMATS
@pytest.mark.parametrize("tokens", [1, 40, 128 * 160])
def test_token_attn_nan_that_is_seen(cuda_lib, fp8, tokens):
    """Keys that are all NaN, in a list of one CTA, of a cluster, and of several
    clusters: the result is NaN, not that of a query that sees nothing."""
    import torch
    wave = cuda_lib
    kv = _cache(wave, 1, 64, tokens, 1, pages=(tokens + 127) // 128, fp8=fp8)
    k = torch.full((tokens, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    kv.append(0, 1, k, v)
    if fp8:  # the append's codes of NaN are its own matter: set E4M3's
        pb, off, _ = kv.layout()
        codes = kv.pool[off:].view(torch.uint8)
        for p in kv.entry_pages(0, 1):
            codes[p * pb:(p + 1) * pb].view(2, 128, 64)[0] = 0x7F
    q = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = torch.zeros_like(q), torch.zeros(2, 1, device="cuda")
    nodes, own = [(0, 1)] * 2, [tokens, 0]
    ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "same", own)), dtype=torch.uint8, device="cuda")
    kv.token_attn(nodes, "same", q, O, own_tokens=own, lse=lse, workspace=ws)
    kv.status()
    assert torch.isnan(O[0]).all() and torch.isnan(lse[0]).all()
    assert (O[1] == 0).all() and torch.isneginf(lse[1]).all()


@FORMATS
def test_token_attn_large_and_small_values(cuda_lib, fp8):
    """Peaked weights and magnitudes far from 1 (keys and values of 2^40 and 2^-40)."""
    import torch
    H, d, T = 2, 64, 300
    for power in (40, -40):
        w = _World(cuda_lib, H, d, T, 1, fp8=fp8, seed=11, scale=2.0 ** power)
        w.add(0, 1)
        k, v = w.entries[0, 1]
        q = _bf(w.rng, 1, H, d, scale=4 * 2.0 ** -power)
        O = torch.empty(1, H, d, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(1, w.kv.token_attn_workspace([(0, 1)], "same")), dtype=torch.uint8, device="cuda")
        w.kv.token_attn([(0, 1)], "same", _dev(q), O, workspace=ws)
        o, _, a = otok.token_attention(q[0], k, v)
        _within(torch_to_f64(O)[0], o, U * np.abs(o) + (2.0 ** -8 + 2.0 ** -12) * a, f"2^{power}")


# ------------------------------------------------------------- used together
@FORMATS
def test_tokens_stream_through_a_block(cuda_lib, fp8):
    """Tokens arrive one at a time in two nodes: projection with bias, rotary at
    their positions, write, attention over history and the tokens before them,
    out-projection with bias and residual, MLP -- against the oracle, which
    takes each step from the library's own bf16 results of the step before."""
    import torch
    H, d, T, dim = 3, 64, 132, 136
    rng = np.random.default_rng(12)
    w = _World(cuda_lib, H, d, T, 2, prefix=9, fp8=fp8, seed=13)
    for c in range(2):
        w.add(c, 0)
    nodes = [(2, 1), (3, 2)]
    kv = w.kv
    held = {}
    for n in nodes:
        kv.alloc(*n)
        held[n] = [otok.Fp8Entry(T, H, d) for _ in range(2)] if fp8 else [np.zeros((T, H, d)) for _ in range(2)]
    # the second node reads the first's entry as history: start with it written
    first = [_bf(rng, T, H, d) for _ in range(2)]
    kv.write_tokens([nodes[0]], [0], _dev(first[0]), _dev(first[1]), [T])
    for i in range(2):
        if fp8:
            held[nodes[0]][i].write(0, first[i])
        else:
            held[nodes[0]][i][:] = first[i]
    Wqkv, Bqkv = _bf(rng, 3 * H * d, dim, scale=dim ** -0.5), _bf(rng, 3 * H * d, scale=0.1)
    Wo, Bo = _bf(rng, dim, H * d, scale=(H * d) ** -0.5), _bf(rng, dim, scale=0.1)
    W1, B1 = _bf(rng, 512, dim, scale=dim ** -0.5), _bf(rng, 512, scale=0.1)
    W2, B2 = _bf(rng, dim, 512, scale=512 ** -0.5), _bf(rng, dim, scale=0.1)
    dev = {n: _dev(x) for n, x in (("Wqkv", Wqkv), ("Bqkv", Bqkv), ("Wo", Wo), ("Bo", Bo), ("W1", W1),
                                   ("B1", B1), ("W2", W2), ("B2", B2))}
    empty = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f64 = torch_to_f64
    start = 126
    for n in nodes[1:]:
        pre = [_bf(rng, start, H, d) for _ in range(2)]
        kv.write_tokens([n], [0], _dev(pre[0]), _dev(pre[1]), [start])
        for i in range(2):
            if fp8:
                held[n][i].write(0, pre[i])
            else:
                held[n][i][:start] = pre[i]
    for t in range(start, T):
        x = _bf(rng, 2, dim)
        X, P = _dev(x), empty(2, 3 * H * d)
        kv.linear_bias(X, dev["Wqkv"], P, bias=dev["Bqkv"])
        pos = np.array([[40 * c + t, t // 8, t % 8] for c, _ in nodes])
        Q, K, V = P.view(2, 3, H, d).unbind(1)
        before = f64(P).reshape(2, 3, H, d)
        kv.rotary(torch.from_numpy(pos.astype(np.int32)).cuda(), Q, K)       # in place
        kv.write_tokens(nodes, [t, t], K, V)
        own = [t + 1, t + 1]
        O = empty(2, H, d)
        ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "progressive", own)), dtype=torch.uint8, device="cuda")
        kv.token_attn(nodes, "progressive", Q, O, own_tokens=own, workspace=ws)
        Y, U1, Z = empty(2, dim), empty(2, 512), empty(2, dim)
        kv.linear_bias(O.view(2, H * d), dev["Wo"], Y, bias=dev["Bo"], R=X)
        kv.linear_bias(Y, dev["W1"], U1, bias=dev["B1"], act="gelu_tanh")
        kv.linear_bias(U1, dev["W2"], Z, bias=dev["B2"], R=Y)
        kv.status()
        # each step against the oracle on what it was given
        got = f64(P).reshape(2, 3, H, d)
        for i in range(2):
            ref = otok.rotary(before[:, i], pos, oblock.rope_groups(d))
            _within(got[:, i], ref, _rotary_tol(before[:, i], ref), f"rotary of token {t}")
        lin = otok.linear_bias(x, Wqkv, Bqkv).reshape(before.shape)
        _within(before, lin, U * 1.1 * np.abs(lin) + 2.0 ** -14, "projection")
        for j, n in enumerate(nodes):
            for i in range(2):
                new = got[j, 1 + i][None] if i == 0 else before[j, 2][None]
                if fp8:
                    held[n][i].write(t, new)
                else:
                    held[n][i][t] = new[0]
            w.entries[n] = tuple(e.values(T) if fp8 else e for e in held[n])
        for j, n in enumerate(nodes):
            k, v = otok.node_tokens(n, "progressive", 0, w.entries, w.prefix, t + 1)
            o, _, a = otok.token_attention(got[j, 0], k, v)
            _within(f64(O)[j], o, U * np.abs(o) + (2.0 ** -8 + 2.0 ** -12) * a, f"attention of token {t}")
        y = otok.linear_bias(f64(O).reshape(2, -1), Wo, Bo, x)
        u = otok.linear_bias(f64(Y), W1, B1, None, "gelu_tanh")
        z = otok.linear_bias(f64(U1), W2, B2, f64(Y))
        for name, a, b in (("out", Y, y), ("up", U1, u), ("down", Z, z)):
            _within(f64(a), b, U * 1.1 * np.abs(b) + 2.0 ** -13, f"{name} of token {t}")
    # once the unit is whole, the round's attention reads the same entries
    if not fp8:
        kvw = _dev(held[nodes[0]][0]), _dev(held[nodes[0]][1])
        kv.append(9, 0, *kvw)
        assert np.array_equal(_pages(kv, nodes[0]), _pages(kv, (9, 0)))


# ------------------------------------------------- streams, graphs, timeouts
def test_token_ops_in_a_graph_on_a_side_stream(cuda_lib):
    """Captured and replayed on another stream, with new data in the same buffers."""
    import torch
    w = _World(cuda_lib, 2, 64, 200, 1, seed=14, pages=40)
    for c in range(8):
        w.add(c, 1)
    kv, nodes, own = w.kv, [(7, 1)], [200]
    X = torch.empty(1, 128, dtype=torch.bfloat16, device="cuda")
    W = _dev(_bf(w.rng, 2 * 64, 128, scale=0.1))
    Q = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    O = torch.empty_like(Q)
    pos = torch.tensor([[5, 6, 7]], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "same", own)), dtype=torch.uint8, device="cuda")

    def step():
        kv.linear_bias(X, W, Q.view(1, 128))
        kv.rotary(pos, Q)
        kv.write_tokens([(7, 1)], [199], Q, Q)
        kv.token_attn(nodes, "same", Q, O, own_tokens=own, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        X.copy_(_dev(_bf(w.rng, 1, 128)))
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x = _bf(w.rng, 1, 128)
        X.copy_(_dev(x))
        graph.replay()
        torch.cuda.synchronize()
        replayed = O.clone()
        O.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(replayed, O), f"replay {i}"
    del graph


def test_captured_across_streams_and_other_nodes(cuda_lib):
    """A capture whose launches follow a fill, a copy, another library's kernel and a
    join of two streams (a launch that may start early is captured as an edge of
    its own kind, from each of these)."""
    import torch
    w = _World(cuda_lib, 2, 64, 200, 1, seed=15, pages=40)
    for c in range(4):
        w.add(c, 1)
    kv, nodes = w.kv, [(3, 1)]
    A, B = (_dev(_bf(w.rng, 40, 128)) for _ in range(2))
    W = _dev(_bf(w.rng, 128, 128, scale=0.1))
    X, Y, Z, O = (torch.empty(40, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    pos = torch.zeros(40, 3, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "same", [200])), dtype=torch.uint8, device="cuda")
    other = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        Y.zero_()
        kv.linear_bias(A, W, X, R=Y)                       # after a fill
        other.wait_stream(here)
        with torch.cuda.stream(other):
            kv.linear_bias(B, W, Z)                        # after the fork
            kv.rotary(pos, Z.view(40, 2, 64))
        kv.rotary(pos, X.view(40, 2, 64))
        here.wait_stream(other)
        kv.linear_bias(X, W, Y, R=Z)                       # after the join
        X.copy_(Y)
        kv.rotary(pos, X.view(40, 2, 64), inverse=True)    # after a copy
        X.mul_(0.5)
        O.zero_()
        kv.token_attn(nodes, "same", X.view(40, 2, 64)[:1], O.view(40, 2, 64)[:1], own_tokens=[200], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = [t.clone() for t in (X, Y, Z, O)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for t in (X, Y, Z, O):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (X, Y, Z, O)))
    kv.status()
    del graph


@pytest.mark.parametrize("M,K,N", [(40, 4096, 1536), (300, 8960, 1536), (3000, 1536, 4608)],
                         ids=["cluster", "split pairs", "pairs"])
def test_linear_timeout_is_reported(cuda_lib, M, K, N):
    """A wait that runs out in the tiled forms is reported, the cluster leaves in
    step, and the next call is right again."""
    import torch
    kv = _cache(cuda_lib)
    a = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    w = torch.full((N, K), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    kv.set_wait_limit(1)
    kv.linear_bias(a, w, y)
    with pytest.raises(cuda_lib.WaveError) as e:
        kv.status()
    assert e.value.code == -5
    kv.set_wait_limit(0)
    kv.linear_bias(a, w, y)
    kv.status()
    assert (y == K * 2.0 ** -10).all()   # 4, 8.75 or 1.5: exact in bf16


@FORMATS
def test_pages_past_four_gigabytes(cuda_lib, fp8):
    """Entries at the end of a pool of 10 GB: page offsets pass 32 bits."""
    import torch
    H, d, T = 24, 128, 300
    fmt = cuda_lib.KV_FP8_E4M3 if fp8 else cuda_lib.KV_BF16
    per = cuda_lib.KVCache.page_bytes(H, d, fmt)
    pages = 10 * 2 ** 30 // per
    w = _World(cuda_lib, H, d, T, 1, fp8=fp8, pages=1)
    w.kv = kv = _cache(cuda_lib, H, d, T, 1, pages=pages, fp8=fp8)
    filler = 0
    while kv.free_pages() >= 12:        # three pages each; host only, nothing is written
        kv.alloc(100 + filler, 1)
        filler += 1
    for c in range(2):
        w.add(c, 0)
    kv.alloc(2, 1)
    assert min(kv.entry_pages(2, 1)) * per > 9 * 2 ** 30
    k, v = (_bf(w.rng, T, H, d) for _ in range(2))
    kv.write_tokens([(2, 1)], [0], _dev(k[:200]), _dev(v[:200]), [200])
    kv.write_tokens([(2, 1)], [200], _dev(k[200:]), _dev(v[200:]), [100])
    if fp8:
        ents = [otok.Fp8Entry(T, H, d) for _ in range(2)]
        for e, x in zip(ents, (k, v)):
            e.write(0, x[:200])
            e.write(200, x[200:])
        k, v = (e.values(T) for e in ents)
    w.entries[2, 1] = (k, v)
    w.check([(2, 1), (2, 1)], own=[300, 129], what="far pages")


def test_token_attn_two_streams(cuda_lib):
    """Calls on two streams at once, a workspace each, and one on a third stream
    with other sizes: the results of calls alone."""
    import torch
    w = _World(cuda_lib, 2, 64, 640, 1, pages=200, seed=16)
    for c in range(30):
        w.add(c, 1)
    kv = w.kv
    cases = [([(29, 1)], [640], 2), ([(28, 1), (29, 1)], [3, 77], 4), ([(5, 1)] * 3, [1, 2, 640], 2)]
    q = [torch.randn(len(n), g, 64, device="cuda").bfloat16() for n, _, g in cases]
    ws = [torch.empty(max(1, kv.token_attn_workspace(n, "same", own, q_heads=g)), dtype=torch.uint8, device="cuda")
          for n, own, g in cases]
    want = []
    for (n, own, g), x, s in zip(cases, q, ws):
        o = torch.empty_like(x)
        kv.token_attn(n, "same", x, o, own_tokens=own, workspace=s)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[torch.empty_like(x) for _ in range(20)] for x in q]
    for i in range(20):
        for (n, own, g), x, s, o, stream in zip(cases, q, ws, got, streams):
            kv.token_attn(n, "same", x, o[i], own_tokens=own, workspace=s, stream=stream)
    torch.cuda.synchronize()
    for w0, os in zip(want, got):
        assert all(torch.equal(o, w0) for o in os)


def test_token_attn_timeout_is_reported(cuda_lib):
    """A wait that runs out is reported, and the next call is right again. 210 MB
    of pages, so that tiles come from HBM, one every 1.4 us per SM."""
    import torch
    kv = _cache(cuda_lib, 8, 128, 128, 1, pages=400, fill=0)
    for c in range(400):
        kv.alloc(c, 1)
    q = torch.ones(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kv.token_attn_workspace([(399, 1)], "same"), dtype=torch.uint8, device="cuda")
    kv.set_wait_limit(1)
    kv.token_attn([(399, 1)], "same", q, torch.empty_like(q), workspace=ws)
    with pytest.raises(cuda_lib.WaveError) as e:
        kv.status()
    assert e.value.code == -5
    kv.set_wait_limit(0)
    o, lse = torch.ones_like(q), torch.zeros(1, 8, device="cuda")
    kv.token_attn([(399, 1)], "same", q, o, lse=lse, workspace=ws)
    kv.status()
    # all scores 0: log of the 51200 tokens; all values 0
    assert not o.any() and (lse.double() - np.log(51200.0)).abs().max() < 2.0 ** -20 * 12


@FORMATS
@pytest.mark.parametrize("d", [64, 128])
def test_token_attn_many_calls_back_to_back(cuda_lib, fp8, d):
    """Long lists, hundreds of calls with nothing between them: equal bytes. (Tiles
    land in any order and the warps' teams drift apart.)"""
    import torch
    H, T = 6, 1280
    kv = _cache(cuda_lib, H, d, T, 1, pages=300, fp8=fp8, fill=0)
    K, V = (torch.randn(T, H, d, device="cuda").bfloat16() for _ in range(2))
    for c in range(30):
        kv.append(c, 1, K, V)
    q = torch.randn(2, H, d, device="cuda").bfloat16()
    nodes, own = [(29, 1), (28, 1)], [T, 77]
    ws = torch.empty(kv.token_attn_workspace(nodes, "same", own), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(300)]
    for o in outs:
        kv.token_attn(nodes, "same", q, o, own_tokens=own, workspace=ws)
    kv.status()
    assert torch.isfinite(outs[0].float()).all() and all(torch.equal(o, outs[0]) for o in outs)


# ---------------------------------------------- what lies beside the outputs
@pytest.mark.parametrize("M,K,N", [(1, 64, 24), (13, 264, 520), (37, 1000, 1544), (300, 72, 200), (984, 4096, 1536),
                                   (1500, 200, 776), (4000, 136, 1544)])
def test_rows_around_a_dense_layer_stay(cuda_lib, M, K, N):
    """Rows before and behind Y, and columns beside it, in every form."""
    import torch
    kv, rng = _cache(cuda_lib), np.random.default_rng(21)
    a, w = _bf(rng, M, K), _bf(rng, N, K, scale=K ** -0.5)
    big = torch.full((M + 300, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = big[150:150 + M, 8:8 + N]
    kv.linear_bias(_dev(a), _dev(w), Y, act="silu")
    kv.status()
    want = otok.linear_bias(a, w, None, None, "silu")
    size = np.abs(a) @ np.abs(w).T
    _within(torch_to_f64(Y), want, (U + 2.0 ** -14) * np.abs(want) + (2 * K + 16) * 2.0 ** -23 * size)
    Y.fill_(7.0)
    assert (big == 7.0).all()


@FORMATS
def test_rows_around_the_other_outputs_stay(cuda_lib, fp8):
    """Rows behind rotated ones, behind O and lse; pages of other entries, and the pool
    around them, under a write."""
    import torch
    H, d = 3, 64
    w = _World(cuda_lib, H, d, 300, 1, fp8=fp8, seed=22)
    for c in range(3):
        w.add(c, 1)
    kv = w.kv
    big = torch.full((90, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.randint(-9, 9, (77, 3), dtype=torch.int32, device="cuda")
    kv.rotary(pos, torch.ones(77, H, d, dtype=torch.bfloat16, device="cuda"), Qout=big[5:82])
    assert (big[:5] == 7.0).all() and (big[82:] == 7.0).all() and not (big[5:82] == 7.0).any()
    big.fill_(7.0)
    lse = torch.full((90, H), 7.0, device="cuda")
    nodes, own = [(2, 1)] * 3, [300, 1, 0]
    ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "same", own)), dtype=torch.uint8, device="cuda")
    kv.token_attn(nodes, "same", torch.ones(3, H, d, dtype=torch.bfloat16, device="cuda"), big[5:8], own_tokens=own,
                  lse=lse[5:8], workspace=ws)
    for t in (big, lse):
        assert (t[:5] == 7.0).all() and (t[8:] == 7.0).all() and not (t[5:8] == 7.0).any()
    pb, off, _ = kv.layout()
    before = kv.pool.clone()
    x = _dev(_bf(w.rng, 2, H, d))
    kv.write_tokens([(1, 1)], [200], x, x, [2])
    kv.status()
    changed = (kv.pool != before).nonzero().flatten().cpu().numpy()
    page = kv.entry_pages(1, 1)[1]
    scales = range(0)
    if fp8:
        at = kv.scale_offset() + page * 2 * H * 4
        scales = range(at, at + 2 * H * 4)
    own_bytes = np.array([off + page * pb <= i < off + (page + 1) * pb or i in scales for i in changed])
    assert changed.size and own_bytes.all()


def test_two_threads_with_a_handle_each(cuda_lib):
    """Calls of two threads at once, on their own handles and streams, give what one
    thread's calls give."""
    import threading

    import torch
    worlds = [_World(cuda_lib, 2, 64, 300, 1, fp8=fp8, seed=23 + fp8, pages=40) for fp8 in (False, True)]
    for w in worlds:
        for c in range(4):
            w.add(c, 1)

    def steps(w, out):
        kv, gen = w.kv, torch.Generator(device="cuda").manual_seed(5)
        X = torch.randn(300, 128, generator=gen, device="cuda").bfloat16()
        W = torch.randn(128, 128, generator=gen, device="cuda").bfloat16()
        pos = torch.arange(900, device="cuda", dtype=torch.int32).view(300, 3)
        Y, O = torch.empty_like(X), torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
        nodes = [(3, 1)]
        ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "same", [300])), dtype=torch.uint8, device="cuda")
        for i in range(60):
            M = (1, 20, 300)[i % 3]
            kv.linear_bias(X[:M], W, Y[:M], act="silu")
            kv.rotary(pos[:M], Y[:M].view(M, 2, 64))
            kv.write_tokens([(3, 1)], [i], Y[:1].view(1, 2, 64), Y[:1].view(1, 2, 64))
            kv.token_attn(nodes, "same", Y[:1].view(1, 2, 64), O, own_tokens=[300], workspace=ws)
            out.append((Y[:M].clone(), O.clone()))

    def run(w, out, errors):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                steps(w, out)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    torch.cuda.synchronize()
    pools, errors, alone, together = [w.kv.pool.clone() for w in worlds], [], [[], []], [[], []]
    for w, out in zip(worlds, alone):
        run(w, out, errors)
    torch.cuda.synchronize()
    for w, p in zip(worlds, pools):
        w.kv.pool.copy_(p)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(w, out, errors)) for w, out in zip(worlds, together)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not errors and all(len(o) == 60 for o in together)
    for a, b in zip(alone, together):
        for (y, o), (yy, oo) in zip(a, b):
            assert torch.equal(y, yy) and torch.equal(o, oo)
    for w in worlds:
        w.kv.status()


def test_chained_launches_wait_for_events(cuda_lib):
    """A launch that may start before the kernel ahead of it in its stream has ended
    still starts behind an event of another stream, whose work is late."""
    import torch
    w = _World(cuda_lib, 2, 64, 200, 1, seed=25)
    w.add(0, 1)
    kv, other = w.kv, torch.cuda.Stream()
    W = torch.eye(128, device="cuda").bfloat16()
    pos = torch.zeros(300, 3, dtype=torch.int32, device="cuda")
    K = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    own, O = [200], torch.empty_like(K)
    ws = torch.empty(max(1, kv.token_attn_workspace([(0, 1)], "same", own)), dtype=torch.uint8, device="cuda")
    for M in (1, 40, 300):
        X, T = (torch.zeros(M, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        Y, Z = torch.empty_like(X), torch.empty_like(X)
        for i in range(1, 9):
            here = torch.cuda.current_stream()
            other.wait_stream(here)
            with torch.cuda.stream(other):
                torch.cuda._sleep(200000)
                X.fill_(float(i))
                K.fill_(float(i))
                kv.linear_bias(X, W, T)
            kv.linear_bias(Z.zero_(), W, Y)             # a kernel just ahead of the wait
            here.wait_stream(other)
            kv.linear_bias(T, W, Y)
            kv.rotary(pos[:M], Y.view(M, 2, 64), Qout=Z.view(M, 2, 64))
            kv.write_tokens([(0, 1)], [0], K, K)
            kv.token_attn([(0, 1)], "same", K, O, own_tokens=[1], workspace=ws)
            assert (T == i).all() and (Y == i).all() and (Z == i).all() and (O == i).all(), (M, i)
    kv.status()
