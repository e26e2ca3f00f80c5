"""What the single-token operators keep of their operands, where a tolerance for
long sums would hide a loss: the weights of attention over few tokens.

Tolerances, per element (u = 2^-8, half a bf16 step): u |ref| for the one rounding,
and for attention (w + 2^-18) A with A the weighted mean of |V|, w what a weight may lose.
"""
import numpy as np
import pytest

from oracle import block as oblock
from oracle import token as otok
from test_gpu_token import U, _cache, _dev, _within
from wave_testlib import torch_to_f64

pytestmark = pytest.mark.gpu


def _two_kinds(T, H, d):
    """Keys of score 0 and, every other one, of score -t (t a head's own) for the query
    (sqrt(d), 0, ...); values 1 and about -e^t, so that the sum nearly cancels and
    what a weight loses is all that is left."""
    t = oblock.bf16_round(np.linspace(0.013, 2.9, H))
    k, v = np.zeros((T, H, d)), np.ones((T, H, d))
    k[1::2, :, 0] = -t
    v[1::2] = -oblock.bf16_round(np.exp(t)[:, None] * (1 + np.arange(d) / 4096.0))
    return k, v


def _attend(wave, k, v, q, own):
    """O of len(own) tokens of one entry, each seeing its first own[i] tokens."""
    import torch
    T, H, d = k.shape
    kv = _cache(wave, H, d, T, 1, pages=(T + 127) // 128)
    kv.append(0, 1, _dev(k), _dev(v))
    nodes = [(0, 1)] * len(own)
    O = torch.empty(len(own), q.shape[1], d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(1, kv.token_attn_workspace(nodes, "same", own, q_heads=q.shape[1])), dtype=torch.uint8,
                     device="cuda")
    kv.token_attn(nodes, "same", _dev(q), O, own_tokens=own, workspace=ws)
    kv.status()
    return torch_to_f64(O)


@pytest.mark.parametrize("T", [2, 384])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 16])
def test_attention_keeps_its_weights(cuda_lib, T, d, group):
    """bf16 pool: a weight's leading 8 bits and the next 8 reach the sum (w = 2^-15: the
    rest after the first 8 is below 2^-7 of the weight, its rounding 2^-8 of that)."""
    H = 24
    k, v = _two_kinds(T, H, d)
    own = [T, T - 1] if group == 1 else [T]
    q = np.zeros((len(own), H * group, d))
    q[..., 0] = oblock.bf16_round(np.float64(d ** 0.5))
    got = _attend(cuda_lib, k, v, q, own)
    for i, n in enumerate(own):
        o, _, a = otok.token_attention(q[i], k[:n], v[:n])
        _within(got[i], o, U * np.abs(o) + (2.0 ** -15 + 2.0 ** -18) * a, f"{n} of {T} tokens")


@pytest.mark.parametrize("T", [2, 384])
@pytest.mark.parametrize("at", [0, 1])
def test_attention_takes_infinite_values(cuda_lib, T, at):
    """An infinite V that is seen, at a weight of exactly 1 and at one with more bits
    than a bf16 holds, gives that infinity."""
    k, v = _two_kinds(T, 24, 64)
    v[at, :, :32], v[at, :, 32:] = np.inf, -np.inf
    q = np.zeros((1, 24, 64))
    q[..., 0] = 8.0
    got = _attend(cuda_lib, k, v, q, [T])[0]
    assert np.isposinf(got[:, :32]).all() and np.isneginf(got[:, 32:]).all()


@pytest.mark.parametrize("M", [16, 400])
@pytest.mark.parametrize("act,most", [("gelu_erf", 12.5), ("gelu_tanh", 10.0), ("silu", 80.0)])
def test_activations_keep_their_tails(cuda_lib, act, most, M):
    """One product a result, so that no sum's tolerance hides the activation: every
    result is good to 2^-14 of itself and the one rounding, whatever its size."""
    import torch
    kv = _cache(cuda_lib)
    x = oblock.bf16_round(np.linspace(-most, most, 2000))
    w = np.zeros((2000, 8))
    w[:, 0] = x
    a = np.zeros((M, 8))
    a[:, 0] = 1.0
    Y = torch.empty(M, 2000, dtype=torch.bfloat16, device="cuda")
    kv.linear_bias(_dev(a), _dev(w), Y, act=act)
    kv.status()
    ref = np.broadcast_to(otok.activation(x, act), (M, 2000))
    _within(torch_to_f64(Y), ref, (U + 2.0 ** -14) * np.abs(ref), act)
