"""Pins of the single-token oracle: against the chunk oracle it must agree with,
closed forms, finite differences and torch's own functions."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import block as oblock
from oracle import quant
from oracle import token as otok


def test_linear_bias_is_torchs_layer():
    g = torch.Generator().manual_seed(1)
    x, w, b, r = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 7), (6, 7), (6,), (5, 6)))
    y = torch.nn.functional.linear(x, w, b)
    f = torch.nn.functional
    for act, fn in (("none", lambda v: v), ("gelu_tanh", lambda v: f.gelu(v, approximate="tanh")),
                    ("gelu_erf", f.gelu), ("silu", f.silu)):
        got = otok.linear_bias(x.numpy(), w.numpy(), b.numpy(), r.numpy(), act)
        np.testing.assert_allclose(got, (fn(y) + r).numpy(), rtol=1e-12, atol=1e-13)
    assert otok.activation(np.array([-1e4, 1e4]), "silu").tolist() == [0.0, 1e4]


@pytest.mark.parametrize("d", [64, 128])
def test_rotary_of_a_chunk_is_the_blocks(d):
    rng = np.random.default_rng(2)
    grid, chunk = (2, 3, 4), 5
    x = rng.standard_normal((24, 2, d))
    t = np.arange(24)
    pos = np.stack([chunk * 2 + t // 12, t // 4 % 3, t % 4], 1)
    want = oblock.apply_rope(x, oblock.rope_angles(chunk, *grid, d))
    np.testing.assert_allclose(otok.rotary(x, pos, oblock.rope_groups(d)), want, rtol=0, atol=1e-12)


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("ladder", ["axis", "ladder"])
def test_rotary_inverse_is_its_gradient(layout, ladder):
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((3, 2, 64)), rng.standard_normal((3, 2, 64))
    pos = rng.integers(-50, 50, (3, 3))
    turn = lambda v, **k: otok.rotary(v, pos, (10, 9, 8), 100.0, layout, ladder, **k)  # noqa: E731
    np.testing.assert_allclose(turn(turn(x), inverse=True), x, rtol=0, atol=1e-12)
    back = turn(g, inverse=True)   # d <g, turn(x)> / dx, against differences
    for at in ((0, 0, 0), (1, 1, 31), (2, 0, 33), (2, 1, 63)):
        e = np.zeros_like(x)
        e[at] = 1e-4
        diff = ((turn(x + e) - turn(x - e)) * g).sum() / 2e-4
        assert abs(diff - back[at]) < 1e-8
    # the five pairs past the axes' 27 are copied
    keep = np.arange(54, 64) if layout == "interleaved" else np.r_[27:32, 59:64]
    assert np.array_equal(turn(x)[..., keep], x[..., keep])


def test_rotary_scores_depend_on_distance():
    rng = np.random.default_rng(4)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    for layout in ("interleaved", "halves"):
        turn = lambda v, p: otok.rotary(v, np.array([p]), (12, 10, 10), layout=layout)  # noqa: E731
        a = (turn(q, (7, 2, 3)) * turn(k, (4, 1, 1))).sum()
        b = (turn(q, (107, 32, 13)) * turn(k, (104, 31, 11))).sum()
        assert abs(a - b) < 1e-10


def test_fp8_entry_written_whole_is_the_append():
    x = oblock.bf16_round(np.random.default_rng(5).standard_normal((200, 2, 64)))
    ent = otok.Fp8Entry(200, 2, 64)
    ent.write(0, x)
    codes, scales = quant.quantize_entry(x)
    assert np.array_equal(ent.codes, codes) and np.array_equal(ent.scales, scales)


def test_fp8_entry_token_by_token():
    rng = np.random.default_rng(6)
    x = oblock.bf16_round(rng.standard_normal((140, 2, 64)) * np.exp(rng.standard_normal((140, 1, 1))))
    x[0] = 0.0  # a zero first token leaves no scale behind
    ent, scales = otok.Fp8Entry(140, 2, 64), []
    for t in range(140):
        ent.write(t, x[t:t + 1])
        scales.append(ent.scales.copy())
    assert all((b[0] >= a[0]).all() for a, b in zip(scales[1:128], scales[2:128]))  # only grows
    whole = otok.Fp8Entry(140, 2, 64)
    whole.write(0, x)
    assert np.array_equal(ent.scales, whole.scales)      # amax of the page in the end
    # every token within a half step of its first rounding, and of later ones: each
    # time the scale grows a kept value moves by at most 2^-4 of itself or half the
    # smallest step (2^-10) of the new scale
    grown = sum((b > a).any() for a, b in zip(scales, scales[1:])) + 1
    err = np.abs(ent.values(140) - x)
    top = np.repeat(ent.scales, 128, 0)[:140][:, :, None]
    assert (err <= grown * (np.abs(x) * 2.0 ** -4 * 1.1 + top * 2.0 ** -10)).all()
    # a rewrite with the same token changes nothing
    before = ent.codes.copy()
    ent.write(139, x[139:])
    assert np.array_equal(ent.codes, before) and ent.written == 140


def test_token_attention_is_a_row_of_the_chunks():
    rng = np.random.default_rng(7)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((50, 4, 64)), rng.standard_normal((50, 4, 64))
    want = oatt.attend(q, k, v)
    for i in range(3):
        o, lse, a = otok.token_attention(q[i], k, v)
        np.testing.assert_allclose(o, want[i], rtol=0, atol=1e-13)
        assert (np.abs(o) <= a + 1e-15).all()
    # grouped heads: each K/V head serves two query heads
    o, lse, _ = otok.token_attention(q[0], k[:, :2], v[:, :2])
    np.testing.assert_allclose(o, oatt.attend(q[:1], k[:, [0, 0, 1, 1]], v[:, [0, 0, 1, 1]])[0], atol=1e-13)
    # joined halves by their log-sum-exp
    (o1, l1, _), (o2, l2, _) = (otok.token_attention(q[0], k[s], v[s]) for s in (slice(0, 20), slice(20, 50)))
    o, lse, _ = otok.token_attention(q[0], k, v)
    w1, w2 = np.exp(l1 - lse)[:, None], np.exp(l2 - lse)[:, None]
    np.testing.assert_allclose(w1 * o1 + w2 * o2, o, atol=1e-13)
    o, lse, _ = otok.token_attention(q[0], k[:0], v[:0])
    assert not o.any() and np.isneginf(lse).all()


def test_node_tokens_cut_the_own_entry():
    ents = {(c, l): (np.full((4, 1, 2), 10 * c + l), np.full((4, 1, 2), -c)) for c in range(3) for l in range(3)}
    k, _ = otok.node_tokens((2, 1), "progressive", 0, ents, None, 3)
    assert k[:, 0, 0].tolist() == [0] * 4 + [10] * 4 + [21] * 3
    k, _ = otok.node_tokens((0, 1), "progressive", 0, ents, None, 0)
    assert k.shape == (0, 1, 2)
