"""The dense layer with bias, each form by sizes that reach it: results against a
64-bit layer, and waits that run out.

Tolerance per element: u |ref| (u = 2^-8, half a bf16 step) for the rounding, 2^-14 |ref| for
the activation, and (2 K + 16) 2^-23 (sum |a||w| + |b| + |r|) for K fp32 additions that
may truncate.
"""
import math

import pytest

from dense_forms import FORMS, LONG, SMS, form_of, name

pytestmark = pytest.mark.gpu


@pytest.fixture()
def kv(cuda_lib):
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count != SMS:
        pytest.skip(f"the sizes are chosen for {SMS} SMs")
    pool = torch.empty(4096 + 2 * 128 * 64 * 2, dtype=torch.uint8, device="cuda")
    return cuda_lib.KVCache(1, 64, 1, 1, pool=pool)


def _activate(y, act):
    import torch
    if act == "gelu_tanh":
        return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    if act == "gelu_erf":
        return y * torch.special.erfc(-y / math.sqrt(2)) / 2
    return y * torch.special.expit(y) if act == "silu" else y


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("form", list(FORMS), ids=name)
def test_form(kv, form, act):
    """Random data, with a bias, a residual and columns beside every row; the result in
    place of the residual; and neither bias nor residual."""
    import torch
    for i, (M, K, N) in enumerate(FORMS[form]):
        assert form_of(kv.lib, M, K, N) == form
        gen = torch.Generator(device="cuda").manual_seed(1000 * M + K + i)

        def normal(rows, cols, pad, scale=1.0):
            wide = torch.full((rows, cols + pad), math.nan, device="cuda").bfloat16()
            wide[:, :cols] = torch.randn(rows, cols, generator=gen, device="cuda") * scale
            return wide[:, :cols]
        A, W, R = normal(M, K, 24), normal(N, K, 0, K ** -0.5), normal(M, N, 40)
        bias = normal(1, N, 0)[0]
        y = A.double() @ W.double().T
        size = A.double().abs() @ W.double().abs().T

        def check(got, ref, size, what):
            tol = (2.0 ** -8 + 2.0 ** -14) * ref.abs() + (2 * K + 16) * 2.0 ** -23 * size
            bad = ~((got.double() - ref).abs() <= tol)
            assert not bad.any(), (f"{what}, {M} x {K} x {N}: {int(bad.sum())} of {bad.numel()} off, the first at "
                                   f"{bad.nonzero()[0].tolist()}")
        ref = _activate(y + bias.double(), act) + R.double()
        full = size + bias.double().abs() + R.double().abs()
        big = torch.full((M + 260, N + 8), 7.0, device="cuda").bfloat16()
        Y = big[130:130 + M, :N]
        kv.linear_bias(A, W, Y, bias=bias, R=R, act=act)
        check(Y, ref, full, "bias and residual")
        assert (big[:130] == 7).all() and (big[130 + M:] == 7).all() and (big[:, N:] == 7).all()
        kv.linear_bias(A, W, R, bias=bias, R=R, act=act)
        check(R, ref, full, "in place")
        Y = torch.full((M, N), 7.0, device="cuda").bfloat16()
        kv.linear_bias(A, W, Y, act=act)
        check(Y, _activate(y, act), size, "alone")
        again = torch.empty_like(Y)
        kv.linear_bias(A, W, again, act=act)
        assert torch.equal(Y, again)
        kv.status()


@pytest.mark.parametrize("form", list(LONG), ids=name)
def test_form_reports_a_wait_that_runs_out(kv, cuda_lib, form):
    """The call that gave up is reported, whatever its cluster, and the next is right."""
    import torch
    M, K, N = LONG[form]
    assert form_of(kv.lib, M, K, N) == form
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
    assert (y == K * 2.0 ** -10).all()
