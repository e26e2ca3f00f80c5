"""The dense layer with bias, each form by sizes that reach it: waits that run out."""
import pytest

from dense_forms import LONG, SMS, form_of, name

pytestmark = pytest.mark.gpu


@pytest.fixture()
def kv(cuda_lib):
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count != SMS:
        pytest.skip(f"the sizes are chosen for {SMS} SMs")
    pool = torch.empty(4096 + 2 * 128 * 64 * 2, dtype=torch.uint8, device="cuda")
    return cuda_lib.KVCache(1, 64, 1, 1, pool=pool)


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
