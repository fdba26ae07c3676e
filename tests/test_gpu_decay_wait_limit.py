"""A wait of the bf16 decay kernels that runs out ends the launch with an error status, and the next
call is right.  The wait is that of the second of two launches for the states of the first: with one
to three heads of 2^19 tokens those are a walk of 400 microseconds and more."""
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from test_gpu_decay import DEV, check_forward, forward, inputs

pytestmark = pytest.mark.gpu
T, SHORT = 1 << 19, 40                    # tokens; microseconds


def rows(g, H):
    return (torch.randn(1, T, H, 128, generator=g, device=DEV) / 11).bfloat16()


def gave_up(call):
    """call under the short limit: reported once, and read back clear."""
    with binding.decay_wait_limit(SHORT):
        call()
    assert binding.device_status() == "GDN_ERR_TIMEOUT"
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (1, 3)])
def test_prefill(Hqk, Hv):
    g = torch.Generator(device=DEV).manual_seed(664)
    q, k, v = rows(g, Hqk), rows(g, Hqk), rows(g, Hv)
    lam = torch.tensor([0.99, 0.3, 1.0][:Hv], device=DEV)
    o, S = torch.empty_like(v), torch.empty(1, Hv, 128, 128, device=DEV)
    call = lambda: binding.gdn_decay_fwd(q, k, v, lam, None, o, S)  # noqa: E731
    call()
    assert binding.device_status() == "GDN_OK"
    want = o.clone(), S.clone()
    for _ in range(3):
        gave_up(call)
        d = inputs((2, 200), 2, 6, torch.bfloat16, 665)      # another call takes the same SMs
        check_forward(d, *forward(d), "after")
        call()
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
        assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (1, 2)])
def test_gradients(Hqk, Hv):
    """Rows of bf16, and of fp32 for shared heads."""
    g = torch.Generator(device=DEV).manual_seed(666)
    q, k, v, dO = rows(g, Hqk), rows(g, Hqk), rows(g, Hv), rows(g, Hv)
    lam = torch.tensor([0.99, 0.4][:Hv], device=DEV)
    out = [torch.empty_like(t) for t in (q, k, v)] + [torch.empty(1, Hv, 128, 128, device=DEV)]
    call = lambda: binding.gdn_decay_bwd(q, k, v, lam, None, dO, None, *out)  # noqa: E731
    call()
    assert binding.device_status() == "GDN_OK"
    want = [t.clone() for t in out]
    for _ in range(2):
        gave_up(call)
        call()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert binding.device_status() == "GDN_OK"
