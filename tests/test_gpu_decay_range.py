"""Constant-decay linear attention with large and small values: a chunk's scores carry powers of a
strong decay, and neither they nor what the causal mask hides may leave the range of an fp32."""
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from test_gpu_decay import DEV, DTYPES, IDS, backward, check_backward, check_forward, dev, forward, inputs, upstream

pytestmark = pytest.mark.gpu
STRONG = torch.tensor([0.0, 0.02, 0.3, 0.334, 0.34, 0.5, 0.64, 0.65])


def scaled(d, **exps):
    return {n: (t if t is None or n not in exps else t * 2.0 ** exps[n]) for n, t in d.items()}


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [64, 150, 1130])
@pytest.mark.parametrize("eq,ek,ev", [(14, 14, 2), (16, 16, 0), (0, 0, 30), (20, 20, 24), (-14, -14, 0), (-16, 20, -20), (-24, -24, 4), (24, -36, -26)])
def test_prefill(dtype, T, eq, ek, ev):
    d = scaled(inputs((1, T), 1, 8, dtype, 400 + T), q=eq, k=ek, v=ev, S0=ek + ev)
    d["decay"] = STRONG
    check_forward(d, *forward(d), f"T={T} 2^({eq},{ek},{ev})")
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [64, 150])
@pytest.mark.parametrize("eq,ek,ev,eg", [(0, 0, 5, 24), (14, 14, 0, 16), (10, 10, 16, 16), (-10, -10, 0, -16)])
def test_gradients(dtype, T, eq, ek, ev, eg):
    """A loss scale, and operands that are not normalised."""
    d = scaled(inputs((1, T), 2, 8, dtype, 420 + T), q=eq, k=ek, v=ev, S0=ek + ev)
    d["decay"] = STRONG[1:].repeat(2)[:8].contiguous()
    dO, dSF = upstream(d, 421)
    dO, dSF = dO * 2.0 ** eg, dSF * 2.0 ** (eq + eg)
    check_backward(d, dO, dSF, backward(d, dO, dSF), f"T={T} 2^({eq},{ek},{ev},{eg})")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_a_large_later_token_leaves_the_earlier_rows(dtype):
    """Scores above the diagonal are large and masked: the rows before are those without them."""
    d = inputs((1, 64), 1, 8, dtype, 440)
    d["decay"] = STRONG
    o, _ = forward(d, S_final=None)
    d["k"][:, 11] *= 2.0 ** 40
    big, _ = forward(d, S_final=None)
    assert torch.equal(o[:, :11], big[:, :11])
    check_forward(d, big, None, "large key")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_packed_prefill(dtype):
    n = [50, 130, 1, 70]
    d = scaled(inputs((sum(n),), 1, 8, dtype, 441, states=4), q=16, k=16, S0=16)
    d["decay"] = STRONG
    x = dev(d)
    cu = torch.tensor([0, 50, 180, 181, 251], dtype=torch.int32)
    o, SF = torch.empty_like(x["v"]), torch.empty((4, 8, 128, 128), device=DEV)
    binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, cu.to(DEV))
    for i in range(4):
        a, e = int(cu[i]), int(cu[i + 1])
        part = {k: (v[None, a:e] if k in ("q", "k", "v") else v) for k, v in d.items()}
        part["S0"] = d["S0"][i:i + 1]
        check_forward(part, o[None, a:e], SF[i:i + 1], f"sequence {i}")
