"""Forms of the decay walk's calls: no end state with one chunk and with segments, packed calls of
one chunk, short prompts packed against alone."""
import numpy as np
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from test_gpu_decay import DEV, DTYPES, IDS, backward, check_backward, check_forward, dev, forward, inputs, upstream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [1, 40, 64])
@pytest.mark.parametrize("s0", [True, False])
def test_one_chunk_without_an_end_state(dtype, T, s0):
    d = inputs((2, T), 2, 6, dtype, 450 + T, s0=s0)
    o, _ = forward(d, S_final=None)
    check_forward(d, o, None, f"T={T}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Hqk,Hv,T", [(1, 2, 1130), (12, 36, 1800)])
def test_segments_without_an_end_state(dtype, Hqk, Hv, T):
    """A prompt that is scored and not continued; with a head before the segments, and without."""
    d = inputs((1, T), Hqk, Hv, dtype, 460 + Hv)
    assert binding.decay_fwd_workspace_bytes(1, T, Hv, dtype) > 0
    o, _ = forward(d, S_final=None)
    check_forward(d, o, None, f"T={T}")
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Hqk,Hv,T", [(1, 1, 50), (1, 4, 1130), (6, 12, 1800)])
def test_gradients_without_dS0(dtype, Hqk, Hv, T):
    d = inputs((1, T), Hqk, Hv, dtype, 470 + Hv)
    dO, dSF = upstream(d, 471)
    check_backward(d, dO, dSF, backward(d, dO, dSF, with_dS0=False), f"T={T}")


def packed(d, lengths, end=True):
    x = dev(d)
    N = len(lengths)
    cu = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device=DEV)
    o = torch.full_like(x["v"], 7.0)
    SF = torch.full((N, *x["v"].shape[1:2], 128, 128), float("nan"), device=DEV) if end else None
    binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, cu)
    torch.cuda.synchronize()
    return o, SF


def sequence(d, lengths, i):
    a = sum(lengths[:i])
    part = {k: (v[None, a:a + lengths[i]].contiguous() if k in ("q", "k", "v") else v) for k, v in d.items()}
    part["S0"] = None if d["S0"] is None else d["S0"][i:i + 1].contiguous()
    return part


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("lengths", [[20, 0, 1, 30], [64], [40], [1] * 9])
@pytest.mark.parametrize("end", [True, False])
def test_packed_call_of_one_chunk(dtype, lengths, end):
    """All sequences together are no longer than a chunk."""
    total = sum(lengths)
    d = inputs((total + 3 if total < 61 else total,), 1, 3, dtype, 480 + total, states=len(lengths))
    o, SF = packed(d, lengths, end)
    assert (o[total:] == 7.0).all()
    a = 0
    for i, n in enumerate(lengths):
        if n == 0:
            assert not end or torch.equal(SF[i].cpu(), d["S0"][i])
            continue
        check_forward(sequence(d, lengths, i), o[None, a:a + n], SF[i:i + 1] if end else None, f"sequence {i} of {n}")
        a += n


def test_a_short_prompt_packed_is_as_exact_as_alone():
    """bf16: the scores of a sequence of one chunk have two pieces, whatever the call packs beside it."""
    lengths = [64, 200, 1, 37, 63, 90, 5]
    d = inputs((sum(lengths),), 2, 6, torch.bfloat16, 490, states=len(lengths))
    o, SF = packed(d, lengths)
    a = 0
    for i, n in enumerate(lengths):
        if n <= 64:
            alone = forward(sequence(d, lengths, i))
            assert torch.equal(o[None, a:a + n], alone[0]) and torch.equal(SF[i:i + 1], alone[1]), n
        a += n
