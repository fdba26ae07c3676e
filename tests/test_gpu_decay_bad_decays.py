"""A decay that is NaN or negative is seen: the outputs and states of its head are NaN, in every
call that takes one; the other heads keep their values."""
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from test_gpu_decay import DEV, DTYPES, IDS, backward, dev, forward, inputs, upstream
from test_gpu_tree import bushy, commit, problem, verify

pytestmark = pytest.mark.gpu
BAD = [float("nan"), -0.5, -float("inf")]


def apart(got, want, dim, bad=1):
    """Head `bad` is NaN throughout, the others as they were."""
    rest = [h for h in range(got.shape[dim]) if h != bad]
    assert torch.isnan(got.select(dim, bad).float()).all()
    assert torch.equal(got.index_select(dim, torch.tensor(rest, device=got.device)),
                       want.index_select(dim, torch.tensor(rest, device=got.device)))


def spoil(d, value):
    return {**d, "decay": torch.where(torch.arange(d["decay"].numel()) == 1, torch.tensor(value), d["decay"])}


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("T", [30, 200, 1130])
def test_prefill(dtype, value, T):
    d = inputs((1, T), 1, 3, dtype, 600 + T)
    for got, want in zip(forward(spoil(d, value)), forward(d)):
        apart(got, want, 2 if got.dim() == 4 and got.shape[1] == T else 1)
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", BAD)
def test_packed_prefill(dtype, value):
    d = inputs((100,), 1, 3, dtype, 610, states=3)
    cu = torch.tensor([0, 70, 70, 100], dtype=torch.int32, device=DEV)
    out = []
    for c in (spoil(d, value), d):
        x = dev(c)
        o, SF = torch.empty_like(x["v"]), torch.empty((3, 3, 128, 128), device=DEV)
        binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, cu)
        assert torch.equal(SF[1], x["S0"][1])                # no tokens: the state passes through
        out.append((o, SF[[0, 2]]))
    for got, want in zip(*out):
        apart(got, want, 1)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("T", [30, 200])
def test_gradients(dtype, value, T):
    d = inputs((1, T), 3, 3, dtype, 620 + T)
    dO, dSF = upstream(d, 621)
    for got, want in zip(backward(spoil(d, value), dO, dSF), backward(d, dO, dSF)):
        apart(got, want, 2 if got.shape[1] == T else 1)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", BAD)
def test_decode(dtype, value):
    d = inputs((3,), 1, 3, dtype, 630)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    out = []
    for c in (spoil(d, value), d):
        x = dev(c)
        pool, o, o2, S = x["S0"].clone(), torch.empty_like(x["v"]), torch.empty_like(x["v"]), torch.empty_like(x["S0"])
        binding.gdn_decay_decode_step(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, S)
        binding.gdn_decay_decode_step_slots(x["q"], x["k"], x["v"], x["decay"], pool, slots, o2)
        out.append((o, S, o2, pool))
    for got, want in zip(*out):
        apart(got, want, 1)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", BAD)
def test_trees(dtype, value):
    d = problem(2, 12, 1, 3, dtype, 640)
    d["slots"] = torch.tensor([3, 1], dtype=torch.int32)
    parents = bushy(2, 12)
    parents[:, 9:] = -2                                      # padding rows stay as they were
    got, want = verify(spoil(d, value), parents, "decay"), verify(d, parents, "decay")
    apart(got[:, :9], want[:, :9], 2)
    assert (got[:, 9:] == 9.0).all()
    accepted = torch.tensor([5, 8], dtype=torch.int32)
    got, want = commit(spoil(d, value), parents, accepted, "decay"), commit(d, parents, accepted, "decay")
    apart(got[[3, 1]], want[[3, 1]], 1)
    rest = [0, 2, 4]
    assert torch.equal(got[rest], want[rest])
