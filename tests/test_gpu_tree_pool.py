"""Draft trees and the state cache over a pool: slots that several entries share, captured and replayed
calls on new inputs, and pools whose offsets pass 32 bits."""
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from test_gpu_tree import DEV, DTYPES, FORMATS, IDS, RULES, bushy, problem

pytestmark = pytest.mark.gpu


def gates(x, rule):
    return (x["alpha"], x["beta"]) if rule == "delta" else (x["decay"],)


def tree(x, rule, parents, pool, slots, o):
    (binding.gdn_decode_tree if rule == "delta" else binding.gdn_decay_decode_tree)(
        x["q"], x["k"], x["v"], *gates(x, rule), parents, pool, slots, o)


def commit(x, rule, parents, accepted, pool, slots):
    (binding.gdn_tree_commit if rule == "delta" else binding.gdn_decay_tree_commit)(
        x["k"], x["v"], *gates(x, rule), parents, accepted, pool, slots)


def ids(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rule", RULES)
def test_sequences_that_continue_one_state(rule):
    """Verification reads only: several trees may start from the same slot."""
    x = {k: v.to(DEV) for k, v in problem(4, 12, 1, 3, torch.bfloat16, 800).items()}
    p = bushy(4, 12).to(DEV)
    shared, apart = torch.zeros_like(x["v"]), torch.zeros_like(x["v"])
    tree(x, rule, p, x["pool"], ids(5, 5, 2, 5), shared)
    pool = x["pool"][[5, 5, 2, 5]].contiguous()
    tree(x, rule, p, pool, None, apart)
    assert torch.equal(shared, apart)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_one_snapshot_for_many_slots(fmt):
    """A shared prefix: one state stored twice, one snapshot loaded into three slots."""
    pool = problem(2, 1, 1, 2, torch.float32, 810, n_slots=6)["pool"].to(DEV)
    codes = torch.zeros(4, 2, 128, 128, dtype=torch.int8, device=DEV).view(FORMATS[fmt])
    scales = torch.zeros(4, 2, 128, device=DEV)
    before = pool.clone()
    binding.gdn_state_store(pool, ids(3, 3, 1), codes, scales, ids(0, 2, 3))
    assert torch.equal(codes[0].view(torch.int8), codes[2].view(torch.int8)) and torch.equal(scales[0], scales[2])
    binding.gdn_state_load(codes, scales, ids(0, 2, 0, 3), pool, ids(0, 4, 5, 2))
    want = codes[0].float() * scales[0][..., None]
    assert all(torch.equal(pool[s], want) for s in (0, 4, 5))
    assert torch.equal(pool[2], codes[3].float() * scales[3][..., None])
    assert torch.equal(pool[[1, 3]], before[[1, 3]])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rule", RULES)
def test_a_captured_step(dtype, rule):
    """Load, verification, commit, one token and a snapshot in one graph, replayed on new inputs."""
    a, b = (problem(3, 7, 1, 3, dtype, s) for s in (820, 821))
    a["decay"] = b["decay"]
    x = {k: v.to(DEV) for k, v in a.items()}
    p, acc = bushy(3, 7).to(DEV), ids(6, 2, 4)
    last = {k: v[:, 0].contiguous().to(DEV) for k, v in problem(3, 1, 1, 3, dtype, 822).items() if k in ("q", "k", "v", "alpha", "beta")}
    codes, scales = torch.zeros(2, 3, 128, 128, dtype=torch.int8, device=DEV), torch.zeros(2, 3, 128, device=DEV)
    o, o1 = torch.zeros_like(x["v"]), torch.zeros_like(last["v"])

    def step():
        binding.gdn_state_load(codes, scales, ids0, x["pool"], slot0)
        tree(x, rule, p, x["pool"], x["slots"], o)
        commit(x, rule, p, acc, x["pool"], x["slots"])
        if rule == "delta":
            binding.gdn_decode_step_slots(last["q"], last["k"], last["v"], last["alpha"], last["beta"], x["pool"], x["slots"], o1)
        else:
            binding.gdn_decay_decode_step_slots(last["q"], last["k"], last["v"], x["decay"], x["pool"], x["slots"], o1)
        binding.gdn_state_store(x["pool"], x["slots"], codes, scales, rows)

    ids0, slot0, rows = ids(0), x["slots"][:1].clone(), ids(0, 1, -1)

    def put(d):
        for k in x:
            x[k].copy_(d[k].to(DEV))
        slot0.copy_(x["slots"][:1])
        binding.gdn_state_store(x["pool"], x["slots"][:1], codes, scales, ids0)
        o.zero_()

    put(b)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (o, o1, x["pool"], codes, scales)]
    put(a)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(2):
        put(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip((o, o1, x["pool"], codes, scales), want))


def test_past_32_bit_offsets():
    """Pool and cache of more than 2^31 values: their last rows, against the same calls on small ones."""
    Hv, n = 48, (1 << 31) // (48 * 128 * 128) + 3
    x = {k: v.to(DEV) for k, v in problem(1, 5, 16, 6, torch.bfloat16, 830, n_slots=1).items()}
    x["v"], x["alpha"], x["beta"] = (x[k].repeat_interleave(8, dim=2).contiguous() for k in ("v", "alpha", "beta"))
    x["k"], x["q"] = x["k"].contiguous(), x["q"].contiguous()
    state = x["pool"].repeat_interleave(8, dim=1).contiguous()
    p, acc = torch.tensor([[-1, 0, 1, 1, 3]], dtype=torch.int32, device=DEV), ids(4)
    pool = torch.empty((n, Hv, 128, 128), device=DEV)
    codes, scales = torch.empty((n, Hv, 128, 128), dtype=torch.int8, device=DEV), torch.empty((n, Hv, 128), device=DEV)
    pool[n - 1], pool[n - 2] = state[0], 5.0
    outs = []
    for P, C, S, at in ((pool, codes, scales, n - 1),
                        (state.clone(), torch.empty_like(codes[:1]), torch.empty_like(scales[:1]), 0)):
        o, row = torch.zeros_like(x["v"]), ids(at)
        tree(x, "delta", p, P, row, o)
        commit(x, "delta", p, acc, P, row)
        binding.gdn_state_store(P, row, C, S, row)
        outs.append([o, P[at].clone(), C[at].clone(), S[at].clone()])
        P[at] = 0.0
        binding.gdn_state_load(C, S, row, P, row)
        outs[-1].append(P[at].clone())
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert (pool[n - 2] == 5.0).all()
