"""GPU parity of the constant-decay linear attention: prefill, packed prefill, gradients, decode."""
import numpy as np
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from oracle import decay as ref
from decay_bounds import BF16, F32, check, out_bounds, state_bounds

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "fp32"]
LAMBDAS = [0.4, 0.93, 0.998, 0.71, 1.0, 0.85]


def lam_of(Hv, values=LAMBDAS):
    return torch.tensor([values[i % len(values)] for i in range(Hv)], dtype=torch.float32)


def inputs(lead, Hqk, Hv, dtype, seed, s0=True, states=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {"q": (r(*lead, Hqk, 128) / 11).to(dtype), "k": (r(*lead, Hqk, 128) / 11).to(dtype),
         "v": r(*lead, Hv, 128).to(dtype), "decay": lam_of(Hv)}
    d["S0"] = r(lead[0] if states is None else states, Hv, 128, 128) * 0.2 if s0 else None
    return d


def dev(d):
    return {k: (None if v is None else v.to(DEV)) for k, v in d.items()}


def forward(d, S_final="new", **kw):
    x = dev(d)
    o = torch.full_like(x["v"], float("nan"))
    B, T, Hv = x["v"].shape[:3]
    SF = torch.full((B, Hv, 128, 128), float("nan"), device=DEV) if S_final == "new" else S_final
    binding.gdn_decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, **kw)
    torch.cuda.synchronize()
    return o, SF


def check_forward(d, o, SF, what):
    lam = np.exp(np.maximum(np.log(np.maximum(d["decay"].double().numpy(), 1e-300)), -87.0))
    args = (d["q"], d["k"], d["v"], lam, d["S0"])
    (ro, rS), (mo, mS) = ref.decay_forward(*args), ref.decay_forward_majorant(*args)
    bf16, T = d["q"].dtype == torch.bfloat16, d["q"].shape[1]
    check(o, ro, mo, *out_bounds(bf16, T), f"{what} o")
    if SF is not None:
        check(SF, rS, mS, 0.0, state_bounds(bf16, T), f"{what} S_final")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 128, 200, 321])
def test_prefill(dtype, T):
    d = inputs((2, T), 2, 6, dtype, 10 + T)
    check_forward(d, *forward(d), f"T={T}")
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (3, 3), (1, 5)])
def test_prefill_in_segments(dtype, Hqk, Hv):
    """Few heads: segments, whose start states a launch of its own computes; ragged end."""
    d = inputs((1, 1130), Hqk, Hv, dtype, 40 + Hv)
    assert binding.decay_fwd_workspace_bytes(1, 1130, Hv, dtype) > 0
    check_forward(d, *forward(d), f"heads {Hqk}/{Hv}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("s0", [True, False])
def test_prefill_in_segments_behind_a_head(dtype, s0):
    """A quarter of the device's width in heads: the first launch walks the sequence's head too."""
    d = inputs((1, 1800), 12, 36, dtype, 46, s0=s0)
    check_forward(d, *forward(d), "head")
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_prefill_without_states(dtype):
    d = inputs((3, 130), 1, 3, dtype, 50, s0=False)
    check_forward(d, *forward(d), "no S0")
    o, _ = forward(d, S_final=None)
    check_forward(d, o, None, "no S_final")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [90, 700])
def test_prefill_at_the_ends_of_the_decay(dtype, T):
    """0 (as e^-87), heads that forget within a chunk (the scales' floor), and 1."""
    d = inputs((1, T), 1, 7, dtype, 60 + T)
    d["decay"] = torch.tensor([0.0, 1e-30, 0.02, 0.25, 0.34, 0.99999, 1.0])
    check_forward(d, *forward(d), "decay ends")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [70, 1130])
def test_prefill_in_place(dtype, T):
    d = inputs((1, T), 1, 2, dtype, 70)
    o, SF = forward(d)
    x = dev(d)
    o2 = torch.empty_like(x["v"])
    binding.gdn_decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], o2, x["S0"])
    assert torch.equal(o, o2) and torch.equal(SF, x["S0"])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_prefill_of_nothing(dtype):
    d = inputs((2, 0), 1, 2, dtype, 71)
    assert torch.equal(forward(d)[1].cpu(), d["S0"])
    d["S0"] = None
    assert torch.count_nonzero(forward(d)[1]).item() == 0
    d = inputs((0, 5), 1, 2, dtype, 72)
    forward(d)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_prefill_repeats_bit_for_bit(dtype):
    d = inputs((1, 900), 2, 4, dtype, 73)
    first = forward(d)
    for _ in range(4):
        again = forward(d)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


LENGTHS = [0, 1, 63, 64, 65, 130, 7, 200, 0]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_packed_prefill(dtype):
    """Lengths around a chunk, empty ones, rows behind the last sequence left as they were."""
    total, N = sum(LENGTHS), len(LENGTHS)
    d = inputs((total + 9,), 2, 6, dtype, 80, states=N)
    x = dev(d)
    cu = torch.tensor(np.cumsum([0] + LENGTHS), dtype=torch.int32)
    o = torch.full_like(x["v"], 7.0)
    SF = torch.full((N, 6, 128, 128), float("nan"), device=DEV)
    binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, cu.to(DEV))
    torch.cuda.synchronize()
    assert (o[total:] == 7.0).all()
    for i, n in enumerate(LENGTHS):
        a = int(cu[i])
        part = {k: (v[None, a:a + n] if k in ("q", "k", "v") else v) for k, v in d.items()}
        part["S0"] = d["S0"][i:i + 1]
        if n == 0:
            assert torch.equal(SF[i].cpu(), d["S0"][i])
        else:
            check_forward(part, o[None, a:a + n], SF[i:i + 1], f"sequence {i} of {n}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_packed_prefill_keeps_bad_values_apart(dtype, value):
    """A sequence of NaN or infinities reaches no other sequence, although its rows share tiles."""
    n = [30, 40, 50, 64]
    d = inputs((sum(n),), 1, 3, dtype, 81, states=4)
    clean = {k: v.clone() for k, v in d.items()}
    for name in ("q", "k", "v"):
        d[name][30:70] = value
    x = dev(d)
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device=DEV)
    o, SF = torch.empty_like(x["v"]), torch.empty((4, 3, 128, 128), device=DEV)
    binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, cu)
    for i in (0, 2, 3):
        a, e = int(cu[i]), int(cu[i + 1])
        part = {k: (v[None, a:e] if k in ("q", "k", "v") else v) for k, v in clean.items()}
        part["S0"] = clean["S0"][i:i + 1]
        check_forward(part, o[None, a:e], SF[i:i + 1], f"sequence {i}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_packed_prefill_keeps_bad_values_from_long_sequences(dtype, value):
    """As above behind sequences of two to six chunks, whose last chunk is cut by their end."""
    n = [70, 3, 101, 20, 190, 64, 230, 5, 129, 1, 333, 40]
    d = inputs((sum(n),), 2, 4, dtype, 87, states=len(n))
    clean = {k: v.clone() for k, v in d.items()}
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32)
    for i in range(1, len(n), 2):
        for name in ("q", "k", "v"):
            d[name][cu[i]:cu[i + 1]] = value
    x = dev(d)
    o, SF = torch.empty_like(x["v"]), torch.empty((len(n), 4, 128, 128), device=DEV)
    binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, cu.to(DEV))
    for i in range(0, len(n), 2):
        a, e = int(cu[i]), int(cu[i + 1])
        part = {k: (v[None, a:e] if k in ("q", "k", "v") else v) for k, v in clean.items()}
        part["S0"] = clean["S0"][i:i + 1]
        check_forward(part, o[None, a:e], SF[i:i + 1], f"sequence {i}")


def test_packed_prefill_clamps_a_bad_table():
    """Offsets out of range or out of order: some result, every access inside the arrays."""
    d = inputs((100,), 1, 2, torch.bfloat16, 82, states=4)
    x = dev(d)
    for table in ([0, 500, 20, 90, 1 << 30], [-50, 40, 30, -7, 100], [100, 100, 0, 0, 0]):
        o, SF = torch.zeros_like(x["v"]), torch.empty((4, 2, 128, 128), device=DEV)
        binding.gdn_decay_fwd_varlen(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF,
                                     torch.tensor(table, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert torch.isfinite(SF).all() and binding.device_status() == "GDN_OK"


# ------------------------------------------------------------------ gradients

def backward(d, dO, dSF, with_dS0=True, **kw):
    x = dev(d)
    nan = lambda t, dt=None: torch.full(t.shape, float("nan"), dtype=dt or t.dtype, device=DEV)  # noqa: E731
    dq, dk, dv = nan(d["q"]), nan(d["k"]), nan(d["v"])
    B, T, Hv = d["v"].shape[:3]
    dS0 = torch.full((B, Hv, 128, 128), float("nan"), device=DEV) if with_dS0 else None
    binding.gdn_decay_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], dO.to(DEV),
                          None if dSF is None else dSF.to(DEV), dq, dk, dv, dS0, **kw)
    torch.cuda.synchronize()
    return dq, dk, dv, dS0


def check_backward(d, dO, dSF, got, what):
    args = (d["q"], d["k"], d["v"], d["decay"], d["S0"], dO, dSF)
    r, m = ref.decay_backward(*args), ref.decay_backward_majorant(*args)
    bf16, T = d["q"].dtype == torch.bfloat16, d["q"].shape[1]
    for i, name in enumerate(("dq", "dk", "dv")):
        check(got[i], r[i], m[i], *out_bounds(bf16, T), f"{what} {name}")
    if got[3] is not None:
        check(got[3], r[3], m[3], 0.0, state_bounds(bf16, T), f"{what} dS0")


def upstream(d, seed, state=True):
    g = torch.Generator().manual_seed(seed)
    dO = torch.randn(d["v"].shape, generator=g).to(d["v"].dtype)
    B, Hv = d["v"].shape[0], d["v"].shape[2]
    return dO, (torch.randn(B, Hv, 128, 128, generator=g) * 0.2 if state else None)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 128, 200])
def test_gradients(dtype, T):
    """Shared QK heads (summed over three V heads), both states."""
    d = inputs((2, T), 2, 6, dtype, 100 + T)
    dO, dSF = upstream(d, 101 + T)
    check_backward(d, dO, dSF, backward(d, dO, dSF), f"T={T}")
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (2, 2), (1, 4)])
def test_gradients_in_segments(dtype, Hqk, Hv):
    d = inputs((1, 1130), Hqk, Hv, dtype, 140 + Hv)
    dO, dSF = upstream(d, 141)
    check_backward(d, dO, dSF, backward(d, dO, dSF), f"heads {Hqk}/{Hv}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("state", [False, True])
def test_gradients_in_segments_behind_a_head(dtype, state):
    d = inputs((1, 1800), 6, 12, dtype, 146, s0=state)
    dO, dSF = upstream(d, 147, state=state)
    check_backward(d, dO, dSF, backward(d, dO, dSF), "head")
    assert binding.device_status() == "GDN_OK"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("state", [False, True])
def test_gradients_without_states(dtype, state):
    d = inputs((2, 100), 2, 2, dtype, 150, s0=state)
    dO, dSF = upstream(d, 151, state=not state)
    check_backward(d, dO, dSF, backward(d, dO, dSF), "one state")
    got = backward(d, dO, dSF, with_dS0=False)
    check_backward(d, dO, dSF, got, "no dS0")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gradients_at_the_ends_of_the_decay(dtype):
    d = inputs((1, 150), 1, 6, dtype, 160)
    d["decay"] = torch.tensor([1e-30, 0.02, 0.25, 0.34, 0.99999, 1.0])
    dO, dSF = upstream(d, 161)
    check_backward(d, dO, dSF, backward(d, dO, dSF), "decay ends")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gradients_of_nothing(dtype):
    d = inputs((2, 0), 1, 2, dtype, 170)
    dO, dSF = upstream(d, 171)
    assert torch.equal(backward(d, dO, dSF)[3].cpu(), dSF)
    assert torch.count_nonzero(backward(d, dO, None)[3]).item() == 0


def test_gradients_match_differences():
    """fp32, through the library's own forward."""
    d = inputs((1, 70), 1, 2, torch.float32, 180)
    dO, dSF = upstream(d, 181)
    grads = backward(d, dO, dSF)

    def loss(x):
        o, S = forward(x)
        return float((o.double().cpu() * dO.double()).sum() + (S.double().cpu() * dSF.double()).sum())

    g = torch.Generator().manual_seed(182)
    for name, grad in zip(("q", "k", "v", "S0"), grads):
        way = torch.randn(d[name].shape, generator=g)
        h = 2.0 ** -7
        up, down = (loss({**d, name: d[name] + s * h * way}) for s in (1, -1))
        got = float((grad.double().cpu() * way.double()).sum())
        # the loss is linear in q, v and S0 and in k: only roundings of a sum of about 2e4 terms
        assert abs((up - down) / (2 * h) - got) <= 2e-3 * max(1.0, abs(got)), name


def test_gradients_repeat_bit_for_bit():
    d = inputs((1, 500), 2, 6, torch.bfloat16, 190)
    dO, dSF = upstream(d, 191)
    first = backward(d, dO, dSF)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, backward(d, dO, dSF)))


# ------------------------------------------------------------------ streams, graphs, workspaces

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_captured_and_on_another_stream(dtype):
    """Forward and gradients captured into one graph on a side stream and replayed on new inputs,
    while the same calls run eagerly on the default stream with their own workspaces."""
    d, e = inputs((1, 700), 1, 3, dtype, 200), inputs((1, 700), 1, 3, dtype, 201)
    dO, dSF = upstream(d, 202)
    want, want_b = forward(e), backward(e, dO, dSF)
    x = dev(d)
    s = torch.cuda.Stream()
    dOd, dSd = dO.to(DEV), dSF.to(DEV)
    out = [torch.empty_like(x["v"]), torch.empty_like(x["S0"])]
    grads = [torch.empty_like(x["q"]), torch.empty_like(x["k"]), torch.empty_like(x["v"]), torch.empty_like(x["S0"])]
    wf = torch.empty(max(1, binding.decay_fwd_workspace_bytes(1, 700, 3, dtype)), dtype=torch.uint8, device=DEV)
    wb = torch.empty(max(1, binding.decay_bwd_workspace_bytes(1, 700, 1, 3, dtype)), dtype=torch.uint8, device=DEV)

    def run():
        binding.gdn_decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], *out, workspace=wf)
        binding.gdn_decay_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], dOd, dSd, *grads, workspace=wb)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        run()
    for name in ("q", "k", "v", "S0"):
        x[name].copy_(e[name])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph.replay()
    eager = forward(e)                                   # at the same time, workspaces of its own
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(eager, want))
    assert all(torch.equal(a, b) for a, b in zip(grads, want_b))


def test_allocated_workspace_outlives_the_call_on_a_side_stream():
    """Without a workspace the binding allocates one; work that reuses its memory comes after."""
    d = inputs((1, 1130), 1, 2, torch.bfloat16, 210)
    want = forward(d)
    x = dev(d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, SF = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    for _ in range(5):
        binding.gdn_decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, stream=s)
        torch.full((binding.decay_fwd_workspace_bytes(1, 1130, 2, torch.bfloat16),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(SF, want[1])


def test_allocated_workspace_is_not_memory_of_another_streams_work():
    """Fills of a freed block still run on the default stream while the call runs on another."""
    d = inputs((1, 1130), 1, 2, torch.bfloat16, 211)
    want = forward(d)
    x = dev(d)
    s = torch.cuda.Stream()
    size = binding.decay_fwd_workspace_bytes(1, 1130, 2, torch.bfloat16)
    o, SF = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    torch.cuda.synchronize()
    for _ in range(10):
        block = torch.empty(size, dtype=torch.uint8, device=DEV)
        torch.cuda._sleep(3_500_000)                     # so that the fills are queued up
        for _ in range(800):
            block.fill_(255)
        del block
        binding.gdn_decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, SF, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(SF, want[1])


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_decode_step(dtype):
    d = inputs((5,), 2, 6, dtype, 300)
    x = dev(d)
    S_new, o = torch.empty_like(x["S0"]), torch.empty_like(x["v"])
    binding.gdn_decay_decode_step(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, S_new)
    args = tuple(d[n][:, None] for n in ("q", "k", "v")) + (d["decay"], d["S0"])
    (ro, rS), (mo, mS) = ref.decay_forward(*args), ref.decay_forward_majorant(*args)
    check(S_new, rS, mS, 0.0, 2 * F32, "S_new")
    check(o, ro[:, 0], mo[:, 0], BF16 if dtype == torch.bfloat16 else 0.0, 140 * F32, "o")
    binding.gdn_decay_decode_step(x["q"], x["k"], x["v"], x["decay"], x["S0"], o, x["S0"])
    assert torch.equal(x["S0"], S_new)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_decode_from_a_pool(dtype):
    """Slots in any order; out of range ones are padding: o row and every state left as they were."""
    d = inputs((6,), 1, 3, dtype, 310, states=9)
    x = dev(d)
    slots = torch.tensor([4, -1, 8, 9, 0, -(1 << 31)], dtype=torch.int32)
    pool, o = x["S0"].clone(), torch.full_like(x["v"], 3.0)
    binding.gdn_decay_decode_step_slots(x["q"], x["k"], x["v"], x["decay"], pool, slots.to(DEV), o)
    use = [0, 2, 4]
    S, o1 = x["S0"][slots[use].long()].clone(), torch.empty_like(x["v"][use])
    binding.gdn_decay_decode_step(*(x[n][use].contiguous() for n in ("q", "k", "v")), x["decay"], S, o1, S)
    assert torch.equal(o[use], o1) and (o[[1, 3, 5]] == 3.0).all()
    assert torch.equal(pool[slots[use].long()], S)
    rest = [i for i in range(9) if i not in slots[use].tolist()]
    assert torch.equal(pool[rest], x["S0"][rest])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_decode_continues_a_prefill(dtype):
    d = inputs((2, 75), 1, 3, dtype, 320)
    whole = forward(d)
    head = {k: (v[:, :70].contiguous() if k in ("q", "k", "v") else v) for k, v in d.items()}
    x = dev(d)
    _, S = forward(head)
    outs = []
    for t in range(70, 75):
        o = torch.empty_like(x["v"][:, t])
        binding.gdn_decay_decode_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v")), x["decay"], S, o, S)
        outs.append(o)
    args = (d["q"], d["k"], d["v"], d["decay"], d["S0"])
    (ro, rS), (mo, mS) = ref.decay_forward(*args), ref.decay_forward_majorant(*args)
    bf16 = dtype == torch.bfloat16
    check(S, rS, mS, 0.0, state_bounds(bf16, 75), "S")
    check(torch.stack(outs, 1), ro[:, 70:], mo[:, 70:], *out_bounds(bf16, 75), "o")
    check(whole[1], rS, mS, 0.0, state_bounds(bf16, 75), "prefill S")


def test_decode_past_32_bit_offsets():
    """A pool of more than 2^31 values: the last slot's states."""
    n = (1 << 31) // (48 * 128 * 128) + 40
    d = inputs((1,), 16, 48, torch.bfloat16, 330)
    x = dev(d)
    pool = torch.empty((n, 48, 128, 128), device=DEV)
    pool[n - 1], pool[n - 2] = x["S0"][0], 5.0
    o, S, o1 = torch.empty_like(x["v"]), x["S0"].clone(), torch.empty_like(x["v"])
    binding.gdn_decay_decode_step_slots(x["q"], x["k"], x["v"], x["decay"], pool, torch.tensor([n - 1], dtype=torch.int32, device=DEV), o)
    binding.gdn_decay_decode_step(x["q"], x["k"], x["v"], x["decay"], S, o1, S)
    assert torch.equal(pool[n - 1], S[0]) and torch.equal(o, o1) and (pool[n - 2] == 5.0).all()
