"""GPU parity of draft trees over a state pool (verification and commit), of the 8-bit state
cache, and a run of all of them as a server would make it."""
import numpy as np
import pytest
import torch

from linear_attention_recurrence_07_b200 import binding
from oracle import decay as ref
from decay_bounds import F32, check, commit_bound, out_bounds, state_bounds, tree_bounds

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "fp32"]
RULES = ["delta", "decay"]


def problem(B, n, Hqk, Hv, dtype, seed, n_slots=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    n_slots = B + 3 if n_slots is None else n_slots
    return {"q": unit(r(B, n, Hqk, 128)).to(dtype), "k": unit(r(B, n, Hqk, 128)).to(dtype), "v": r(B, n, Hv, 128).to(dtype),
            "alpha": torch.exp(-torch.rand(B, n, Hv, generator=g) * 0.3), "beta": torch.sigmoid(r(B, n, Hv)),
            "decay": torch.tensor([0.5, 0.99, 0.9, 1.0, 0.7, 0.97])[:Hv].contiguous(),
            "pool": r(n_slots, Hv, 128, 128) * 0.3,
            "slots": torch.randperm(n_slots, generator=g)[:B].int()}


def chain(B, n):
    return torch.arange(-1, n - 1, dtype=torch.int32).repeat(B, 1)


def star(B, n):
    return torch.full((B, n), -1, dtype=torch.int32)


def bushy(B, n, seed=0):
    """Random earlier parents, several roots, a padded end in every second tree."""
    rng = np.random.default_rng(seed)
    p = np.array([[-1 if i == 0 or rng.random() < 0.1 else rng.integers(max(0, i - 6), i) for i in range(n)] for _ in range(B)])
    p[1::2, n - n // 4:] = -2
    return torch.tensor(p, dtype=torch.int32)


SHAPES = {"chain": chain, "star": star, "bushy": bushy}


def verify(d, parents, rule, fill=9.0, slots=True):
    x = {k: v.to(DEV) for k, v in d.items()}
    o = torch.full_like(x["v"], fill)
    s = x["slots"] if slots else None
    if rule == "delta":
        binding.gdn_decode_tree(x["q"], x["k"], x["v"], x["alpha"], x["beta"], parents.to(DEV), x["pool"], s, o)
    else:
        binding.gdn_decay_decode_tree(x["q"], x["k"], x["v"], x["decay"], parents.to(DEV), x["pool"], s, o)
    torch.cuda.synchronize()
    assert torch.equal(x["pool"].cpu(), d["pool"])
    return o


def commit(d, parents, accepted, rule, slots=True):
    x = {k: v.to(DEV) for k, v in d.items()}
    s = x["slots"] if slots else None
    if rule == "delta":
        binding.gdn_tree_commit(x["k"], x["v"], x["alpha"], x["beta"], parents.to(DEV), accepted.to(DEV), x["pool"], s)
    else:
        binding.gdn_decay_tree_commit(x["k"], x["v"], x["decay"], parents.to(DEV), accepted.to(DEV), x["pool"], s)
    torch.cuda.synchronize()
    return x["pool"]


def reference(d, parents, rule, slots=None):
    slots = d["slots"].long() if slots is None else slots
    gates = {"alpha": d["alpha"], "beta": d["beta"]} if rule == "delta" else {"decay": d["decay"]}
    args = (d["q"], d["k"], d["v"], parents.numpy(), d["pool"][slots])
    return ref.tree(*args, **gates), ref.tree(*args, **gates, majorant=True)


def check_outputs(o, d, parents, rule, fill=9.0):
    (ro, _, alive), (mo, _, _) = reference(d, parents, rule)
    n = parents.shape[1]
    check(o[torch.from_numpy(alive)], ro[alive], mo[alive], *tree_bounds(d["q"].dtype == torch.bfloat16, n), rule)
    assert (o[torch.from_numpy(~alive)] == fill).all(), "padding rows were written"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 64])
def test_verification(dtype, rule, shape, n):
    d = problem(3, n, 2, 6, dtype, 500 + n)
    parents = SHAPES[shape](3, n)
    check_outputs(verify(d, parents, rule), d, parents, rule)


@pytest.mark.parametrize("rule", RULES)
def test_padding_and_skipped_sequences(rule):
    """Bad parents pad their subtree, bad slots their sequence; a tree of padding alone."""
    d = problem(4, 6, 1, 3, torch.bfloat16, 520)
    parents = torch.tensor([[-1, 0, 5, 2, 0, 4], [-2, 0, 1, -7, 3, -1], [-3] * 6, [-1, 0, 1, 2, 3, 4]], dtype=torch.int32)
    d["slots"][3] = 99
    o = verify(d, parents, rule)
    assert (o[2:] == 9.0).all()
    part = {k: (v if k in ("pool", "decay") else v[:2]) for k, v in d.items()}
    check_outputs(o[:2], part, parents[:2], rule)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_below_their_node(dtype, rule, value):
    d = problem(1, 20, 1, 2, dtype, 530)
    parents = bushy(1, 20, seed=3)
    parents[0, [9, 12, 17]] = torch.tensor([7, 9, 12], dtype=torch.int32)    # some nodes are below it, most are not
    clean = verify(d, parents, rule)
    for name in ("q", "k", "v", "alpha", "beta"):
        d[name][:, 7] = value
    got = verify(d, parents, rule)
    below = {7}
    for i in range(8, 20):
        if int(parents[0, i]) in below:
            below.add(i)
    assert 1 < len(below) < 13
    rest = [i for i in range(20) if i not in below]
    assert torch.equal(got[:, rest], clean[:, rest])


@pytest.mark.parametrize("rule", RULES)
def test_gates_at_their_ends(rule):
    d = problem(2, 24, 1, 6, torch.float32, 540)
    d["alpha"][:, ::3], d["alpha"][:, 1::3], d["beta"][:, ::2] = 1.0, 1e-30, 0.0
    d["beta"][:, 1::2] = 1.5
    d["decay"] = torch.tensor([1e-30, 0.02, 1.0, 0.5, 0.25, 0.999])
    for parents in (chain(2, 24), bushy(2, 24)):
        check_outputs(verify(d, parents, rule), d, parents, rule)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_a_chain_is_decode_tokens(dtype):
    d = problem(2, 9, 2, 6, dtype, 550)
    x = {k: v.to(DEV) for k, v in d.items()}
    S = x["pool"][x["slots"].long()].clone()
    o, S_new = torch.empty_like(x["v"]), torch.empty_like(S)
    binding.gdn_decode_tokens(x["q"], x["k"], x["v"], x["alpha"], x["beta"], S, o, S_new)
    parents = chain(2, 9)
    (ro, rS, _), (mo, mS, _) = reference(d, parents, "delta")
    check(o, ro, mo, *tree_bounds(dtype == torch.bfloat16, 9), "gdn_decode_tokens")
    check_outputs(verify(d, parents, "delta"), d, parents, "delta")
    pool = commit(d, parents, torch.tensor([8, 8], dtype=torch.int32), "delta")
    check(pool[d["slots"].long().to(DEV)], rS[:, 8], mS[:, 8], 0.0, commit_bound(9), "commit")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("n", [1, 4, 5, 23, 64])
def test_commit(dtype, rule, n):
    """Paths of every length modulo the groups of four; nothing accepted; padding nodes."""
    B = 6
    d = problem(B, n, 1, 3, dtype, 560 + n)
    parents = torch.cat([chain(3, n), bushy(3, n, seed=n)])
    accepted = torch.tensor([n - 1, n // 2, 0, n - 1, -1, n], dtype=torch.int32)
    pool = commit(d, parents, accepted, rule).cpu()
    (_, rS, alive), (_, mS, _) = reference(d, parents, rule)
    for b in range(B):
        slot, leaf = int(d["slots"][b]), int(accepted[b])
        if 0 <= leaf < n and alive[b, leaf]:
            check(pool[slot], rS[b, leaf], mS[b, leaf], 0.0, commit_bound(n), f"sequence {b}")
        else:
            assert torch.equal(pool[slot], d["pool"][slot]), b
    rest = [s for s in range(d["pool"].shape[0]) if s not in d["slots"].tolist()]
    assert torch.equal(pool[rest], d["pool"][rest])


@pytest.mark.parametrize("rule", RULES)
def test_without_slots(rule):
    d = problem(3, 10, 1, 3, torch.bfloat16, 580)
    e = {**d, "slots": torch.arange(3, dtype=torch.int32)}
    parents, accepted = bushy(3, 10), torch.tensor([4, 6, 9], dtype=torch.int32)
    assert torch.equal(verify(d, parents, rule, slots=False), verify(e, parents, rule))
    assert torch.equal(commit(d, parents, accepted, rule, slots=False), commit(e, parents, accepted, rule))


def test_trees_repeat_bit_for_bit_and_in_a_graph():
    d = problem(4, 40, 2, 6, torch.bfloat16, 590)
    parents = bushy(4, 40)
    want = verify(d, parents, "delta")
    x = {k: v.to(DEV) for k, v in d.items()}
    p, o = parents.to(DEV), torch.full_like(x["v"], 9.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.gdn_decode_tree(x["q"], x["k"], x["v"], x["alpha"], x["beta"], p, x["pool"], x["slots"], o)
    for _ in range(3):
        o.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


# ------------------------------------------------------------------ 8-bit state cache

FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def rows(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, 128, 128, generator=g) * torch.exp(3 * torch.randn(*shape, 128, 1, generator=g))
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 1e-33
    x[0, 0, 2, 5] = float("nan")
    x[0, 0, 3, 127] = -float("inf")
    x[0, 0, 4] = 1e-30
    x[0, 0, 5] = 3e38
    x[0, 0, 6, :] = 0
    x[0, 0, 6, 77] = -2.5
    return x


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("Hv", [1, 3])
def test_cache_round_trip(fmt, Hv):
    """Codes and scales exactly as defined; reading gives code * scale; skipped entries untouched."""
    pool = rows(600, 5, Hv)
    p = pool.to(DEV)
    codes = torch.full((7, Hv, 128, 128), 5, dtype=torch.int8, device=DEV).view(FORMATS[fmt])
    scales = torch.full((7, Hv, 128), 2.0, device=DEV)
    slots = torch.tensor([0, 3, -1, 4, 5], dtype=torch.int32, device=DEV)
    cache = torch.tensor([6, 0, 2, 7, 3], dtype=torch.int32, device=DEV)
    binding.gdn_state_store(p, slots, codes, scales, cache)
    c, s = ref.quantise_rows(pool.numpy(), fmt)
    value = codes.float().cpu().numpy()
    for a, b in ((0, 6), (3, 0)):
        assert np.array_equal(value[b], c[a].astype(np.float32))
        assert np.array_equal(scales[b].cpu().numpy(), s[a], equal_nan=True)
    for b in (1, 2, 3, 4, 5):
        assert (codes[b].view(torch.int8) == 5).all() and (scales[b] == 2.0).all()
    out = torch.full_like(p, 8.0)
    binding.gdn_state_load(codes, scales, cache, out, slots)
    for a in (0, 3):
        want = (c[a].astype(np.float32) * s[a][..., None]).astype(np.float32)
        assert np.array_equal(out[a].cpu().numpy(), want, equal_nan=True)
    assert (out[[1, 2, 4]] == 8.0).all()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_cache_ties_and_ends(fmt):
    """Values on the borders between codes, and the largest code."""
    top = 127.0 if fmt == "int8" else 448.0
    x = torch.zeros(1, 1, 128, 128)
    x[..., 0] = top                                          # scale 1
    x[..., 1:] = torch.arange(127) + 0.5 if fmt == "int8" else torch.from_numpy(
        (ref.e4m3_values()[:-1] + ref.e4m3_values()[1:]) / 2).float().repeat(2)[:127]
    x[..., 1:][..., ::2] *= -1
    codes = torch.zeros(1, 1, 128, 128, dtype=torch.int8, device=DEV).view(FORMATS[fmt])
    scales, zero = torch.zeros(1, 1, 128, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.gdn_state_store(x.to(DEV), zero, codes, scales, zero)
    c, _ = ref.quantise_rows(x.numpy(), fmt)
    assert np.array_equal(codes.float().cpu().numpy(), c.astype(np.float32)) and (scales == 1).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rule", RULES)
def test_a_server_run(dtype, rule):
    """Packed prompts -> states into a pool -> a snapshot of one -> a tree of drafts -> its accepted path ->
    one more token -> the snapshot back into another slot, all on one side stream."""
    Hqk, Hv, lengths = 1, 3, [40, 130]
    g = torch.Generator().manual_seed(700)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    T = sum(lengths)
    q, k, v = unit(r(T, Hqk, 128)).to(dtype), unit(r(T, Hqk, 128)).to(dtype), r(T, Hv, 128).to(dtype)
    lam = torch.tensor([0.6, 0.95, 0.999])
    alpha, beta = torch.exp(-torch.rand(T, Hv, generator=g) * 0.1), torch.sigmoid(r(T, Hv))
    cu = torch.tensor([0, 40, 170], dtype=torch.int32)
    d = problem(2, 7, Hqk, Hv, dtype, 701, n_slots=4)
    d["decay"] = lam
    d["slots"] = torch.tensor([2, 0], dtype=torch.int32)
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1, 1, 3, -2, 5]], dtype=torch.int32)
    accepted = torch.tensor([6, 4], dtype=torch.int32)
    x = {n: t.to(DEV) for n, t in d.items()}
    dv = {n: t.to(DEV) for n, t in dict(q=q, k=k, v=v, lam=lam, alpha=alpha, beta=beta, cu=cu).items()}
    pd, ad = parents.to(DEV), accepted.to(DEV)
    last = {n: t.to(DEV) for n, t in problem(2, 1, Hqk, Hv, dtype, 702).items()}
    codes, scales = torch.zeros(2, Hv, 128, 128, dtype=torch.int8, device=DEV), torch.zeros(2, Hv, 128, device=DEV)
    one, three = torch.tensor([1], dtype=torch.int32, device=DEV), torch.tensor([3], dtype=torch.int32, device=DEV)
    o, states = torch.empty_like(dv["v"]), torch.empty(2, Hv, 128, 128, device=DEV)
    pool, o_tree, o_last = torch.zeros(4, Hv, 128, 128, device=DEV), torch.zeros_like(x["v"]), torch.empty_like(last["v"][:, 0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        if rule == "delta":
            binding.gdn_chunk_fwd_varlen(dv["q"], dv["k"], dv["v"], dv["alpha"], dv["beta"], None, o, states, dv["cu"])
        else:
            binding.gdn_decay_fwd_varlen(dv["q"], dv["k"], dv["v"], dv["lam"], None, o, states, dv["cu"])
        pool[x["slots"].long()] = states
        binding.gdn_state_store(pool, x["slots"][:1], codes, scales, one)
        if rule == "delta":
            gates = (x["alpha"], x["beta"])
            binding.gdn_decode_tree(x["q"], x["k"], x["v"], *gates, pd, pool, x["slots"], o_tree)
            binding.gdn_tree_commit(x["k"], x["v"], *gates, pd, ad, pool, x["slots"])
            binding.gdn_decode_step_slots(*(last[n][:, 0].contiguous() for n in ("q", "k", "v", "alpha", "beta")), pool,
                                          x["slots"], o_last)
        else:
            binding.gdn_decay_decode_tree(x["q"], x["k"], x["v"], x["decay"], pd, pool, x["slots"], o_tree)
            binding.gdn_decay_tree_commit(x["k"], x["v"], x["decay"], pd, ad, pool, x["slots"])
            binding.gdn_decay_decode_step_slots(*(last[n][:, 0].contiguous() for n in ("q", "k", "v")), x["decay"], pool,
                                                x["slots"], o_last)
        binding.gdn_state_load(codes, scales, one, pool, three)
    s.synchronize()
    # from the prefill's states on, each step against the reference
    S = states.cpu()
    d["pool"] = torch.zeros(4, Hv, 128, 128)
    d["pool"][d["slots"].long()] = S
    check_outputs(o_tree, d, parents, rule, fill=0.0)
    (_, rS, _), (_, mS, _) = reference(d, parents, rule)
    gates = {"decay": lam} if rule == "decay" else {"alpha": last["alpha"].cpu(), "beta": last["beta"].cpu()}
    after = np.stack([rS[0, 6], rS[1, 4]])
    majs = np.stack([mS[0, 6], mS[1, 4]])
    args = (last["q"].cpu(), last["k"].cpu(), last["v"].cpu(), np.full((2, 1), -1))
    ro, r1, _ = ref.tree(*args, torch.from_numpy(after), **gates)
    mo, m1, _ = ref.tree(*args, torch.from_numpy(majs), **gates, majorant=True)
    bf16 = dtype == torch.bfloat16
    check(pool[x["slots"].long()], r1[:, 0], m1[:, 0], 0.0, commit_bound(5), "states")
    check(o_last, ro[:, 0], mo[:, 0], tree_bounds(bf16, 1)[0], commit_bound(6), "last token")
    c, sc = ref.quantise_rows(S[0].numpy(), "int8")
    assert np.array_equal(pool[3].cpu().numpy(), (c.astype(np.float32) * sc[..., None]).astype(np.float32))
    if rule == "decay":
        args = (q[None, 40:], k[None, 40:], v[None, 40:], lam, None)
        (ro, rS), (mo, mS) = ref.decay_forward(*args), ref.decay_forward_majorant(*args)
        check(o[None, 40:], ro, mo, *out_bounds(bf16, 130), "prompt")
        check(states[1:], rS, mS, 0.0, state_bounds(bf16, 130), "prompt state")
