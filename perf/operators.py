"""Measured cases of the per-head-decay linear attention, the verification of draft trees over a
state pool, and the 8-bit state cache: inputs, plain forms, 64-bit results and the work of a pass.

Operators (per sequence and V head the state S is dk x dv = 128 x 128, fp32; V head h reads q and k
of QK head h / (Hv / Hqk)):

  decay_fwd      S_t = lam_h S_{t-1} + k_t v_t^T, o_t = S_t^T q_t for whole prompts
  decay_varlen   the same for prompts of different lengths packed back to back
  decay_bwd      gradients of <dO, o> + <dS_final, S_final> with respect to q, k, v, S0
  decay_decode   one token for each sequence, states in place (slots: states picked from a pool)
  tree           outputs of a tree of drafted tokens from a pool state, gated delta rule
                 (S = alpha (I - beta k k^T) S_parent + beta k v^T) or decay rule
  tree_commit    the states after the accepted path of each tree, in place
  state_store    pool states to 8-bit codes with one scale per key row
  state_load     codes and scales back to pool states
"""
import math

import torch

own = False

D = 128                     # head dimension of keys and values
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_QMAX = {"int8": 127.0, "e4m3": 448.0}
_TINY = 1e-30               # a row whose largest magnitude is below this is stored as zeros


def listed():
    return [
        # one long prompt, 16 QK heads under 48 V heads, no earlier state: the prefill headline's shape
        {"name": "fwd_B1_T4096", "op": "decay_fwd", "B": 1, "T": 4096, "Hqk": 16, "Hv": 48, "dtype": "bf16", "s0": False},
        # a batch of long prompts that continue from cached states: the largest prefill
        {"name": "fwd_B8_T8192", "op": "decay_fwd", "B": 8, "T": 8192, "Hqk": 16, "Hv": 48, "dtype": "bf16", "s0": True},
        # a short fp32 prompt (reference precision, debugging, small models), odd length
        {"name": "fwd_fp32_T257", "op": "decay_fwd", "B": 1, "T": 257, "Hqk": 2, "Hv": 6, "dtype": "fp32", "s0": True},
        # continuous batching: 16 prompts of 1 .. 2048 tokens in one packed call
        {"name": "varlen_N16", "op": "decay_varlen", "N": 16, "longest": 2048, "mix": 5, "Hqk": 48, "Hv": 48, "dtype": "bf16", "s0": True},
        # a training step's gradients at the headline's length, heads not shared
        {"name": "bwd_B1_T4096", "op": "decay_bwd", "B": 1, "T": 4096, "Hqk": 48, "Hv": 48, "dtype": "bf16", "s0": False},
        # gradients with shared QK heads, a ragged length and gradients through both states
        {"name": "bwd_B2_T1000", "op": "decay_bwd", "B": 2, "T": 1000, "Hqk": 16, "Hv": 48, "dtype": "bf16", "s0": True},
        # one decode step of a large batch, states in place
        {"name": "decode_B256", "op": "decay_decode", "B": 256, "Hqk": 16, "Hv": 48, "dtype": "bf16", "slots": False},
        # one decode step of three sequences out of a pool: the latency of a nearly idle server
        {"name": "decode_slots_B3", "op": "decay_decode", "B": 3, "Hqk": 16, "Hv": 48, "dtype": "bf16", "slots": True},
        # a wide tree of drafts for a small batch, gated delta rule
        {"name": "tree_B16_n48", "op": "tree", "rule": "delta", "B": 16, "n": 48, "Hqk": 16, "Hv": 48, "dtype": "bf16"},
        # the accepted paths of 7-node trees for a decode batch, gated delta rule
        {"name": "commit_B128_n7", "op": "tree_commit", "rule": "delta", "B": 128, "n": 7, "Hqk": 16, "Hv": 48, "dtype": "bf16"},
        # snapshots of 64 sequences' states into the 8-bit cache
        {"name": "store_int8_N64", "op": "state_store", "N": 64, "Hv": 48, "format": "int8"},
        # 24 snapshots brought back for prompts that share a prefix
        {"name": "load_e4m3_N24", "op": "state_load", "N": 24, "Hv": 48, "format": "e4m3"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [(16, 48), (48, 48), (2, 6), (8, 8), (5, 15), (1, 4), (24, 48)]


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_fwd", "decay_varlen", "decay_bwd", "decay_bwd", "decay_decode",
                     "tree", "tree", "tree_commit", "state_store", "state_load"])
    Hqk, Hv = rng.choice(_HEADS)
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    if op == "decay_fwd":
        tokens = 8 * 8192 * 48 // Hv if dtype == "bf16" else 24576 // Hv
        T = _log(rng, 1, min(tokens, 16384))
        B = _log(rng, 1, max(1, min(64, tokens // T)))
        return {"op": op, "B": B, "T": T, "Hqk": Hqk, "Hv": Hv, "dtype": dtype, "s0": rng.random() < 0.5}
    if op == "decay_varlen":
        longest = _log(rng, 1, 4096 if dtype == "bf16" else 300)
        N = _log(rng, 1, max(1, min(32, 65536 * 8 // (longest * Hv))))
        return {"op": op, "N": N, "longest": longest, "mix": rng.randrange(1 << 20), "Hqk": Hqk, "Hv": Hv, "dtype": dtype, "s0": rng.random() < 0.5}
    if op == "decay_bwd":
        tokens = 2 * 4096 * 48 // Hv if dtype == "bf16" else 24576 // Hv
        T = _log(rng, 1, min(tokens, 8192))
        B = _log(rng, 1, max(1, min(16, tokens // T)))
        return {"op": op, "B": B, "T": T, "Hqk": Hqk, "Hv": Hv, "dtype": dtype, "s0": rng.random() < 0.5}
    if op == "decay_decode":
        return {"op": op, "B": _log(rng, 1, 256), "Hqk": Hqk, "Hv": Hv, "dtype": dtype, "slots": rng.random() < 0.5}
    if op in ("tree", "tree_commit"):
        n = _log(rng, 1, 64)
        B = _log(rng, 1, max(1, min(128, 1024 // n)))
        return {"op": op, "rule": rng.choice(["delta", "decay"]), "B": B, "n": n, "Hqk": Hqk, "Hv": Hv, "dtype": dtype}
    return {"op": op, "N": _log(rng, 1, 128), "Hv": Hv, "format": rng.choice(["int8", "e4m3"])}


# ------------------------------------------------------------------ inputs

def _decay(Hv, dev):
    """One constant per head, geometrically spaced: from about 0.4 (short memory) to 0.996."""
    h = torch.arange(1, Hv + 1, dtype=torch.float64, device=dev)
    return torch.exp(-torch.exp2(-8.0 * h / Hv)).float()


def _unit(gen, *shape):
    x = torch.randn(*shape, generator=gen, device="cuda")
    return x / x.norm(dim=-1, keepdim=True)


def _lengths(case):
    """N lengths in 1 .. longest, one of them the longest, spread over their logarithm."""
    g = torch.Generator().manual_seed(case["mix"])
    x = torch.exp(torch.rand(case["N"], generator=g, dtype=torch.float64) * math.log(case["longest"]))
    n = x.round().clamp(1, case["longest"]).long()
    n[case["mix"] % case["N"]] = case["longest"]
    return n


def _parents(case, seed):
    """Trees in node order: a root at most nodes' start, each later node under a random earlier one;
    every other tree is padded at its end (parent -2)."""
    g = torch.Generator().manual_seed(seed)
    B, n = case["B"], case["n"]
    i = torch.arange(n)
    up = torch.floor(torch.rand(B, n, generator=g) * i).long()                 # any earlier node
    near = (i - 1 - torch.floor(torch.rand(B, n, generator=g) * 3).long())     # one of the last three
    p = torch.where(torch.rand(B, n, generator=g) < 0.5, up, near).clamp(min=0)
    p = torch.where((i == 0) | (torch.rand(B, n, generator=g) < 0.05), torch.full_like(p, -1), p)
    size = torch.randint(1, n + 1, (B,), generator=g)
    size[::2] = n
    p = torch.where(i < size[:, None], p, torch.full_like(p, -2))
    acc = torch.floor(torch.rand(B, generator=g) * size).long()                # a node of each tree
    return p.int().cuda(), acc.int().cuda()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, Hv = case["op"], case["Hv"]
    s = {"case": case}
    f32 = dict(dtype=torch.float32, device=dev)
    if op in ("state_store", "state_load"):
        N = case["N"]
        slots = N + 5                                   # a pool and a cache somewhat larger than the batch
        s["slots"] = torch.randperm(slots, generator=gen, device=dev)[:N].int()
        s["cache_slots"] = torch.randperm(slots, generator=gen, device=dev)[:N].int()
        s["scales"] = torch.zeros(slots, Hv, D, **f32)
        if op == "state_store":
            s["pool"] = torch.randn(slots, Hv, D, D, generator=gen, device=dev) * torch.exp(
                torch.randn(slots, Hv, D, 1, generator=gen, device=dev))
            s["codes"] = torch.zeros(slots, Hv, D, D, device=dev, dtype=torch.int8).view(_CODES[case["format"]])
        else:
            s["scales"].copy_(torch.rand(slots, Hv, D, generator=gen, device=dev) * 0.02)
            if case["format"] == "int8":
                s["codes"] = torch.randint(-127, 128, (slots, Hv, D, D), generator=gen, device=dev, dtype=torch.int8)
            else:
                s["codes"] = (torch.randn(slots, Hv, D, D, generator=gen, device=dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["pool"] = torch.zeros(slots, Hv, D, D, **f32)
        return s
    Hqk, dt = case["Hqk"], _DT[case["dtype"]]
    s["decay"] = _decay(Hv, dev)
    if op == "decay_varlen":
        n = _lengths(case)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).int().to(dev)
        lead, states = (int(n.sum()),), case["N"]
    elif op == "decay_decode":
        lead, states = (case["B"],), case["B"]
    elif op in ("tree", "tree_commit"):
        lead, states = (case["B"], case["n"]), case["B"]
    else:
        lead, states = (case["B"], case["T"]), case["B"]
    s["q"] = _unit(gen, *lead, Hqk, D).to(dt)
    s["k"] = _unit(gen, *lead, Hqk, D).to(dt)
    s["v"] = torch.randn(*lead, Hv, D, generator=gen, device=dev).to(dt)
    s["o"] = torch.zeros(*lead, Hv, D, device=dev, dtype=dt)

    def state(scale, rows):
        return torch.randn(rows, Hv, D, D, generator=gen, device=dev) * scale

    if op in ("decay_fwd", "decay_varlen", "decay_bwd"):
        s["S0"] = state(0.1, states) if case["s0"] else None
        s["S_final"] = torch.empty(states, Hv, D, D, **f32)
    if op == "decay_bwd":
        s["dO"] = torch.randn(*lead, Hv, D, generator=gen, device=dev).to(dt)
        s["dS_final"] = state(0.1, states) if case["s0"] else None
        for name in ("q", "k", "v"):
            s["d" + name] = torch.empty_like(s[name])
        s["dS0"] = torch.empty(states, Hv, D, D, **f32)
    elif op == "decay_decode":
        rows = states + 7 if case["slots"] else states
        s["pool"] = state(0.1, rows)
        s["slots"] = torch.randperm(rows, generator=gen, device=dev)[:states].int() if case["slots"] else None
    elif op in ("tree", "tree_commit"):
        s["parents"], s["accepted"] = _parents(case, seed)
        s["pool"] = state(0.1, states + 3)
        s["slots"] = torch.randperm(states + 3, generator=gen, device=dev)[:states].int()
        if case["rule"] == "delta":
            s["alpha"] = torch.exp(-torch.rand(*lead, Hv, generator=gen, device=dev) * 0.1 - 0.001)
            s["beta"] = torch.sigmoid(torch.randn(*lead, Hv, generator=gen, device=dev))
    return s


# ------------------------------------------------------------------ plain forms (32 bits)

def _powers(decay, e):
    """decay[h] ** e for an integer tensor e: [*e.shape, Hv]."""
    return torch.exp(e.double()[..., None] * torch.log(decay.double())).float()


def _rows(x, Hv):
    """[B, T, H, D] in any type to fp32 [B, Hv, T, D], shared heads repeated."""
    return x.float().repeat_interleave(Hv // x.shape[2], dim=2).transpose(1, 2)


def _walk(x, y, z, decay, H0, C=128):
    """o_t = sum_{s <= t} lam^(t-s) (x_t . y_s) z_s + lam^t H0^T x_t for [B, Hv, T, D] operands."""
    B, H, T, _ = x.shape
    n = -(-T // C)
    x, y, z = (torch.nn.functional.pad(t, (0, 0, 0, n * C - T)).reshape(B, H, n, C, D) for t in (x, y, z))
    i = torch.arange(C, device=x.device)
    e = i[:, None] - i[None, :]
    mask = _powers(decay, e.clamp(min=0)).permute(2, 0, 1) * (e >= 0)          # [H, C, C]
    o = ((x @ y.transpose(-1, -2)) * mask[:, None]) @ z
    w = _powers(decay, C - i).t()                                              # state one token after the chunk
    part = (y * w[:, None, :, None]).transpose(-1, -2) @ z                     # [B, H, n, D, D]
    m = torch.arange(n, device=x.device)
    f = m[:, None] - 1 - m[None, :]
    carry = _powers(decay, C * f.clamp(min=0)).permute(2, 0, 1) * (f >= 0)     # [H, n, n]
    start = (carry @ part.reshape(B, H, n, D * D)).reshape(B, H, n, D, D)
    if H0 is not None:
        start = start + _powers(decay, C * m).t()[:, :, None, None] * H0[:, :, None]
    o = o + _powers(decay, i).t()[:, None, :, None] * (x @ start)
    return o.reshape(B, H, n * C, D)[:, :, :T]


def _end(y, z, decay, S0, L, off):
    """lam^(L-1+off) S0 + sum_s lam^(L-1+off-s) y_s z_s^T; L: [B] lengths of zero-padded rows."""
    e = (L[:, None] - 1 + off) - torch.arange(y.shape[2], device=y.device)
    w = _powers(decay, e.clamp(min=0)).permute(0, 2, 1)                        # rows past the end are zero
    S = (y * w[..., None]).transpose(-1, -2) @ z
    if S0 is not None:
        S = S + _powers(decay, L - 1 + off)[..., None, None] * S0
    return S


def _lam(decay, S0):
    return None if S0 is None else decay[:, None, None] * S0


def _plain_fwd(s):
    c = s["case"]
    q, k, v = (_rows(s[n], c["Hv"]) for n in ("q", "k", "v"))
    o = _walk(q, k, v, s["decay"], _lam(s["decay"], s["S0"]))
    L = torch.full((c["B"],), c["T"], device=q.device)
    S = _end(k, v, s["decay"], _lam(s["decay"], s["S0"]), L, 0)
    return o.transpose(1, 2).to(s["o"].dtype), S


def _plain_varlen(s):
    c = s["case"]
    cu = s["cu"].long()
    L = cu[1:] - cu[:-1]
    t = torch.arange(c["longest"], device=cu.device)
    inside = t < L[:, None]
    rows = (cu[:-1, None] + t).clamp(max=s["v"].shape[0] - 1)
    q, k, v = (_rows(s[n][rows] * inside[..., None, None], c["Hv"]) for n in ("q", "k", "v"))
    H0 = _lam(s["decay"], s["S0"])
    o = _walk(q, k, v, s["decay"], H0).transpose(1, 2).to(s["o"].dtype)
    return o[inside], _end(k, v, s["decay"], H0, L, 0)


def _plain_bwd(s):
    c = s["case"]
    Hv, G = c["Hv"], c["Hv"] // c["Hqk"]
    q, k, v, g = (_rows(s[n], Hv) for n in ("q", "k", "v", "dO"))
    lam, S0, dS = s["decay"], s["S0"], s["dS_final"]
    qr, kr, vr, gr = (x.flip(2) for x in (q, k, v, g))
    dq = _walk(g, v, k, lam, None if S0 is None else _lam(lam, S0).transpose(-1, -2))
    dk = _walk(vr, gr, qr, lam, None if dS is None else dS.transpose(-1, -2)).flip(2)
    dv = _walk(kr, qr, gr, lam, dS).flip(2)
    L = torch.full((c["B"],), c["T"], device=q.device)
    dS0 = _end(qr, gr, lam, dS, L, 1)
    fold = lambda x: x.reshape(c["B"], c["Hqk"], G, c["T"], D).sum(2).transpose(1, 2).to(s["q"].dtype)  # noqa: E731
    return fold(dq), fold(dk), dv.transpose(1, 2).to(s["v"].dtype), dS0


def _plain_decode(s):
    c = s["case"]
    G = c["Hv"] // c["Hqk"]
    q, k = (s[n].float().repeat_interleave(G, dim=1) for n in ("q", "k"))
    at = s["slots"].long() if c["slots"] else slice(None)
    S = s["decay"][:, None, None] * s["pool"][at] + k[..., :, None] * s["v"].float()[..., None, :]
    o = (q[..., None, :] @ S)[..., 0, :].to(s["o"].dtype)
    s["pool"][at] = S
    return o, s["pool"]


def _tree_paths(parents):
    """reach[b, i, j]: node j is node i or an ancestor of it; alive[b, i]: i's path has no padding."""
    n = parents.shape[1]
    i = torch.arange(n, device=parents.device)
    p = parents.long()
    ok = (p >= -1) & (p < i)
    step = (p[..., None] == i) & ok[..., None]
    reach = (step | (i[:, None] == i)).float()
    for _ in range(6):                       # paths of up to 2^6 steps
        reach = (reach @ reach > 0).float()
    alive = ~((reach * (~ok)[:, None, :].float()).sum(-1) > 0)
    return reach, alive


def _tree_gates(s):
    """log gates [B, Hv, n] and write strengths [B, Hv, n] or None (decay rule)."""
    c = s["case"]
    if c["rule"] == "delta":
        return torch.log(s["alpha"].double()).transpose(1, 2), s["beta"].transpose(1, 2)
    return torch.log(s["decay"].double())[None, :, None].expand(c["B"], c["Hv"], c["n"]), None


def _tree_updates(s):
    """S, K, reach, alive, path decays and the rows u of the update S + sum k u^T, per V head."""
    c = s["case"]
    S = s["pool"][s["slots"].long()]
    k, v = (_rows(s[n], c["Hv"]) for n in ("k", "v"))
    reach, alive = _tree_paths(s["parents"])
    la, beta = _tree_gates(s)
    b = la @ reach.double().transpose(-1, -2)                                  # log decay of each node's path
    up = reach[:, None]
    gam = (torch.exp((b[..., :, None] - b[..., None, :]) * up) * up).float()   # decay from j's write to i
    root = torch.exp(b).float()[..., None]
    u = v
    if beta is not None:
        strict = gam - torch.eye(c["n"], device=gam.device)
        A = beta[..., None] * strict * (k @ k.transpose(-1, -2))
        u = beta[..., None] * (v - root * (k @ S))
        P = -A
        for _ in range(6):                   # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)..., A^64 = 0
            u = u + P @ u
            P = P @ P
    return S, k, u, reach, alive, gam, root


def _plain_tree(s):
    c = s["case"]
    S, k, u, reach, alive, gam, root = _tree_updates(s)
    q = _rows(s["q"], c["Hv"])
    o = root * (q @ S) + (gam * (q @ k.transpose(-1, -2))) @ u
    return (o.transpose(1, 2) * alive[..., None, None]).to(s["o"].dtype)        # padding rows stay zero


def _plain_commit(s):
    c = s["case"]
    S, k, u, reach, alive, gam, root = _tree_updates(s)
    leaf = s["accepted"].long().clamp(min=0)
    take = lambda x: torch.gather(x, 2, leaf[:, None, None, None].expand(-1, x.shape[1], 1, x.shape[3]))  # noqa: E731
    w = take(gam)[:, :, 0]                                                     # [B, Hv, n] decay from each write
    new = take(root) * S + (k * w[..., None]).transpose(-1, -2) @ u
    keep = (s["accepted"] >= 0) & torch.gather(alive, 1, leaf[:, None])[:, 0]
    s["pool"][s["slots"].long()] = torch.where(keep[:, None, None, None], new, S)
    return s["pool"]


def _plain_store(s):
    c = s["case"]
    qmax = _QMAX[c["format"]]
    x = s["pool"][s["slots"].long()]
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, qmax)        # tensors on both sides: correctly rounded quotients, not products with 1 / x
    zero = amax < _TINY
    y = torch.where(zero, torch.zeros_like(x), x * (top / amax))
    y = torch.round(y).clamp(-qmax, qmax).to(torch.int8) if c["format"] == "int8" else y.to(torch.float8_e4m3fn)
    at = s["cache_slots"].long()
    s["codes"].view(torch.int8)[at] = y.view(torch.int8)
    s["scales"][at] = torch.where(zero, torch.zeros_like(amax), amax / top)[..., 0]
    return s["codes"], s["scales"]


def _plain_load(s):
    at = s["cache_slots"].long()
    s["pool"][s["slots"].long()] = s["codes"].view(torch.int8)[at].view(s["codes"].dtype).float() * s["scales"][at][..., None]
    return s["pool"]


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    from linear_attention_recurrence_07_b200 import binding as g
    c = s["case"]
    op = c["op"]
    if op == "decay_fwd":
        g.gdn_decay_fwd(s["q"], s["k"], s["v"], s["decay"], s["S0"], s["o"], s["S_final"])
        return s["o"], s["S_final"]
    if op == "decay_varlen":
        g.gdn_decay_fwd_varlen(s["q"], s["k"], s["v"], s["decay"], s["S0"], s["o"], s["S_final"], s["cu"])
        return s["o"], s["S_final"]
    if op == "decay_bwd":
        g.gdn_decay_bwd(s["q"], s["k"], s["v"], s["decay"], s["S0"], s["dO"], s["dS_final"],
                        s["dq"], s["dk"], s["dv"], s["dS0"])
        return s["dq"], s["dk"], s["dv"], s["dS0"]
    if op == "decay_decode":
        if c["slots"]:
            g.gdn_decay_decode_step_slots(s["q"], s["k"], s["v"], s["decay"], s["pool"], s["slots"], s["o"])
        else:
            g.gdn_decay_decode_step(s["q"], s["k"], s["v"], s["decay"], s["pool"], s["o"], s["pool"])
        return s["o"], s["pool"]
    if op == "tree":
        if c["rule"] == "delta":
            g.gdn_decode_tree(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["parents"], s["pool"], s["slots"], s["o"])
        else:
            g.gdn_decay_decode_tree(s["q"], s["k"], s["v"], s["decay"], s["parents"], s["pool"], s["slots"], s["o"])
        return s["o"]
    if op == "tree_commit":
        if c["rule"] == "delta":
            g.gdn_tree_commit(s["k"], s["v"], s["alpha"], s["beta"], s["parents"], s["accepted"], s["pool"], s["slots"])
        else:
            g.gdn_decay_tree_commit(s["k"], s["v"], s["decay"], s["parents"], s["accepted"], s["pool"], s["slots"])
        return s["pool"]
    if op == "state_store":
        g.gdn_state_store(s["pool"], s["slots"], s["codes"], s["scales"], s["cache_slots"])
        return s["codes"], s["scales"]
    g.gdn_state_load(s["codes"], s["scales"], s["cache_slots"], s["pool"], s["slots"])
    return s["pool"]


_PLAIN = {"decay_fwd": _plain_fwd, "decay_varlen": _plain_varlen, "decay_bwd": _plain_bwd, "decay_decode": _plain_decode,
          "tree": _plain_tree, "tree_commit": _plain_commit, "state_store": _plain_store, "state_load": _plain_load}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the work of a pass

def work(case):
    op, Hv = case["op"], case["Hv"]
    st = Hv * D * D * 4                                   # one sequence's states, bytes
    if op == "state_store" or op == "state_load":
        return {"bytes": case["N"] * (st + st // 4 + Hv * D * 4), "flops": case["N"] * Hv * D * D * 2}
    Hqk, e = case["Hqk"], 4 if case["dtype"] == "fp32" else 2
    row = lambda qk, vv: D * e * (qk * Hqk + vv * Hv)     # noqa: E731  bytes of one token's rows
    if op == "decay_varlen":
        tokens, N = int(_lengths(case).sum()), case["N"]
        return {"bytes": tokens * row(2, 2) + N * st * (2 if case["s0"] else 1), "flops": tokens * Hv * 4 * D * D}
    if op == "decay_decode":
        return {"bytes": case["B"] * (row(2, 2) + 2 * st), "flops": case["B"] * Hv * 4 * D * D}
    if op == "tree":                                      # two products with the state, node by node ones besides
        n, B = case["n"], case["B"]
        rule = 2 if case["rule"] == "delta" else 1
        return {"bytes": B * (n * (row(2, 2) + (8 * Hv if rule == 2 else 0)) + st),
                "flops": B * Hv * (rule * 2 * n * D * D + rule * 2 * n * n * D)}
    if op == "tree_commit":                               # half of the nodes' rows, and the states in and out
        n, B = case["n"], case["B"]
        return {"bytes": B * (n / 2 * row(1, 1) + 2 * st), "flops": B * Hv * n / 2 * 4 * D * D}
    B, T = case["B"], case["T"]
    if op == "decay_fwd":
        return {"bytes": B * (T * row(2, 2) + st * (2 if case["s0"] else 1)), "flops": B * T * Hv * 4 * D * D}
    return {"bytes": B * (T * row(4, 3) + st * (3 if case["s0"] else 1)), "flops": B * T * Hv * 10 * D * D}


# ------------------------------------------------------------------ 64-bit results, token by token

def _heads64(x, Hv):
    return x.double().repeat_interleave(Hv // x.shape[-2], dim=-2)


def _exact_rows(s, pieces):
    """The recurrence for [B, T] rows with lengths `pieces` (all T where None)."""
    Hv = s["case"]["Hv"]
    q, k, v = (_heads64(s[n], Hv) for n in ("q", "k", "v"))
    lam = s["decay"].double()[:, None, None]
    B, T = q.shape[:2]
    S = torch.zeros(B, Hv, D, D, dtype=torch.float64, device=q.device) if s["S0"] is None else s["S0"].double()
    o = torch.empty_like(v)
    for t in range(T):
        new = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = new if pieces is None else torch.where((t < pieces)[:, None, None, None], new, S)
        o[:, t] = torch.einsum("bhij,bhi->bhj", S, q[:, t])
    return o, S


def _exact_tree(s):
    """Every node's own state, from its parent's."""
    c = s["case"]
    B, n, Hv = c["B"], c["n"], c["Hv"]
    k, v = _heads64(s["k"], Hv), s["v"].double()
    q = _heads64(s["q"], Hv)
    base = s["pool"][s["slots"].long()].double()
    states = torch.zeros(n + 1, B, Hv, D, D, dtype=torch.float64, device=k.device)
    states[n] = base
    par = s["parents"].cpu().tolist()
    live = [[False] * n for _ in range(B)]
    o = torch.zeros_like(v)
    rows = torch.arange(B, device=k.device)
    for i in range(n):
        src = []
        for b in range(B):
            p = par[b][i]
            live[b][i] = p == -1 or (0 <= p < i and live[b][p])
            src.append(p if 0 <= p < i else n)
        S = states[torch.tensor(src, device=k.device), rows]
        ki, vi = k[:, i], v[:, i]
        if c["rule"] == "delta":
            a, be = s["alpha"][:, i].double()[..., None], s["beta"][:, i].double()[..., None]
            u = be * (vi - a * torch.einsum("bhij,bhi->bhj", S, ki))
            S = a[..., None] * S + ki[..., :, None] * u[..., None, :]
        else:
            S = s["decay"].double()[:, None, None] * S + ki[..., :, None] * vi[..., None, :]
        states[i] = S
        on = torch.tensor([live[b][i] for b in range(B)], device=k.device)
        o[:, i] = torch.einsum("bhij,bhi->bhj", S, q[:, i]) * on[:, None, None]
    return o, states, live


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "decay_fwd":
        return _exact_rows(s, None)
    if op == "decay_varlen":
        cu = s["cu"].tolist()
        L = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device="cuda")
        pad = {"case": case, "decay": s["decay"], "S0": s["S0"]}
        for name in ("q", "k", "v"):
            pad[name] = torch.nn.utils.rnn.pad_sequence([s[name][a:b] for a, b in zip(cu, cu[1:])], batch_first=True)
        o, S = _exact_rows(pad, L)
        return torch.cat([o[i, :b - a] for i, (a, b) in enumerate(zip(cu, cu[1:]))]), S
    if op == "decay_bwd":
        B, T, Hqk, Hv = case["B"], case["T"], case["Hqk"], case["Hv"]
        q, k, v, g = (_heads64(s[n], Hv) for n in ("q", "k", "v", "dO"))
        lam = s["decay"].double()[:, None, None]
        zero = torch.zeros(B, Hv, D, D, dtype=torch.float64, device="cuda")
        S = zero.clone() if s["S0"] is None else s["S0"].double()
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(v)
        for t in range(T):
            S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
            dq[:, t] = torch.einsum("bhij,bhj->bhi", S, g[:, t])
        G = zero if s["dS_final"] is None else s["dS_final"].double()
        for t in range(T - 1, -1, -1):
            G = G + q[:, t, :, :, None] * g[:, t, :, None, :]
            dk[:, t] = torch.einsum("bhij,bhj->bhi", G, v[:, t])
            dv[:, t] = torch.einsum("bhij,bhi->bhj", G, k[:, t])
            G = lam * G
        share = lambda x: x.reshape(B, T, Hqk, Hv // Hqk, D).sum(3)  # noqa: E731
        return share(dq), share(dk), dv, G
    if op == "decay_decode":
        Hv = case["Hv"]
        q, k, v = (_heads64(s[n], Hv) for n in ("q", "k", "v"))
        pool = s["pool"].double()
        at = s["slots"].tolist() if case["slots"] else list(range(case["B"]))
        o = torch.empty_like(v)
        for b, i in enumerate(at):
            pool[i] = s["decay"].double()[:, None, None] * pool[i] + torch.einsum("hi,hj->hij", k[b], v[b])
            o[b] = torch.einsum("hij,hi->hj", pool[i], q[b])
        return o, pool
    if op == "tree":
        return _exact_tree(s)[0]
    if op == "tree_commit":
        _, states, live = _exact_tree(s)
        pool = s["pool"].double()
        for b, (slot, leaf) in enumerate(zip(s["slots"].tolist(), s["accepted"].tolist())):
            if leaf >= 0 and live[b][leaf]:
                pool[slot] = states[leaf, b]
        return pool
    qmax = _QMAX[case["format"]]
    if op == "state_store":                   # the definition's 32-bit roundings, each done from 64 bits
        codes, scales = s["codes"].float(), s["scales"].double()
        for i, j in zip(s["slots"].tolist(), s["cache_slots"].tolist()):
            x = s["pool"][i].double()
            top = x.abs().max(-1, keepdim=True).values
            inv = (qmax / top).float().double()
            y = (x * inv).float().double()
            y = torch.where(top < _TINY, torch.zeros_like(y), y)
            codes[j] = torch.round(y).clamp(-qmax, qmax).float() if case["format"] == "int8" else y.float().to(torch.float8_e4m3fn).float()
            scales[j] = torch.where(top < _TINY, torch.zeros_like(top), top / qmax)[..., 0]
        return (codes.to(torch.int8) if case["format"] == "int8" else codes.double()), scales
    pool = s["pool"].double()
    for i, j in zip(s["slots"].tolist(), s["cache_slots"].tolist()):
        pool[i] = s["codes"].view(torch.int8)[j].view(s["codes"].dtype).double() * s["scales"][j].double()[..., None]
    return pool
