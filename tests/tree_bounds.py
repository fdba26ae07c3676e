"""Error bounds of the delta-rule trees that do not grow along a path.

A majorant of the delta rule adds the rank-one correction that the rule subtracts, so it grows
with the depth where the rule itself forgets.  Here an error is carried by the rule's own
transition instead.  Write the computed update rows as u~_i, each the exact function of the
rows before it plus a local error eps_i, and let S~_i = alpha_i S~_p + k_i u~_i^T with exact
arithmetic.  By induction over the path the errors E_i = S~_i - S_i obey

    E_i = M_i E_p + k_i eps_i^T,   M_i = alpha_i (I - beta_i k_i k_i^T),

and |M_i| = alpha_i max(1, |1 - beta_i |k_i|^2|) is below one here.  Column by column, in the
2-norm: |E_i| <= |M_i| |E_p| + |k_i| |eps_i|, and o_i = S~_i^T q_i is off by |q_i| |E_i| and what
its own sums add.  eps_i counts, relative to what a dot product of two vectors can reach (the
product of their norms):

    dots   bf16: S in two pieces of 8 truncated bits each (2^-14) and sixteen accumulations that
           truncate (2^-22 each); fp32: two dropped products of pieces (2^-7 and 2^-14, twice), six
           truncating MMAs in each of eight steps (2^-22 of a step's share, so 6 of the whole, and
           8 additions)
    grams  bf16 products are exact; eight truncating accumulations; fp32 as the dots
    gates  a path's log2 in 64 bits from fp32 logarithms (2^-23 of it, 2^-23 for each at least),
           and an fp32 power
    sums   one addition for every ancestor, and four products around them
"""
import numpy as np

F32, MMA = 2.0 ** -24, 2.0 ** -22
DOT = {True: 2.0 ** -14 + 16 * MMA, False: 2.0 ** -20 + 6 * MMA + 8 * F32}
GRAM = {True: 8 * MMA + F32, False: 2.0 ** -20 + 48 * MMA}


def _np(x):
    return np.asarray(x.double().cpu().numpy(), dtype=np.float64)


def paths(parents):
    """Nodes from the root down to each node, itself included; None for padding."""
    out = []
    for i, p in enumerate(parents):
        up = None if not -1 <= p < i else [] if p == -1 else out[p]
        out.append(None if up is None else up + [i])
    return out


class DeltaTree:
    """Exact values of one sequence (norms over the key dimension) and the bounds of its nodes."""

    def __init__(self, q, k, v, parents, S, alpha, beta, bf16):
        n, Hv = v.shape[:2]
        q, k = np.repeat(q, Hv // q.shape[1], axis=1), np.repeat(k, Hv // k.shape[1], axis=1)
        self.paths = paths(parents)
        self.kn, self.qn = np.linalg.norm(k, axis=-1)[..., None], np.linalg.norm(q, axis=-1)[..., None]     # [n, Hv, 1]
        self.alpha, self.beta, self.v = alpha[..., None], beta[..., None], np.abs(v)
        self.lg = np.log2(alpha)[..., None]
        self.rootn = np.linalg.norm(S, axis=1)                       # [Hv, dv]
        self.o, self.u = np.zeros_like(v), np.zeros_like(v)
        self.norm, self.state = np.zeros((n, Hv, v.shape[-1])), [None] * n
        self.m = self.alpha * np.maximum(1.0, np.abs(1.0 - self.beta * self.kn ** 2))
        for i, path in enumerate(self.paths):
            if path is None:
                continue
            P = S if len(path) == 1 else self.state[path[-2]]
            a, b = self.alpha[i], self.beta[i]
            self.u[i] = b * (v[i] - a * np.einsum("hij,hi->hj", P, k[i]))
            self.state[i] = a[..., None] * P + k[i][:, :, None] * self.u[i][:, None, :]
            self.o[i] = np.einsum("hij,hi->hj", self.state[i], q[i])
            self.norm[i] = np.linalg.norm(self.state[i], axis=1)
        self.bf16 = bf16

    def _sums(self, path, xn, last):
        """Errors of x^T S along a path's expanded form: (relative to every term, its additions)."""
        i, gate = path[-1], 0.0
        terms, errors = 0.0, 0.0
        for j in reversed(path):                                     # gate: log2 of the product below j down to i
            if j != i or last:
                t = 2.0 ** gate * xn * self.kn[j] * np.abs(self.u[j])
                terms, errors = terms + t, errors + t * (GRAM[self.bf16] + 2.0 ** -23 * (np.abs(gate) + len(path) + 4))
            gate = gate + self.lg[j]
        t = 2.0 ** gate * xn * self.rootn
        errors = errors + t * (DOT[self.bf16] + 2.0 ** -23 * (np.abs(gate) + len(path) + 4))
        return terms + t, errors

    def verification(self):
        """|o~ - o| of every node before its rounding."""
        E, out = np.zeros_like(self.norm), np.zeros_like(self.norm)
        for i, path in enumerate(self.paths):
            if path is None:
                continue
            adds = (len(path) + 4) * F32
            terms, errors = self._sums(path, self.kn[i], False)
            eps = self.beta[i] * (errors + adds * (terms + self.v[i]))
            E[i] = self.m[i] * (E[path[-2]] if len(path) > 1 else 0.0) + self.kn[i] * eps
            terms, errors = self._sums(path, self.qn[i], True)
            out[i] = self.qn[i] * E[i] + errors + adds * terms
        return out

    def commit(self, leaf):
        """Bound of every column's error (2-norm, so of each element too) of the state after `leaf`:
        token updates in fp32, four nodes at a time.  A dot product of 128 in partial sums is below 24
        roundings, a group's update rounds the state and each write at most ten times."""
        path = self.paths[leaf]
        E, start = 0.0, self.rootn
        for g in range(0, len(path), 4):
            group, writes = path[g:g + 4], 0.0
            for j in group:
                reach = self.kn[j] * (start + writes)                # what S^T k_j and its terms can reach
                eps = self.beta[j] * (32 * F32 * reach + 4 * F32 * self.v[j])
                writes = writes + self.kn[j] * np.abs(self.u[j])
                E = self.m[j] * E + self.kn[j] * eps
            E = E + 10 * F32 * (start + writes)
            start = self.norm[group[-1]]
        return E


def delta_trees(d, parents, slots=None):
    """One DeltaTree for each sequence of a problem (see test_gpu_tree)."""
    slots = d["slots"].tolist() if slots is None else slots
    bf16 = str(d["q"].dtype) == "torch.bfloat16"
    x = {n: _np(d[n]) for n in ("q", "k", "v", "alpha", "beta", "pool")}
    return [DeltaTree(x["q"][b], x["k"][b], x["v"][b], parents[b].tolist(), x["pool"][s], x["alpha"][b], x["beta"][b], bf16)
            for b, s in enumerate(slots)]


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def compare(got, ref, bound, what, sharp=0.1):
    """got within bound of ref, and the bound itself well below the values (a bound that anything
    meets checks nothing)."""
    bound = 1.01 * bound
    assert np.median(bound) <= sharp * rms(ref), f"{what}: bound {np.median(bound):.2e} against values of {rms(ref):.2e}"
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err / bound)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond the bound; worst at {at}: got {got[at]}, "
                             f"want {ref[at]}, bound {bound[at]}")
