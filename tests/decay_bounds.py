"""Error bounds of the GPU tests of the decay rule and the trees.

A result is a sum of products; `maj` is the same sum over absolute values (oracle.decay).  A
rounding of relative size u inside the sum moves the result by at most u * maj, one of the
result itself by u * |ref|.  Half a step is 2^-8 relative in bf16 and 2^-24 in fp32.
"""
import numpy as np

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def check(got, ref, maj, u_out, u_terms, what):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    bound = 1.001 * (u_out * np.abs(ref) + u_terms * maj) + 1e-25 * (1 + maj.max(initial=0))
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err / bound)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond the bound; worst at {at}: got {got[at]}, "
                             f"want {ref[at]}, bound {bound[at]}")


def chunks(T):
    return -(-T // 64)


def out_bounds(bf16, T):
    """(u_out, u_terms) of o, dq, dk, dv.  bf16: the result, and H or P once each (a term has one of
    them); the fp32 rest is below 2^-14.  fp32: a term passes a dot product of 128, the decay, a sum of
    64, and 64 + 2 additions for every chunk that its state has passed."""
    if bf16:
        return BF16, BF16 + 2.0 ** -14
    return 0.0, (128 + 64 + 8 + 66 * chunks(T)) * F32


def state_bounds(bf16, T):
    """u_terms of a state.  fp32: 64 + 2 additions per chunk.  bf16: weight and product (2), twelve MMAs
    that truncate (2^-22 each), two additions per chunk; 40 for joining segments."""
    return ((66 if not bf16 else 52) * chunks(T) + 48) * F32


def tree_bounds(bf16, n):
    """bf16: the result, and S in two truncated pieces (2^-14) under k and under q, one after the other;
    fp32: dot products of 128 in six truncating MMAs per 16 columns, and a substitution of n steps."""
    if bf16:
        return BF16, 2.0 ** -13 + (300 + 4 * n) * F32
    return 0.0, (600 + 70 * n) * F32


def commit_bound(path):
    """Per node a dot product of 128 and a few more; the state passes three roundings."""
    return 140 * max(path, 1) * F32
