"""The depth-independent bounds of the delta-rule trees: they agree with the oracle's values, stay far
below them at every node, and mistakes at the deepest nodes fall outside."""
import numpy as np
import pytest
import torch

from oracle import decay as ref
from test_gpu_tree import SHAPES, bushy, chain, problem
from tree_bounds import compare, delta_trees, rms

U_OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
DTYPES = [torch.bfloat16, torch.float32]


def oracle(d, parents):
    return ref.tree(d["q"], d["k"], d["v"], parents.numpy(), d["pool"][d["slots"].long()], alpha=d["alpha"], beta=d["beta"])


@pytest.mark.parametrize("shape", list(SHAPES))
def test_values_are_the_oracles(shape):
    d = problem(2, 64, 1, 3, torch.bfloat16, 700)
    parents = SHAPES[shape](2, 64)
    o, S, alive = oracle(d, parents)
    for b, t in enumerate(delta_trees(d, parents)):
        assert [p is not None for p in t.paths] == alive[b].tolist()
        assert np.abs(t.o - o[b]).max() < 1e-12
        for i in np.flatnonzero(alive[b]):
            assert np.abs(t.state[i] - S[b, i]).max() < 1e-12


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [17, 33, 64])
def test_bounds_do_not_grow_with_the_depth(dtype, n):
    d = problem(2, n, 1, 3, dtype, 710 + n)
    for t in delta_trees(d, chain(2, n)):
        bound = t.verification()
        for i in range(n):
            assert np.median(bound[i]) <= 0.02 * rms(t.o[i]), i
            assert np.median(t.commit(i)) <= 2e-3 * rms(t.state[i]), i


@pytest.mark.parametrize("dtype", DTYPES)
def test_mistakes_on_deep_paths_are_seen(dtype):
    """Planted in the oracle: outputs of zero, ancestors past bit 31 lost, the last ancestor lost, a
    commit that stops before its last node or before its last group."""
    d = problem(1, 64, 1, 3, dtype, 730)
    parents = chain(1, 64)
    (t,) = delta_trees(d, parents)
    bound, kept = t.verification() + U_OUT[dtype] * np.abs(t.o), np.float64(t.o)
    for i in (40, 62, 63):
        compare(kept[i], t.o[i], bound[i], "as it is")
        with pytest.raises(AssertionError, match="beyond"):
            compare(0 * kept[i], t.o[i], bound[i], "zeros")
        path = t.paths[i]
        q, k = (np.repeat(x[0].double().numpy(), 3, axis=1) for x in (d["q"], d["k"]))
        for lost in ([j for j in path[:-1] if j >= 32], [path[-2]]):
            gate = 2.0 ** (np.cumsum(t.lg[:, :, 0], axis=0)[i] - np.cumsum(t.lg[:, :, 0], axis=0))     # [n, Hv]
            wrong = kept[i] - sum((gate[j] * (q[i] * k[j]).sum(-1))[:, None] * t.u[j] for j in lost)
            with pytest.raises(AssertionError, match="beyond"):
                compare(wrong, t.o[i], bound[i], "ancestors lost")
    col = t.commit(63)[:, None, :]
    compare(t.state[63], t.state[63], np.broadcast_to(col, t.state[63].shape), "as it is", sharp=0.02)
    for early in (62, 59):
        with pytest.raises(AssertionError, match="beyond"):
            compare(t.state[early], t.state[63], np.broadcast_to(col, t.state[63].shape), "stopped early", sharp=0.02)


def test_the_growing_majorant_would_not_see_them():
    """Why these bounds are beside the majorants of oracle.decay."""
    d = problem(1, 64, 1, 3, torch.bfloat16, 730)
    parents = chain(1, 64)
    o, _, _ = oracle(d, parents)
    mo, _, _ = ref.tree(d["q"], d["k"], d["v"], parents.numpy(), d["pool"][d["slots"].long()], alpha=d["alpha"],
                        beta=d["beta"], majorant=True)
    assert np.median(2.0 ** -13 * mo[0, 63]) > rms(o[0, 63])


def test_padding_has_no_path():
    d = problem(2, 24, 1, 1, torch.float32, 740)
    t = delta_trees(d, bushy(2, 24))[1]
    assert t.paths[-1] is None and (t.verification()[-1] == 0).all()
