"""GPU parity of the delta-rule trees along deep paths, held to bounds that do not grow with the depth."""
import numpy as np
import pytest
import torch

from test_gpu_tree import DTYPES, IDS, bushy, chain, commit, problem, verify
from tree_bounds import compare, delta_trees

pytestmark = pytest.mark.gpu


def shapes(n):
    """A chain, a bushy tree, a chain with a side node at every third step."""
    comb = [-1]
    for i in range(1, n):
        comb.append(i - 1 if i % 3 else max(i - 2, 0))
    return torch.cat([chain(1, n), bushy(1, n, seed=n), torch.tensor([comb], dtype=torch.int32)])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [9, 17, 33, 48, 49, 64])
def test_verification(dtype, n):
    d = problem(3, n, 2, 6, dtype, 750 + n)
    parents = shapes(n)
    o = verify(d, parents, "delta").double().cpu().numpy()
    for b, t in enumerate(delta_trees(d, parents)):
        bound = t.verification() + (2.0 ** -8 * np.abs(t.o) if dtype == torch.bfloat16 else 2.0 ** -24 * np.abs(t.o))
        for i, path in enumerate(t.paths):
            if path is not None:
                compare(o[b, i], t.o[i], bound[i], f"tree {b}, node {i} at depth {len(path)}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [9, 34, 63, 64])
def test_commit(dtype, n):
    d = problem(6, n, 1, 3, dtype, 770 + n)
    parents = torch.cat([chain(5, n), shapes(n)[2:]])
    accepted = torch.tensor([n - 1, n - 2, n - 3, n - 4, n // 2, n - 1], dtype=torch.int32)
    pool = commit(d, parents, accepted, "delta").double().cpu().numpy()
    for b, t in enumerate(delta_trees(d, parents)):
        leaf = int(accepted[b])
        bound = np.broadcast_to(t.commit(leaf)[:, None, :], t.state[leaf].shape)
        compare(pool[int(d["slots"][b])], t.state[leaf], bound, f"sequence {b}, depth {len(t.paths[leaf])}", sharp=0.02)
