"""Refusals of the constant-decay, tree and state-cache entry points (no GPU: every check
comes before any launch), and of their binding."""
import ctypes
import os

import pytest
import torch

from linear_attention_recurrence_07_b200 import binding

FAKE = ctypes.c_void_p(0x1000)          # aligned, never dereferenced: checks reject first
ODD = ctypes.c_void_p(0x1004)           # 4-byte aligned only
BYTE = ctypes.c_void_p(0x1001)
INVALID, UNSUPPORTED = binding.GDN_ERR_INVALID_ARG, binding.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIBRARY_PATH):
        from linear_attention_recurrence_07_b200 import build
        build.build()
    return binding.library()


def caller(fn, order, defaults):
    def call(**change):
        args = {**defaults, **change}
        return fn(*(args[n] for n in order.split()))
    return call


def entries(lib):
    """name -> (call with changes, required pointers, 4-byte pointers, n-like zero that makes it a no-op)."""
    size = dict(Hqk=1, Hv=1, dk=128, dv=128, dtype=1, stream=None)
    P = lambda *names: {n: FAKE for n in names}  # noqa: E731
    return {
        "fwd": (caller(lib.gdn_decay_fwd, "q k v decay S0 o SF B T Hqk Hv dk dv dtype ws wb stream",
                       {**size, **P("q", "k", "v", "decay", "o"), "S0": None, "SF": None, "B": 1, "T": 64, "ws": None, "wb": 0}),
                ["q", "k", "v", "decay", "o"], [], "B"),
        "varlen": (caller(lib.gdn_decay_fwd_varlen, "q k v decay S0 o SF cu N T Hqk Hv dk dv dtype stream",
                          {**size, **P("q", "k", "v", "decay", "o", "cu"), "S0": None, "SF": None, "N": 1, "T": 64}),
                   ["q", "k", "v", "decay", "o", "cu"], ["cu"], "N"),
        "step": (caller(lib.gdn_decay_decode_step, "q k v decay S o SN B Hqk Hv dk dv dtype stream",
                        {**size, **P("q", "k", "v", "decay", "S", "o", "SN"), "B": 1}),
                 ["q", "k", "v", "decay", "S", "o", "SN"], [], "B"),
        "slots": (caller(lib.gdn_decay_decode_step_slots, "q k v decay pool slots o B n_slots Hqk Hv dk dv dtype stream",
                         {**size, **P("q", "k", "v", "decay", "pool", "slots", "o"), "B": 1, "n_slots": 1}),
                  ["q", "k", "v", "decay", "pool", "slots", "o"], ["slots"], "B"),
        "bwd": (caller(lib.gdn_decay_bwd, "q k v decay S0 dO dSF dq dk_ dv_ dS0 B T Hqk Hv dk dv dtype ws wb stream",
                       {**size, **P("q", "k", "v", "decay", "dO", "dq", "dk_", "dv_"), "S0": None, "dSF": None, "dS0": None,
                        "B": 1, "T": 64, "ws": None, "wb": 0}),
                ["q", "k", "v", "decay", "dO", "dq", "dk_", "dv_"], [], "B"),
        "tree": (caller(lib.gdn_decode_tree, "q k v alpha beta parents pool slots o B n n_slots Hqk Hv dk dv dtype stream",
                        {**size, **P("q", "k", "v", "alpha", "beta", "parents", "pool", "slots", "o"), "B": 1, "n": 4, "n_slots": 1}),
                 ["q", "k", "v", "alpha", "beta", "parents", "pool", "o"], ["parents", "slots"], "B"),
        "commit": (caller(lib.gdn_tree_commit, "k v alpha beta parents acc pool slots B n n_slots Hqk Hv dk dv dtype stream",
                          {**size, **P("k", "v", "alpha", "beta", "parents", "acc", "pool", "slots"), "B": 1, "n": 4, "n_slots": 1}),
                   ["k", "v", "alpha", "beta", "parents", "acc", "pool"], ["parents", "acc", "slots"], "B"),
        "decay_tree": (caller(lib.gdn_decay_decode_tree, "q k v decay parents pool slots o B n n_slots Hqk Hv dk dv dtype stream",
                              {**size, **P("q", "k", "v", "decay", "parents", "pool", "slots", "o"), "B": 1, "n": 4, "n_slots": 1}),
                       ["q", "k", "v", "decay", "parents", "pool", "o"], ["parents", "slots"], "B"),
        "decay_commit": (caller(lib.gdn_decay_tree_commit, "k v decay parents acc pool slots B n n_slots Hqk Hv dk dv dtype stream",
                                {**size, **P("k", "v", "decay", "parents", "acc", "pool", "slots"), "B": 1, "n": 4, "n_slots": 1}),
                         ["k", "v", "decay", "parents", "acc", "pool"], ["parents", "acc", "slots"], "B"),
    }


NAMES = ["fwd", "varlen", "step", "slots", "bwd", "tree", "commit", "decay_tree", "decay_commit"]


@pytest.mark.parametrize("name", NAMES)
def test_sizes_and_types(lib, name):
    call, _, _, count = entries(lib)[name]
    assert call(**{count: -1}) == INVALID
    assert call(Hqk=0) == INVALID
    assert call(Hv=0) == INVALID
    assert call(dtype=7) == INVALID
    assert call(Hqk=2, Hv=3) == UNSUPPORTED
    assert call(dk=64) == UNSUPPORTED
    assert call(dv=256) == UNSUPPORTED
    assert call(**{count: 0}) == binding.GDN_OK


@pytest.mark.parametrize("name", NAMES)
def test_pointers(lib, name):
    call, required, words, _ = entries(lib)[name]
    for p in required:
        assert call(**{p: None}) == INVALID, p
        assert call(**{p: BYTE}) == INVALID, p
        if p not in words:
            assert call(**{p: ODD}) == INVALID, p


def test_limits(lib):
    e = entries(lib)
    for name in ("fwd", "varlen", "bwd"):
        call, _, _, count = e[name]
        assert call(T=-1) == INVALID
        assert call(**{count: 65536}) == UNSUPPORTED
        assert call(Hv=65536) == UNSUPPORTED
    for name in ("step", "slots", "tree", "commit", "decay_tree", "decay_commit"):
        assert e[name][0](B=1 << 20, Hv=1 << 12) == UNSUPPORTED
    for name in ("tree", "commit", "decay_tree", "decay_commit"):
        call = e[name][0]
        assert call(n=0) == INVALID
        assert call(n=65) == UNSUPPORTED
        assert call(n_slots=-1) == INVALID
        assert call(slots=None, B=2, n_slots=1) == INVALID
    assert e["slots"][0](n_slots=-1) == INVALID


def test_workspaces(lib):
    e = entries(lib)
    need = lib.gdn_decay_fwd_workspace(1, 4096, 2, 128, 128, 1)
    assert need > 0 and need % (2 * 65536) == 0
    big = dict(T=4096, Hqk=2, Hv=2)
    assert e["fwd"][0](**big) == INVALID
    assert e["fwd"][0](**big, ws=FAKE, wb=need - 1) == INVALID
    assert e["fwd"][0](**big, ws=ctypes.c_void_p(0x1010), wb=need) == INVALID
    need = lib.gdn_decay_bwd_workspace(1, 64, 1, 3, 128, 128, 0)
    assert need == 2 * 64 * 3 * 128 * 4
    assert e["bwd"][0](Hv=3, ws=FAKE, wb=need - 1) == INVALID
    assert lib.gdn_decay_fwd_workspace(1, 64, 1, 128, 128, 1) == 0
    assert lib.gdn_decay_fwd_workspace(1, 4096, 1, 64, 128, 1) == 0
    assert lib.gdn_decay_fwd_workspace(-1, 4096, 1, 128, 128, 1) == 0
    assert lib.gdn_decay_bwd_workspace(1, 64, 2, 3, 128, 128, 0) == 0


def test_empty_sequences_need_no_tokens(lib):
    e = entries(lib)
    assert e["fwd"][0](T=0, q=None, k=None, v=None, decay=None, o=None) == binding.GDN_OK
    assert e["bwd"][0](T=0, q=None, k=None, v=None, decay=None, dO=None, dq=None, dk_=None, dv_=None) == binding.GDN_OK


def test_state_cache(lib):
    base = dict(pool=FAKE, slots=FAKE, codes=FAKE, scales=FAKE, cs=FAKE, N=1, n_slots=1, n_cache=1, Hv=1, dk=128, dv=128,
                code=0, stream=None)
    store = caller(lib.gdn_state_store, "pool slots codes scales cs N n_slots n_cache Hv dk dv code stream", base)
    load = caller(lib.gdn_state_load, "codes scales cs pool slots N n_slots n_cache Hv dk dv code stream", base)
    for call in (store, load):
        for bad in (dict(N=-1), dict(n_slots=-1), dict(n_cache=-1), dict(code=2), dict(Hv=0), dict(pool=None), dict(slots=None),
                    dict(codes=None), dict(scales=None), dict(cs=None), dict(pool=ODD), dict(codes=ODD), dict(scales=ODD),
                    dict(slots=BYTE), dict(cs=BYTE)):
            assert call(**bad) == INVALID, bad
        assert call(dk=64) == UNSUPPORTED
        assert call(N=1 << 20, Hv=1 << 12) == UNSUPPORTED
        assert call(N=0, pool=None, slots=None) == binding.GDN_OK


def test_binding_refuses_wrong_tensors():
    """Host tensors, shapes and types are refused before the library is called."""
    x = torch.zeros(1, 4, 1, 128)
    lam, S = torch.ones(1), torch.zeros(1, 1, 128, 128)
    with pytest.raises(binding.GdnError, match="CUDA"):
        binding.gdn_decay_fwd(x, x, x, lam, None, x, None)
    with pytest.raises(binding.GdnError, match="dimensions"):
        binding.gdn_decay_fwd(x[0], x, x, lam, None, x, None)
    with pytest.raises(binding.GdnError, match="dtype"):
        binding.gdn_decay_bwd(x.half(), x, x, lam, None, x, None, x, x, x, None)
    with pytest.raises(binding.GdnError, match="CUDA"):
        binding.gdn_decay_decode_step(x[0], x[0], x[0], lam, S, x[0], S)
    with pytest.raises(binding.GdnError, match="dimensions"):
        binding.gdn_decode_tree(x, x, x, lam, lam, lam, S[0], None, x)
    with pytest.raises(binding.GdnError, match="CUDA"):
        binding.gdn_state_store(S, torch.zeros(1, dtype=torch.int32), S.to(torch.int8), torch.zeros(1, 1, 128),
                                torch.zeros(1, dtype=torch.int32))
    with pytest.raises(binding.GdnError, match="required"):
        binding.gdn_decay_fwd_varlen(x[0], x[0], x[0], lam, None, x[0], None, None)
