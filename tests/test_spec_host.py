"""The speculative-decoding calls without a GPU: what they refuse before
anything is launched, and the references that the GPU tests use pinned to what
they stand for."""
import ctypes
import os
import re

import numpy as np
import pytest

from spec_helpers import SpecCache, random_parents, tree_reference, verify_reference

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def S():
    from int4_kivi_quantized_s4kv_b200 import build
    build.build()
    import int4_kivi_quantized_s4kv_b200 as S
    return S


def test_constants(S):
    defs = dict(re.findall(r"#define\s+(S4KV_\w+)\s+(\d+)u?\b", open(os.path.join(ROOT, "include", "s4kv.h")).read()))
    assert int(defs["S4KV_MAX_TREE_NODES"]) == S.MAX_TREE_NODES
    assert int(defs["S4KV_EFLAG_TREE"]) == S.EFLAG_TREE and int(defs["S4KV_EFLAG_PROBS"]) == S.EFLAG_PROBS


FAKE = 0x100000  # a non-null, aligned address that is never dereferenced


def test_tree_attention_refusals(S):
    L, P = S.lib(), ctypes.c_void_p
    c = S.s4kv_cache_t(FAKE, FAKE, FAKE, None, 10, 2, 4, 128, 16)
    bad_dim = S.s4kv_cache_t(FAKE, FAKE, FAKE, None, 10, 2, 4, 64, 16)
    bad_bits = S.s4kv_cache_t(FAKE, FAKE, FAKE, None, 10, 2, 4, 128, 16, 3)

    def call(**kw):
        a = dict(cache=c, q=FAKE, k=FAKE, v=FAKE, hq=8, n=4, cu=FAKE, par=FAKE, sl=FAKE, bt=FAKE, batch=1, maxp=1, most=4,
                 scale=0.088, out=FAKE, ws=FAKE, wsb=1 << 30)
        a.update(kw)
        return L.s4kv_tree_attention(ctypes.byref(a["cache"]) if a["cache"] else None, P(a["q"]), P(a["k"]), P(a["v"]),
                                     a["hq"], a["n"], P(a["cu"]), P(a["par"]), P(a["sl"]), P(a["bt"]), a["batch"],
                                     a["maxp"], a["most"], a["scale"], P(a["out"]), P(a["ws"]), a["wsb"], P(0))

    assert call(cache=None) == S.ERR_INVALID_ARG
    for kw in (dict(cache=bad_dim), dict(cache=bad_bits), dict(hq=18), dict(hq=7), dict(most=65)):
        assert call(**kw) == S.ERR_UNSUPPORTED, kw
    for kw in (dict(n=-1), dict(batch=-1), dict(batch=5), dict(maxp=0), dict(maxp=1 << 27), dict(most=0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=0.0), dict(scale=-1.0)):
        assert call(**kw) == S.ERR_INVALID_ARG, kw
    for name in ("q", "k", "v", "cu", "par", "sl", "bt", "out"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 2}) == S.ERR_INVALID_ARG, name
    assert call(n=0) == S.OK and call(batch=0) == S.OK
    assert call(ws=None) == S.ERR_WORKSPACE and call(ws=FAKE + 8) == S.ERR_WORKSPACE


def test_tree_workspace_refusals(S):
    n = ctypes.c_size_t(0)
    f = S.lib().s4kv_tree_workspace_size
    assert f(8, 2, 1, 4, None) == S.ERR_INVALID_ARG
    assert f(8, 2, -1, 4, ctypes.byref(n)) == S.ERR_INVALID_ARG
    assert f(8, 2, 1, 0, ctypes.byref(n)) == S.ERR_INVALID_ARG
    assert f(8, 2, 1, 65, ctypes.byref(n)) == S.ERR_UNSUPPORTED
    assert f(18, 2, 1, 4, ctypes.byref(n)) == S.ERR_UNSUPPORTED
    assert f(524288, 65536, 65536, 64, ctypes.byref(n)) == S.ERR_INVALID_ARG


def test_verify_refusals(S):
    L, P = S.lib(), ctypes.c_void_p

    def call(**kw):
        a = dict(tok=FAKE, par=FAKE, cu=FAKE, n=4, batch=1, most=4, t=FAKE, ts=100, d=FAKE, ds=100, kind=0, vocab=100,
                 u=FAKE, path=FAKE, ln=FAKE, nxt=FAKE, err=None)
        a.update(kw)
        return L.s4kv_verify_tree(P(a["tok"]), P(a["par"]), P(a["cu"]), a["n"], a["batch"], a["most"], P(a["t"]), a["ts"],
                                  P(a["d"]), a["ds"], a["kind"], a["vocab"], P(a["u"]), P(a["path"]), P(a["ln"]), P(a["nxt"]),
                                  P(a["err"]), P(0))

    assert call(most=65) == S.ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(batch=-1), dict(most=0), dict(vocab=0), dict(kind=3), dict(kind=-1), dict(ts=99),
               dict(ds=99), dict(ts=-100), dict(err=FAKE + 1), dict(t=FAKE + 2), dict(d=FAKE + 2), dict(kind=1, t=FAKE + 1)):
        assert call(**kw) == S.ERR_INVALID_ARG, kw
    for name in ("tok", "par", "cu", "t", "u", "path", "ln", "nxt"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
    for name in ("tok", "par", "cu", "u", "path", "ln", "nxt"):
        assert call(**{name: FAKE + 2}) == S.ERR_INVALID_ARG, name
    assert call(batch=0) == S.OK


def test_append_path_refusals(S):
    L, P = S.lib(), ctypes.c_void_p
    c = S.s4kv_cache_t(FAKE, FAKE, FAKE, None, 10, 2, 4, 128, 16)
    bad_dim = S.s4kv_cache_t(FAKE, FAKE, FAKE, None, 10, 2, 4, 64, 16)
    wide = S.s4kv_cache_t(FAKE, FAKE, FAKE, None, 10, 65536, 70000, 128, 16)

    def call(**kw):
        a = dict(cache=c, k=FAKE, v=FAKE, n=4, cu=FAKE, path=FAKE, ln=FAKE, most=4, sl=FAKE, bt=FAKE, batch=1, maxp=1,
                 new=FAKE + 4096)
        a.update(kw)
        return L.s4kv_append_path(ctypes.byref(a["cache"]) if a["cache"] else None, P(a["k"]), P(a["v"]), a["n"], P(a["cu"]),
                                  P(a["path"]), P(a["ln"]), a["most"], P(a["sl"]), P(a["bt"]), a["batch"], a["maxp"],
                                  P(a["new"]), P(0))

    assert call(cache=None) == S.ERR_INVALID_ARG
    assert call(cache=bad_dim) == S.ERR_UNSUPPORTED and call(most=65) == S.ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(batch=-1), dict(batch=5), dict(maxp=0), dict(maxp=1 << 27), dict(most=0), dict(cache=wide),
               dict(cache=wide, batch=65536), dict(new=FAKE), dict(batch=4, new=FAKE + 12), dict(batch=4, new=FAKE - 12)):
        assert call(**kw) == S.ERR_INVALID_ARG, kw
    for name in ("k", "v", "cu", "path", "ln", "sl", "bt", "new"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 2}) == S.ERR_INVALID_ARG, name
    assert call(batch=0) == S.OK


def test_wrappers_refuse_host_tensors_and_wrong_shapes(S):
    import torch
    t = torch.zeros(3, 10)
    i = torch.zeros(3, dtype=torch.int32)
    cu = torch.zeros(2, dtype=torch.int32)
    path, one = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    u = torch.zeros(3)
    with pytest.raises(ValueError, match="CUDA"):
        S.s4kv_verify_tree(i, i, cu, t, t, u, path, one, one)
    with pytest.raises(ValueError, match="uniforms"):
        S.s4kv_verify_tree(i, i, cu, t, t, u[:2], path, one, one)
    with pytest.raises(ValueError, match="draft_probs"):
        S.s4kv_verify_tree(i, i, cu, t, t[:, :9], u, path, one, one)
    with pytest.raises(TypeError):
        S.s4kv_verify_tree(i, i, cu, t, t.half(), u, path, one, one)
    with pytest.raises(ValueError, match="contiguous"):
        S.s4kv_verify_tree(i, i, cu, torch.zeros(10, 3).t(), None, u, path, one, one)


def test_tree_reference_of_a_chain_is_causal_attention(oracle_mod):
    """A chain of drafted tokens whose keys the oracle appends instead: the same attention (lengths chosen so that
    no page fills, so that nothing is quantized)."""
    rng = np.random.default_rng(0)
    c = SpecCache([33, 4], 2, 4, seed=1, gpu=False)
    cu = np.array([0, 5, 8], np.int32)
    q = rng.standard_normal((8, 4, 128)).astype(np.float16)
    k, v = (rng.standard_normal((8, 2, 128)).astype(np.float16) for _ in range(2))
    parents = np.array([-1, 0, 1, 2, 3, -1, 0, 1], np.int32)
    out, _ = tree_reference(c, q, k, v, cu, parents)
    from int4_kivi_quantized_s4kv_b200 import workloads as W
    after = c.lens + np.array([5, 3], np.int32)
    sm = W.slot_mapping(c.bt, [np.arange(33, 38), np.arange(4, 7)])
    assert c.oc.append(k, v, sm, cu, after, c.bt) == 0
    assert np.abs(out - c.oc.prefill_attention(q, cu, after, c.bt)).max() < 1e-6


def test_tree_reference_siblings_do_not_see_each_other():
    rng = np.random.default_rng(1)
    c = SpecCache([20], 1, 4, seed=2, gpu=False)
    q = np.repeat(rng.standard_normal((1, 1, 128)), 3, 0).astype(np.float16)
    k, v = (rng.standard_normal((3, 1, 128)).astype(np.float16) for _ in range(2))
    cu = np.array([0, 3], np.int32)
    a, _ = tree_reference(c, q, k, v, cu, np.array([-1, 0, 0], np.int32))
    k[1] += 1
    v[1] += 1
    b, _ = tree_reference(c, q, k, v, cu, np.array([-1, 0, 0], np.int32))
    assert np.array_equal(a[2], b[2]) and not np.array_equal(a[1], b[1])


@pytest.mark.parametrize("draws", [1, 2])
def test_verify_reference_gives_the_targets_distribution(draws):
    """Integrated over the draft's draws and a grid of random numbers, the token that follows node 0 is distributed
    as the target's row says, whatever the draft."""
    p = np.array([[0.5, 0.125, 0.375]])
    q = np.array([[0.25, 0.5, 0.25]])
    grid = (np.arange(16) + 0.5) / 16
    got = np.zeros(3)
    import itertools
    for toks in itertools.product(range(3), repeat=draws):
        weight = np.prod([q[0, t] for t in toks])
        for us in itertools.product(grid, repeat=draws + 1):
            rows = 1 + draws
            tok = np.array((0, *toks), np.int32)
            path, ln, nxt = verify_reference(tok, np.array([-1] + [0] * draws, np.int32), np.array([0, rows]),
                                             np.repeat(p, rows, 0), np.repeat(q, rows, 0), np.array(us, np.float32), rows)
            follows = tok[path[0, 1]] if ln[0] > 1 else nxt[0]
            got[follows] += weight / 16 ** (draws + 1)
    assert np.abs(got - p[0]).max() < 1 / 16


def test_verify_reference_without_draft_rows():
    """Children chosen without randomness: accepted with the target's probability of their token."""
    p = np.array([[0.5, 0.25, 0.25]] * 3)
    par, cu = np.array([-1, 0, 0], np.int32), np.array([0, 3])
    grid = (np.arange(32) + 0.5) / 32
    got = np.zeros(3)
    for a in grid:
        for b in grid:
            for u0 in grid[::4]:
                path, ln, nxt = verify_reference(np.array([0, 1, 0], np.int32), par, cu, p, None,
                                                 np.array([u0, a, b], np.float32), 3)
                got[[1, 0][path[0, 1] - 1] if ln[0] > 1 else nxt[0]] += 1
    assert np.abs(got / got.sum() - p[0]).max() < 1 / 32


def test_random_parents_are_trees():
    rng = np.random.default_rng(0)
    for n in (0, 1, 2, 64):
        for newest in (0, 1, 3):
            par = random_parents(rng, n, newest)
            assert len(par) == n and all(-1 <= a < i for i, a in enumerate(par))
