"""Tree attention where it can go wrong: waits that run out, logits and values at the ends of their range, keys that
are not finite, many rows over a long context."""
import numpy as np
import pytest

from spec_helpers import SpecCache, random_parents, tree_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import oracle
    oracle.build()
    from int4_kivi_quantized_s4kv_b200 import build
    build.build()


def make_tree(rng, nodes, heads, group, newest):
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    n = int(cu[-1])
    parents = np.concatenate([random_parents(rng, int(x), newest) for x in nodes]).astype(np.int32)
    q = rng.standard_normal((n, heads * group, 128)).astype(np.float16)
    k = rng.standard_normal((n, heads, 128)).astype(np.float16)
    v = rng.standard_normal((n, heads, 128)).astype(np.float16)
    return cu, parents, q, k, v


def run_tree(c, q, k, v, cu, parents, max_nodes, ws=None, sm_scale=None):
    import torch
    qd = c.dev(q)
    out = torch.full_like(qd, float("nan"))
    if ws is None:
        ws = c.S.tree_workspace(q.shape[1], c.H, len(cu) - 1, max_nodes)
    c.S.s4kv_tree_attention(c.gpu, qd, c.dev(k), c.dev(v), c.dev(cu), c.dev(parents), c.lens_dev, c.bt_dev, out, max_nodes,
                            ws, sm_scale)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("group_of_rows", [0, 1])
def test_a_wait_that_runs_out(group_of_rows):
    """A counter of pieces that can never reach its count (its low half is about to wrap): the CTAs that share the unit
    give up after a bounded time, say so, and leave; units of one CTA are right, and with the workspace zero-filled again
    the next call is."""
    rng = np.random.default_rng(31)
    nodes = [16, 2]
    c = SpecCache([3000, 50], 1, seed=32, key_scale=np.ones((1, 128)))
    cu, parents, q, k, v = make_tree(rng, nodes, 1, 4, 3)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    ws = c.S.tree_workspace(4, 1, 2, 16)
    counters = ws[-2 * 2 * 4:].view(c.lens_dev.dtype)  # one unit a sequence, two groups of rows a unit
    counters[group_of_rows] = 0xFFFF
    out = run_tree(c, q, k, v, cu, parents, 16, ws)
    assert c.S.s4kv_get_error(c.gpu) == c.S.EFLAG_TIMEOUT
    assert (np.abs(out - ref) <= bound)[16:].all()
    ws.zero_()
    out = run_tree(c, q, k, v, cu, parents, 16, ws)
    assert c.S.s4kv_get_error(c.gpu) == 0
    assert (np.abs(out - ref) <= bound).all()


@pytest.mark.parametrize("key,query,sm_scale,bits", [(1000.0, 128.0, 8e-7, 4), (4096.0, 128.0, 2e-7, 4), (4096.0, 300.0, 8e-8, 8),
                                                     (12000.0, 50000.0, 1.5e-10, 4), (12000.0, 50000.0, 1.5e-10, 2)])
def test_zero_points_over_the_whole_range(key, query, sm_scale, bits):
    """Queries of one sign against zero points of one sign: their product's sum is 128 times the largest of them, far
    beyond fp16 from finite fp16 inputs, and the answer is finite."""
    rng = np.random.default_rng(33)
    c = SpecCache([200, 31, 640], 2, bits, seed=34, key_scale=np.full((2, 128), key))
    cu, parents, q, k, v = make_tree(rng, [7, 5, 3], 2, 4, 2)
    q = (query * (1 + 0.02 * q.astype(np.float64))).astype(np.float16)
    k = (key * k.astype(np.float64)).astype(np.float16)
    assert np.isfinite(k).all() and all(np.isfinite(x).all() for x in c.k)
    ref, bound = tree_reference(c, q, k, v, cu, parents, sm_scale)
    out = run_tree(c, q, k, v, cu, parents, 7, sm_scale=sm_scale)
    assert (np.abs(out - ref) <= bound).all()
