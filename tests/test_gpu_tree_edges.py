"""Tree attention where it can go wrong: waits that run out, logits and values at the ends of their range, keys that
are not finite, many rows over a long context."""
import numpy as np
import pytest

from spec_helpers import SpecCache, random_parents, tree_reference
from tree_helpers import REMAINDER_BOUND, ROWS, SM_SCALE, TOKENS, filled, remainder_case, remainder_error

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


@pytest.mark.parametrize("bad", [float("-inf"), float("nan")])
@pytest.mark.parametrize("length", [0, 5, 300, 304, 5000])
def test_keys_that_are_not_finite(bad, length):
    """A drafted root with -infinity in its key: heads whose query is positive there give it no weight (a softmax over
    the rest, which for the root of an empty cache is none: NaN), heads whose query is negative have an infinite logit: NaN,
    in the rows that see it and in no others.  NaN in the key: NaN in all rows that see it."""
    rng = np.random.default_rng(35)
    nodes = [13, 9]
    c = SpecCache([length, 70], 2, seed=36, key_scale=np.ones((2, 128)))
    cu, parents, q, k, v = make_tree(rng, nodes, 2, 4, 3)
    parents[6], parents[7] = -1, 6  # a second root, which is the bad one
    x = 6
    seen = np.zeros(22, bool)
    for i in range(13):
        a = i
        while a >= 0:
            seen[i] |= a == x
            a = parents[a]
    assert seen[x] and 2 <= seen.sum() < 13
    q[:, :2, 5], q[:, 2:4, 5] = 8, -8
    k[x, 0] = 0
    k[x, 0, 5] = -1100  # as good as -infinity: exp(-774) is 0 in 64 bits
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    if length == 0:
        ref[x, :2] = np.nan
    ref[seen, 2:4] = np.nan
    if np.isnan(bad):
        ref[seen, :4] = np.nan
    k[x, 0, 5] = bad
    out = run_tree(c, q, k, v, cu, parents, 13)
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    good = ~np.isnan(ref)
    assert (np.abs(out - ref)[good] <= bound[good]).all()
    assert c.S.s4kv_get_error(c.gpu) == 0


@pytest.mark.parametrize("level", [-2000.0, -120.0, 0.0, 120.0, 2000.0])
def test_logits_of_one_level_behind_a_key_without_weight(level):
    """The only key of the first tile has the logit -infinity; all logits behind it are near one level, far below or
    above 0 (a channel in which all keys are the same, and so exact)."""
    rng = np.random.default_rng(37)
    keys, values = rng.standard_normal((112, 1, 128)), rng.standard_normal((112, 1, 128))
    keys[:, :, 9] = 16
    c = filled(keys, values)
    q = rng.standard_normal((1, 1, 128)).astype(np.float16)
    q[:, :, 9] = level / 16 * 128 ** 0.5
    ck, cv, up = (x[:, 0] for x in c.cached(0))
    s = ck @ q[0, 0].astype(np.float64) * 128 ** -0.5
    w = np.exp(s - s.max())
    w /= w.sum()
    # tree_reference's bound over the cached tokens alone, with 2^-14 for the least that a key can lose
    lost = up * 2.0 ** -13 + 2.0 ** -14 + (2 * np.abs(ck) + up) * 2.0 ** -20
    d = (lost @ np.abs(q[0, 0].astype(np.float64))).max() * 128 ** -0.5
    ref = w @ cv
    bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2 * d + 2.0 ** -19) * (w @ np.abs(cv))
    k, v = np.zeros((1, 1, 128), np.float16), rng.standard_normal((1, 1, 128)).astype(np.float16)
    k[0, 0, 5] = -np.inf if q[0, 0, 5] > 0 else np.inf
    out = run_tree(c, q, k, v, np.array([0, 1], np.int32), np.array([-1], np.int32), 1)[0, 0]
    assert (np.abs(out - ref) <= bound).all()
    assert c.S.s4kv_get_error(c.gpu) == 0


def test_results_in_the_queries_place():
    """The output may be the queries' own tensor, whole units and cut ones."""
    rng = np.random.default_rng(39)
    nodes = [9, 40, 3]
    c = SpecCache([3000, 100, 7], 2, seed=40, key_scale=np.ones((2, 128)))
    cu, parents, q, k, v = make_tree(rng, nodes, 2, 4, 3)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    d = [c.dev(x) for x in (q, k, v, cu, parents)]
    c.S.s4kv_tree_attention(c.gpu, *d, c.lens_dev, c.bt_dev, d[0], 40, c.S.tree_workspace(8, 2, 3, 40))
    assert (np.abs(d[0].float().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_remainders_of_the_keys(bits):
    """What fp16 loses of code * scale comes back through the second product: measured alone, where the logits without
    it would be off by 1 of this measure, and by 2 with it subtracted."""
    c, q, exact, parts, _ = remainder_case(bits, True)
    k, v = np.zeros((ROWS, 1, 128), np.float16), np.zeros((ROWS, 1, 128), np.float16)
    v[:, 0, 127] = 1
    level = (2 ** bits - 1) / 2 ** bits
    out = run_tree(c, q, k, v, np.array([0, ROWS], np.int32), np.full(ROWS, -1, np.int32), ROWS, sm_scale=SM_SCALE)[:, 0]
    logits = np.log(out[:, :TOKENS] / level) - np.log(out[:, 127:])
    assert remainder_error(logits, exact, parts) <= REMAINDER_BOUND


def test_many_rows_over_a_long_context():
    """512 query rows a kv head over 6011 tokens, 8 blocks of rows, and 448 over 2100."""
    rng = np.random.default_rng(41)
    nodes = [64, 56]
    c = SpecCache([6011, 2100], 2, seed=42, key_scale=np.ones((2, 128)))
    cu, parents, q, k, v = make_tree(rng, nodes, 2, 8, 4)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    out = run_tree(c, q, k, v, cu, parents, 64)
    assert (np.abs(out - ref) <= bound).all()
    assert c.S.s4kv_get_error(c.gpu) == 0
