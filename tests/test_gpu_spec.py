"""The speculative-decoding calls on the GPU (s4kv_tree_attention,
s4kv_verify_tree, s4kv_append_path) against plain references in 64 bits."""
import ctypes

import numpy as np
import pytest

from int4_kivi_quantized_s4kv_b200 import workloads as W
from spec_helpers import SpecCache, random_parents, tree_reference, verify_reference

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


def make_tree(rng, nodes, heads, group, key_scale, newest):
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    n = int(cu[-1])
    parents = np.concatenate([random_parents(rng, int(x), newest) for x in nodes]).astype(np.int32)
    q = rng.standard_normal((n, heads * group, 128)).astype(np.float16)
    k = (rng.standard_normal((n, heads, 128)) * key_scale).astype(np.float16)
    v = rng.standard_normal((n, heads, 128)).astype(np.float16)
    return cu, parents, q, k, v


def run_tree(c, q, k, v, cu, parents, max_nodes=64, ws=None, sm_scale=None, out=None, lens=None, bt=None):
    import torch
    S = c.S
    qd = c.dev(q)
    out = torch.full_like(qd, float("nan")) if out is None else out
    if ws is None:
        ws = S.tree_workspace(q.shape[1], c.H, len(cu) - 1, max_nodes)
    S.s4kv_tree_attention(c.gpu, qd, c.dev(k), c.dev(v), c.dev(cu), c.dev(parents), c.lens_dev if lens is None else lens,
                          c.bt_dev if bt is None else bt, out, max_nodes, ws, sm_scale)
    torch.cuda.synchronize()
    return out


def close(got, ref, bound):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    err = np.nan_to_num(np.abs(got - ref))
    assert (err <= np.nan_to_num(bound)).all(), (err.max(), float((err / np.nan_to_num(bound, nan=1.0)).max()))


# lengths, nodes a sequence, kv heads, group, code width, newest nodes that may be parents (0: all are roots)
TREES = {
    "one-token": ([1], [1], 1, 1, 4, 1),
    "empty-cache": ([0, 0], [1, 64], 1, 2, 4, 3),
    "page-edges": ([0, 1, 15, 16, 17, 127, 128, 129, 143, 144], [3, 1, 5, 2, 7, 4, 9, 1, 6, 3], 2, 3, 4, 2),
    "tile-edges": ([1023, 1024, 1025, 112, 113, 240], [8, 8, 8, 4, 2, 11], 1, 8, 4, 4),
    "no-nodes": ([40, 100, 0, 33], [0, 4, 0, 0], 2, 4, 4, 2),
    "roots-only": ([50, 200], [6, 17], 1, 4, 4, 0),
    "chain": ([300, 20], [16, 16], 2, 4, 4, 1),
    "wide": ([200, 77], [64, 63], 1, 8, 4, 5),
    "group-7": ([90, 650, 31], [10, 9, 37], 4, 7, 4, 3),
    "group-5": ([333], [13], 3, 5, 4, 3),
    "rows-64": ([400], [64], 2, 1, 4, 3),
    "rows-65": ([400, 7], [13, 13], 2, 5, 4, 3),
    "split-long": ([9000], [16], 1, 4, 4, 3),
    "split-mixed": ([6001, 3, 4200, 0, 129], [9, 64, 33, 2, 1], 2, 6, 4, 3),
    "many": ([(37 * i) % 250 for i in range(150)], [1 + i % 5 for i in range(150)], 2, 4, 4, 2),
    "int8": ([0, 5, 130, 1999, 64], [3, 2, 20, 16, 1], 2, 4, 8, 3),
    "int8-wide": ([517], [64], 1, 8, 8, 3),
    "int2": ([0, 5, 130, 1999, 64], [3, 2, 20, 16, 1], 2, 4, 2, 3),
}


@pytest.mark.parametrize("name", TREES)
def test_tree_attention(name):
    lens, nodes, heads, group, bits, newest = TREES[name]
    rng = np.random.default_rng(len(name) + sum(lens))
    c = SpecCache(lens, heads, bits, seed=sum(nodes))
    cu, parents, q, k, v = make_tree(rng, nodes, heads, group, c.key_scale, newest)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    max_nodes = max(nodes)
    out = run_tree(c, q, k, v, cu, parents, max_nodes)
    close(out, ref, bound)
    assert c.S.s4kv_get_error(c.gpu) == 0
    # a larger bound than needed, and the same workspace twice: the same bits
    ws = c.S.tree_workspace(q.shape[1], heads, len(nodes), 64)
    for bound_n in (64, max_nodes):
        close(run_tree(c, q, k, v, cu, parents, bound_n, ws), ref, bound)
    again = run_tree(c, q, k, v, cu, parents, max_nodes, ws)
    assert np.array_equal(again.cpu().numpy().view(np.uint16), out.cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("scale,what", [(0.0, "equal keys"), (1e-3, "small keys"), (100.0, "large keys")])
def test_tree_attention_key_ranges(scale, what):
    rng = np.random.default_rng(5)
    c = SpecCache([200, 31], 2, 4, seed=9, key_scale=np.full((2, 128), scale))
    cu, parents, q, k, v = make_tree(rng, [7, 5], 2, 4, c.key_scale, 2)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    close(run_tree(c, q, k, v, cu, parents), ref, bound)


@pytest.mark.parametrize("sm_scale", [1e-3, 1.0, 4.0])
def test_tree_attention_logit_scales(sm_scale):
    """Flat and very sharp softmaxes; the reference moves while the cache is read (the largest key comes late)."""
    rng = np.random.default_rng(6)
    c = SpecCache([1500, 700], 1, 4, seed=10)
    cu, parents, q, k, v = make_tree(rng, [9, 4], 1, 4, c.key_scale, 2)
    ref, bound = tree_reference(c, q, k, v, cu, parents, sm_scale)
    close(run_tree(c, q, k, v, cu, parents, sm_scale=sm_scale), ref, bound)


def test_tree_attention_logits_far_apart():
    """One token's logit hundreds above the rest, in the cache's last pages or in the tree; weights underflow."""
    rng = np.random.default_rng(7)
    c = SpecCache([900, 900], 1, 4, seed=11)
    cu, parents, q, k, v = make_tree(rng, [6, 6], 1, 4, c.key_scale, 2)
    q[:] = rng.standard_normal((1, 1, 128)).astype(np.float16) * np.float16(4)
    k[3] = q[3, 0] * np.float16(8)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    close(run_tree(c, q, k, v, cu, parents), ref, bound)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("length", [0, 5, 300])
def test_tree_attention_values_that_are_not_finite(bad, length):
    """A drafted token with an infinity or NaN in its key or value reaches the rows that see it, and no others."""
    rng = np.random.default_rng(21)
    nodes = [40, 9]
    c = SpecCache([length, 70], 2, 4, seed=22)
    cu, parents, q, k, v = make_tree(rng, nodes, 2, 4, c.key_scale, 3)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    who = {}  # node -> the rows that see it, as node numbers
    for b in range(2):
        for i in range(nodes[b]):
            a = i
            while a >= 0:
                who.setdefault(cu[b] + a, []).append(cu[b] + i)
                a = parents[cu[b] + a]
    x = int(cu[0]) + 33
    seen = np.zeros(len(q), bool)
    seen[who[x]] = True
    assert 0 < seen.sum() < 40
    wrong = v.copy()
    wrong[x, 1, 77] = bad
    out = run_tree(c, q, k, wrong, cu, parents).float().cpu().numpy().astype(np.float64)
    hit = np.zeros(out.shape, bool)
    hit[seen, 4:, 77] = True  # query heads 4 - 7 read kv head 1
    assert np.array_equal(out[hit], np.full(hit.sum(), bad), equal_nan=True)
    assert (np.abs(out - ref)[~hit] <= bound[~hit]).all()
    wrong = k.copy()
    wrong[x, 0, 5] = bad
    out = run_tree(c, q, wrong, v, cu, parents).float().cpu().numpy().astype(np.float64)
    hit = np.zeros(out.shape, bool)
    hit[seen, :4] = True
    assert (np.abs(out - ref)[~hit] <= bound[~hit]).all()


def test_tree_attention_leaves_other_rows():
    import torch
    rng = np.random.default_rng(8)
    c = SpecCache([64, 10, 90], 2, 4, seed=12)
    cu, parents, q, k, v = make_tree(rng, [4, 3, 5], 2, 4, c.key_scale, 2)
    q = np.concatenate([q, q[:3]])
    k, v = np.concatenate([k, k[:3]]), np.concatenate([v, v[:3]])
    parents = np.concatenate([parents, np.array([-1, 0, 1], np.int32)])
    out = run_tree(c, q, k, v, cu, parents)
    assert torch.isnan(out[12:]).all() and not torch.isnan(out[:12]).any()


def test_tree_attention_flags_and_skips():
    """Bad lengths, too many nodes and bad parents set their bits; the other sequences are right."""
    import torch
    rng = np.random.default_rng(13)
    c = SpecCache([64, 10, 90, 33], 2, 4, seed=14)
    S = c.S
    cu, parents, q, k, v = make_tree(rng, [4, 3, 5, 2], 2, 4, c.key_scale, 2)
    ref, bound = tree_reference(c, q, k, v, cu, parents)

    def others(out, skipped):
        lo, hi = int(cu[skipped]), int(cu[skipped + 1])
        assert torch.isnan(out[lo:hi]).all()
        r = ref.copy()
        r[lo:hi] = np.nan
        close(out, r, bound)

    for bad in (-1, 16 * c.max_pages + 1):
        lens = c.lens.copy()
        lens[1] = bad
        others(run_tree(c, q, k, v, cu, parents, lens=c.dev(lens)), 1)
        assert S.s4kv_get_error(c.gpu) == S.EFLAG_SEQ_LEN
    others(run_tree(c, q, k, v, cu, parents, max_nodes=4), 2)
    assert S.s4kv_get_error(c.gpu) == S.EFLAG_TREE
    # more nodes claimed than there are: the last sequence is skipped
    over = cu.copy()
    over[-1] += 1
    others(run_tree(c, q, k, v, over, parents), 3)
    assert S.s4kv_get_error(c.gpu) == S.EFLAG_TREE
    # a parent that does not come before its node counts as none
    for bad in (4, 9, -2):
        wrong, meant = parents.copy(), parents.copy()
        wrong[cu[2] + 4], meant[cu[2] + 4] = bad, -1
        out = run_tree(c, q, k, v, cu, wrong)
        assert S.s4kv_get_error(c.gpu) == S.EFLAG_TREE
        close(out, *tree_reference(c, q, k, v, cu, meant))
    # a page outside the pool: flagged, page 0 in its place
    bt = c.bt.copy()
    bt[2, 1] = 1 << 30
    out = run_tree(c, q, k, v, cu, parents, bt=c.dev(bt))
    assert S.s4kv_get_error(c.gpu) == S.EFLAG_PAGE_RANGE
    assert not torch.isnan(out).any()


def test_tree_attention_equals_decode_attention_on_the_grown_cache():
    """A single node a sequence is a decode step: s4kv_append_decode of the same token gives the same attention
    (but for a page that the token completes, which is then quantized)."""
    import torch
    rng = np.random.default_rng(15)
    lens = [5, 64, 100, 1000]
    c = SpecCache(lens, 2, 4, seed=16, room=1)
    cu, parents, q, k, v = make_tree(rng, [1] * 4, 2, 4, c.key_scale, 1)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    close(run_tree(c, q, k, v, cu, parents), ref, bound)
    out = torch.empty_like(c.dev(q))
    c.S.s4kv_append_decode(c.gpu, c.dev(k), c.dev(v), c.dev(q), c.dev(np.array(lens, np.int32) + 1), c.bt_dev, out,
                           c.S.decode_workspace(4, 2))
    close(out, ref, bound)


def test_tree_attention_far_pages():
    """Pages behind the 2^31st byte of the pool."""
    import torch
    rng = np.random.default_rng(17)
    c = SpecCache([500, 80], 8, 4, seed=18)
    S = c.S
    cu, parents, q, k, v = make_tree(rng, [5, 3], 8, 2, c.key_scale, 2)
    near = run_tree(c, q, k, v, cu, parents)
    pages = (1 << 31) // (8 * 2816) + 200
    big = S.S4KVCache(pages, 8, 2)
    used = torch.from_numpy(c.bt.reshape(-1)).cuda()
    far = torch.arange(pages - used.numel(), pages, dtype=torch.int32, device="cuda")
    rec = torch.empty(used.numel() * S.s4kv_page_record_bytes(big), dtype=torch.uint8, device="cuda")
    S.s4kv_gather_pages(c.gpu, used, rec)
    S.s4kv_scatter_pages(big, far, rec)
    big.res_k.copy_(c.gpu.res_k)
    big.res_v.copy_(c.gpu.res_v)
    c.gpu = big
    out = run_tree(c, q, k, v, cu, parents, bt=far.view(2, -1).contiguous())
    assert torch.equal(out, near)


# how the work is dealt out: lengths, nodes, kv heads, group, code width, newest nodes that may be parents
DEALS = {
    # fewer units than CTAs, several sequences a lane, some without nodes
    "parts-of-many": ([(613 * i) % 3500 for i in range(45)], [(0, 1, 3, 9)[i % 4] for i in range(45)], 1, 4, 4, 2),
    # more than half as many units as CTAs: some are cut in two, some are not
    "parts-uneven": ([2100 - 30 * (i % 20) for i in range(50)], [2 + i % 3 for i in range(50)], 2, 2, 4, 2),
    # nearly as many units as CTAs, one of them long: it would be one CTA's alone
    "ranges-one-long": ([(29 * i) % 128 for i in range(70)] + [6300] + [(17 * i) % 128 for i in range(75)],
                        [1 + i % 4 for i in range(146)], 1, 4, 4, 2),
    "ranges-half": ([5500] * 40, [1] * 40, 2, 1, 2, 1),
    # a part a tile; the shortest units that are cut, and the longest that are not
    "parts-of-one-tile": ([900, 641, 640, 639], [8, 3, 5, 2], 4, 4, 4, 2),
    # one unit in as many parts as there may be
    "one-unit": ([40000], [5], 1, 4, 4, 2),
    "int8-two-units": ([20011], [7], 2, 7, 8, 2),
}


@pytest.mark.parametrize("name", DEALS)
def test_tree_attention_deals(name):
    lens, nodes, heads, group, bits, newest = DEALS[name]
    rng = np.random.default_rng(len(name) + sum(lens))
    c = SpecCache(lens, heads, bits, seed=sum(nodes))
    cu, parents, q, k, v = make_tree(rng, nodes, heads, group, c.key_scale, newest)
    ref, bound = tree_reference(c, q, k, v, cu, parents)
    ws = c.S.tree_workspace(q.shape[1], heads, len(nodes), max(nodes))
    out = run_tree(c, q, k, v, cu, parents, max(nodes), ws)
    close(out, ref, bound)
    again = run_tree(c, q, k, v, cu, parents, max(nodes), ws)
    assert np.array_equal(again.cpu().numpy().view(np.uint16), out.cpu().numpy().view(np.uint16))
    assert c.S.s4kv_get_error(c.gpu) == 0


def test_tree_attention_on_two_streams_at_once():
    import torch
    rng = np.random.default_rng(29)
    both = []
    for lens, nodes in (([5000, 33], [6, 9]), ([800] * 5, [4] * 5)):
        c = SpecCache(lens, 2, 4, seed=len(lens))
        cu, parents, q, k, v = make_tree(rng, nodes, 2, 4, c.key_scale, 2)
        d = [c.dev(x) for x in (q, k, v, cu, parents)]
        both.append((c, d, torch.zeros_like(d[0]), c.S.tree_workspace(8, 2, len(lens), max(nodes)), max(nodes),
                     tree_reference(c, q, k, v, cu, parents)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(20):
        for s, (c, d, out, ws, most, _) in zip(streams, both):
            with torch.cuda.stream(s):
                c.S.s4kv_tree_attention(c.gpu, *d, c.lens_dev, c.bt_dev, out, most, ws)
    torch.cuda.synchronize()
    for c, _, out, _, _, ref in both:
        close(out, *ref)
        assert c.S.s4kv_get_error(c.gpu) == 0


def test_tree_attention_captured_and_on_another_stream():
    import torch
    rng = np.random.default_rng(19)
    c = SpecCache([700, 45, 260], 2, 4, seed=20)
    S = c.S
    cu, parents, q, k, v = make_tree(rng, [6, 12, 3], 2, 4, c.key_scale, 2)
    d = [c.dev(x) for x in (q, k, v, cu, parents)]
    out = torch.zeros_like(d[0])
    ws = S.tree_workspace(8, 2, 3, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: S.s4kv_tree_attention(c.gpu, *d, c.lens_dev, c.bt_dev, out, 12, ws)  # noqa: E731
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    first = out.clone()
    close(first, *tree_reference(c, q, k, v, cu, parents))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    # new inputs in the captured buffers: another tree, other queries, a shorter context
    cu2 = np.array([0, 2, 2, 14], np.int32)
    parents2 = np.concatenate([random_parents(rng, 2, 1), random_parents(rng, 12, 3),
                               np.full(len(parents) - 14, -1)]).astype(np.int32)
    q2 = rng.standard_normal(q.shape).astype(np.float16)
    for t, a in zip((d[0], d[3], d[4]), (q2, cu2, parents2)):
        t.copy_(c.dev(a))
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
    torch.cuda.synchronize()
    close(out, *tree_reference(c, q2, k, v, cu2, parents2))
    assert S.s4kv_get_error(c.gpu) == 0


# ------------------------------------------------------------ verification --

def make_verify(rng, nodes, vocab, branch, draft, dtype, sharp=2.0, near=0.5):
    import torch
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    n = int(cu[-1])
    parents = np.concatenate([random_parents(rng, int(x), branch) for x in nodes] or [[]]).astype(np.int32)
    z = torch.from_numpy(rng.standard_normal((n, vocab)) * sharp)
    q = torch.softmax(z, -1)
    p = torch.softmax(z + torch.from_numpy(rng.standard_normal((n, vocab)) * near), -1)
    p, q = p.to(dtype), q.to(dtype)
    qn = q.double().numpy()
    tok = np.zeros(n, np.int32)
    for b, x in enumerate(nodes):
        for i in range(x):
            row = qn[cu[b] + max(0, parents[cu[b] + i])]
            if draft:
                tok[cu[b] + i] = rng.choice(vocab, p=row / row.sum())
            else:
                tok[cu[b] + i] = np.argsort(-row)[min(vocab - 1, i % branch)]
    u = rng.random(n, dtype=np.float32)
    return tok, parents, cu, p, q if draft else None, u


def run_verify(tok, parents, cu, p, q, u, max_nodes, err=None):
    import torch
    import int4_kivi_quantized_s4kv_b200 as S
    dev = lambda a: (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()  # noqa: E731
    B = len(cu) - 1
    path = torch.full((B, max_nodes), 77, dtype=torch.int32, device="cuda")
    length = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    nxt = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    S.s4kv_verify_tree(dev(tok), dev(parents), dev(cu), dev(p), None if q is None else dev(q), dev(u), path, length, nxt, err)
    torch.cuda.synchronize()
    return path.cpu().numpy(), length.cpu().numpy(), nxt.cpu().numpy()


def same(got, ref):
    for g, r in zip(got, ref):
        assert np.array_equal(g, r), (g, r)


def as_np(t):
    return None if t is None else t.double().numpy()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("vocab,branch,nodes", [
    (1, 1, [3, 1]), (2, 2, [5, 1, 9]), (31, 3, [4, 0, 17, 64]), (1000, 1, [6] * 9), (4097, 4, [33, 2, 8, 1]),
    (32003, 2, [7, 12, 1, 5])])
def test_verify(vocab, branch, nodes, draft, dtype):
    import torch
    rng = np.random.default_rng(vocab + branch)
    for near in (0.1, 1.5):
        tok, parents, cu, p, q, u = make_verify(rng, nodes, vocab, branch, draft, getattr(torch, dtype), near=near)
        ref = verify_reference(tok, parents, cu, as_np(p), as_np(q), u, max(nodes))
        same(run_verify(tok, parents, cu, p, q, u, max(nodes)), ref)


def test_verify_large_vocabulary_and_batch():
    import torch
    rng = np.random.default_rng(3)
    tok, parents, cu, p, q, u = make_verify(rng, [3] * 20, 128256, 1, True, torch.float32)
    same(run_verify(tok, parents, cu, p, q, u, 3), verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 3))


@pytest.mark.parametrize("batch,vocab", [(149, 3000), (700, 2600), (2500, 70)])
def test_verify_many_sequences(batch, vocab):
    """Batches that take fewer CTAs a sequence."""
    import torch
    rng = np.random.default_rng(batch)
    tok, parents, cu, p, q, u = make_verify(rng, [1 + b % 3 for b in range(batch)], vocab, 2, True, torch.float32)
    same(run_verify(tok, parents, cu, p, q, u, 3), verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 3))


def test_verify_vocabulary_of_millions():
    """Rows whose chunks have more than one block; the draws fall at the ends and between."""
    import torch
    rng = np.random.default_rng(8)
    V = 5_000_011
    p = torch.rand(6, V, generator=torch.Generator().manual_seed(1))
    p /= p.sum(-1, keepdim=True)
    tok, parents, cu = np.array([0, 9, 0, 9, 0, 9], np.int32), np.array([-1, 0] * 3, np.int32), np.array([0, 2, 4, 6], np.int32)
    for u0 in (0.0, 0.5, 0.9999):
        u = np.array([u0, 0.9] * 3, np.float32) * rng.random(6, dtype=np.float32)
        same(run_verify(tok, parents, cu, p, None, u, 2), verify_reference(tok, parents, cu, as_np(p), None, u, 2))


@pytest.mark.parametrize("u0", [0.0, float(np.float32(1) - np.float32(2) ** -24)])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_ends_of_the_random_numbers(u0, draft):
    """The first and the last entry with mass are drawn at the ends; entries without mass never are."""
    import torch
    rng = np.random.default_rng(4)
    tok, parents, cu, p, q, u = make_verify(rng, [1, 4, 6], 5000, 2, draft, torch.float32)
    p[:, :17] = 0
    p[:, -23:] = 0
    u[:] = u0
    ref = verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 6)
    same(run_verify(tok, parents, cu, p, q, u, 6), ref)
    assert (ref[2] >= 17).all() and (ref[2] < 5000 - 23).all()


def test_verify_same_rows_and_nothing_left():
    """Target and draft alike: everything is accepted; a rejection that leaves nothing falls back on the target's row.
    Without draft rows: the same token twice among the children, and a row of which the children take everything."""
    import torch
    rng = np.random.default_rng(5)
    tok, parents, cu, p, q, u = make_verify(rng, [5, 5], 300, 1, True, torch.float32)
    got = run_verify(tok, parents, cu, q, q, u, 5)
    assert (got[1] == 5).all()
    same(got, verify_reference(tok, parents, cu, as_np(q), as_np(q), u, 5))
    u[:] = 1.0  # outside [0, 1): every test fails, R = max(p - q, 0) = 0
    same(run_verify(tok, parents, cu, q, q, u, 5), verify_reference(tok, parents, cu, as_np(q), as_np(q), u, 5))
    one = torch.zeros(4, 300)
    one[:, 7] = 1
    tok, parents, cu = np.array([1, 7, 7, 7], np.int32), np.array([-1, 0, 0, 0], np.int32), np.array([0, 4], np.int32)
    u = np.array([0.5, 1.0, 1.0, 0.0], np.float32)
    same(run_verify(tok, parents, cu, one, None, u, 4), verify_reference(tok, parents, cu, as_np(one), None, u, 4))


def test_verify_odd_values_and_flags():
    import torch
    import int4_kivi_quantized_s4kv_b200 as S
    rng = np.random.default_rng(6)
    tok, parents, cu, p, q, u = make_verify(rng, [4, 4, 4], 700, 2, True, torch.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # negative entries and NaN count as nothing
    p[:, 5], p[:, 9], q[:, 6] = -1.0, float("nan"), float("nan")
    same(run_verify(tok, parents, cu, p, q, u, 4, err), verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 4))
    assert int(err) == 0
    # a token outside the vocabulary is passed over
    tok[1] = 700
    tok[6] = -1
    same(run_verify(tok, parents, cu, p, q, u, 4, err), verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 4))
    assert int(err) == S.EFLAG_TREE
    err.zero_()
    # rows without mass, and an infinite one
    p[:4] = 0
    p[4:8, 3] = float("inf")
    got = run_verify(tok, parents, cu, p, q, u, 4, err)
    assert int(err) & S.EFLAG_PROBS and got[2][0] == -1 and got[2][1] == -1 and got[2][2] >= 0
    err.zero_()
    # more nodes than the bound, and cu_nodes that run over the end
    got = run_verify(tok, parents, np.array([0, 4, 9, 12], np.int32), p, q, u, 4, err)
    assert int(err) & S.EFLAG_TREE and got[1][1] == 0 and got[2][1] == -1 and (got[0][1] == -1).all()
    err.zero_()
    got = run_verify(tok, parents, np.array([0, 4, 8, 13], np.int32), p, q, u, 5, err)
    assert int(err) & S.EFLAG_TREE and got[1][2] == 0 and (got[0][2] == -1).all()


def test_verify_strided_rows_and_capture():
    import torch
    import int4_kivi_quantized_s4kv_b200 as S
    rng = np.random.default_rng(7)
    tok, parents, cu, p, q, u = make_verify(rng, [5, 2, 8], 1001, 2, True, torch.bfloat16)
    wide = torch.full((15, 1040), 0.5, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:1004] = p.cuda()
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    path = torch.empty(3, 8, dtype=torch.int32, device="cuda")
    length, nxt = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    ud = dev(u)
    args = (dev(tok), dev(parents), dev(cu), wide[:, 3:1004], q.cuda(), ud, path, length, nxt)
    S.s4kv_verify_tree(*args)
    torch.cuda.synchronize()
    same((path.cpu().numpy(), length.cpu().numpy(), nxt.cpu().numpy()),
         verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 8))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.s4kv_verify_tree(*args)
    for _ in range(3):
        u = rng.random(len(u), dtype=np.float32)
        ud.copy_(dev(u))
        g.replay()
        torch.cuda.synchronize()
        same((path.cpu().numpy(), length.cpu().numpy(), nxt.cpu().numpy()),
             verify_reference(tok, parents, cu, as_np(p), as_np(q), u, 8))


# ------------------------------------------------------------------ commit --

def commit_both(c, nodes, paths, rng, max_nodes=None):
    """Append the paths on the GPU, and their rows in the oracle with s4kv_append's restatement."""
    import torch
    S, B = c.S, len(c.lens)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    n, most = int(cu[-1]), max_nodes or max(1, max(nodes))
    k = (rng.standard_normal((n, c.H, 128)) * c.key_scale).astype(np.float16)
    v = rng.standard_normal((n, c.H, 128)).astype(np.float16)
    path = np.full((B, most), -1, np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    ln = np.array([len(x) for x in paths], np.int32)
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    S.s4kv_append_path(c.gpu, c.dev(k), c.dev(v), c.dev(cu), c.dev(path), c.dev(ln), c.lens_dev, c.bt_dev, new)
    torch.cuda.synchronize()
    rows = np.concatenate([cu[b] + np.array(x, np.int64) for b, x in enumerate(paths)]).astype(np.int64)
    after = c.lens + ln
    if len(rows):
        sm = W.slot_mapping(c.bt, [np.arange(int(c.lens[b]), int(after[b])) for b in range(B)])
        assert c.oc.append(k[rows], v[rows], sm, np.concatenate([[0], np.cumsum(ln)]), after, c.bt) == 0
    return after, new.cpu().numpy()


def assert_caches_alike(c, lens):
    assert np.array_equal(c.gpu.pool.cpu().numpy(), c.oc.pool)
    rk, rv = (t.cpu().numpy().view(np.uint16) for t in (c.gpu.res_k, c.gpu.res_v))
    for b, L in enumerate(lens):
        r = int(L) % 16
        assert np.array_equal(rk[b, :, :r], c.oc.res_k[b, :, :r]) and np.array_equal(rv[b, :, :r], c.oc.res_v[b, :, :r])


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_append_path(bits):
    rng = np.random.default_rng(bits)
    lens = [0, 0, 15, 16, 31, 10, 1, 130, 47, 33]
    nodes = [1, 64, 3, 20, 2, 25, 0, 9, 64, 4]
    paths = [[0], list(range(64)), [0, 2], [0], [0, 1], list(range(0, 25, 2)), [], [], sorted(rng.permutation(64)[:50]), [0, 1, 3]]
    c = SpecCache(lens, 3, bits, seed=bits, room=5)
    after, new = commit_both(c, nodes, paths, rng)
    assert np.array_equal(new, after) and c.S.s4kv_get_error(c.gpu) == 0
    assert_caches_alike(c, after)


def test_append_path_refuses_a_sequence_whole():
    import torch
    rng = np.random.default_rng(2)
    c = SpecCache([20, 60, 30, 5], 2, 4, seed=3, room=0)
    S = c.S
    before = [t.clone() for t in (c.gpu.pool, c.gpu.res_k, c.gpu.res_v)]
    k = torch.randn(16, 2, 128, device="cuda").half()
    cu = c.dev(np.array([0, 4, 8, 12, 16], np.int32))

    def call(path, ln, cu=cu):
        new = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        S.s4kv_append_path(c.gpu, k, k, cu, c.dev(np.array(path, np.int32)), c.dev(np.array(ln, np.int32)), c.lens_dev,
                           c.bt_dev, new)
        torch.cuda.synchronize()
        assert np.array_equal(new.cpu().numpy(), c.lens)
        for t, x in zip(before, (c.gpu.pool, c.gpu.res_k, c.gpu.res_v)):
            assert torch.equal(t, x)
        return S.s4kv_get_error(c.gpu)

    none = [[-1] * 5] * 4
    assert call(none, [0] * 4) == 0
    assert call([[0, 1, -1, 3, -1], *none[1:]], [4, 0, 0, 0]) == S.EFLAG_TREE  # a hole in the path
    assert call([[0, 1, 4, -1, -1], *none[1:]], [3, 0, 0, 0]) == S.EFLAG_TREE  # a node of the next sequence
    assert call(none, [6, -1, 0, 0]) == S.EFLAG_TREE                           # lengths outside the bound
    assert call([none[0], [0, 1, 2, 3, 0], *none[2:]], [0, 5, 0, 0]) == S.EFLAG_SEQ_LEN  # 65 tokens in 4 pages
    assert call([[0] + [-1] * 4] * 4, [0, 0, 0, 1], c.dev(np.array([0, 4, 8, 12, 17], np.int32))) == S.EFLAG_TREE


def test_append_path_flags_a_page_outside_the_pool():
    import torch
    c = SpecCache([15, 15], 1, 4, seed=4, room=1)
    S = c.S
    bt = c.bt.copy()
    bt[0, 0] = -1
    k = torch.randn(2, 1, 128, device="cuda").half()
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    pool = c.gpu.pool.clone()
    S.s4kv_append_path(c.gpu, k, k, c.dev(np.array([0, 1, 2], np.int32)), c.dev(np.zeros((2, 1), np.int32)),
                       c.dev(np.ones(2, np.int32)), c.lens_dev, c.dev(bt), new)
    torch.cuda.synchronize()
    assert S.s4kv_get_error(c.gpu) == S.EFLAG_PAGE_RANGE
    changed = (c.gpu.pool != pool).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(bt[1, 0])]


# ---------------------------------------------------------------- together --

@pytest.mark.parametrize("bits", [4, 8])
def test_three_steps_of_speculative_decoding(bits):
    """Attention of the drafted trees, verification and commit, three times, without a look at the host: every
    step's answers against the references on the oracle's cache."""
    import torch
    rng = np.random.default_rng(40 + bits)
    heads, group, V = 2, 4, 500
    c = SpecCache([30, 0, 250, 15], heads, bits, seed=30, room=4)
    S, B, most = c.S, 4, 9
    ws = S.tree_workspace(heads * group, heads, B, most)
    lens_dev, new_dev = c.lens_dev.clone(), torch.empty_like(c.lens_dev)
    path = torch.empty(B, most, dtype=torch.int32, device="cuda")
    ln, nxt = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    toks = [(c.k[b], c.v[b]) for b in range(B)]
    for step in range(3):
        nodes = [int(x) for x in rng.integers(1, most + 1, B)]
        cu, parents, q, k, v = make_tree(rng, nodes, heads, group, c.key_scale, 3)
        tok, _, _, p, qd, u = make_verify(rng, nodes, V, 3, True, torch.float32, near=0.2)
        d = [c.dev(x) for x in (q, k, v, cu, parents)]
        out = torch.full_like(d[0], float("nan"))
        S.s4kv_tree_attention(c.gpu, *d, lens_dev, c.bt_dev, out, most, ws)
        S.s4kv_verify_tree(c.dev(tok), d[4], d[3], p.cuda(), qd.cuda(), c.dev(u), path, ln, nxt, c.gpu.err_flag)
        S.s4kv_append_path(c.gpu, d[1], d[2], d[3], path, ln, lens_dev, c.bt_dev, new_dev)
        lens_dev, new_dev = new_dev, lens_dev
        torch.cuda.synchronize()
        assert S.s4kv_get_error(c.gpu) == 0
        close(out, *tree_reference(c, q, k, v, cu, parents))
        ref = verify_reference(tok, parents, cu, as_np(p), as_np(qd), u, most)
        same((path.cpu().numpy(), ln.cpu().numpy(), nxt.cpu().numpy()), ref)
        rows = [cu[b] + ref[0][b, :ref[1][b]] for b in range(B)]
        after = (c.lens + ref[1]).astype(np.int32)
        sm = W.slot_mapping(c.bt, [np.arange(int(c.lens[b]), int(after[b])) for b in range(B)])
        cat = np.concatenate(rows)
        assert c.oc.append(k[cat], v[cat], sm, np.concatenate([[0], np.cumsum(ref[1])]), after, c.bt) == 0
        toks = [(np.concatenate([toks[b][0], k[rows[b]]]), np.concatenate([toks[b][1], v[rows[b]]])) for b in range(B)]
        c.k, c.v, c.lens = [t[0] for t in toks], [t[1] for t in toks], after
        assert np.array_equal(lens_dev.cpu().numpy(), after)
        assert_caches_alike(c, after)


def test_calls_run_on_their_tensors_device_and_refuse_two():
    """The wrappers take the stream of the tensors' device and refuse host tensors."""
    import torch
    c = SpecCache([20], 1, 4, seed=5)
    S = c.S
    q, k = torch.zeros(1, 4, 128).half(), torch.zeros(1, 1, 128).half().cuda()
    cu, par = c.dev(np.array([0, 1], np.int32)), c.dev(np.array([-1], np.int32))
    ws = S.tree_workspace(4, 1, 1, 1)
    with pytest.raises(ValueError):
        S.s4kv_tree_attention(c.gpu, q, k, k, cu, par, c.lens_dev, c.bt_dev, torch.empty_like(q), 1, ws)
    q = q.cuda()
    with pytest.raises(ValueError):
        S.s4kv_tree_attention(c.gpu, q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu, par, c.lens_dev, c.bt_dev,
                              torch.empty_like(q), 1, ws)
    with pytest.raises(S.S4KVError):
        S.s4kv_tree_attention(c.gpu, q, k, k, cu, par, c.lens_dev, c.bt_dev, torch.empty_like(q), 1, ws[:-16])
    assert isinstance(ctypes.sizeof(S.s4kv_cache_t), int)
