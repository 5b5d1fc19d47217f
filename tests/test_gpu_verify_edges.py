"""Verification of drafted trees at the batch sizes where the number of CTAs a sequence changes."""
import numpy as np
import pytest

from spec_helpers import verify_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int4_kivi_quantized_s4kv_b200 import build
    build.build()


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("batch", [71, 72, 142, 143, 296, 297, 593])
def test_batches_on_both_sides_of_the_switches(batch, draft):
    """8, 4, 2 or 1 CTAs a sequence (148 SMs of 4 CTAs), each with a chunk for every warp."""
    import torch
    import int4_kivi_quantized_s4kv_b200 as S
    rng = np.random.default_rng(batch)
    V, n = 9001, 3 * batch
    cu = np.arange(0, n + 1, 3, dtype=np.int32)
    parents = np.tile(np.array([-1, 0, 0], np.int32), batch)
    z = rng.standard_normal((n, V), dtype=np.float32)
    q = torch.softmax(torch.from_numpy(z), -1)
    p = torch.softmax(torch.from_numpy(z + 0.7 * rng.standard_normal((n, V), dtype=np.float32)), -1)
    u = rng.random(n, dtype=np.float32)
    # children drawn from their parent's draft row by inverting its sum; the likeliest ones without draft rows
    c = np.cumsum(q.double().numpy()[::3], -1)
    tok = np.array([np.searchsorted(c[i // 3], rng.random() * c[i // 3, -1]) for i in range(n)], np.int32).clip(0, V - 1)
    if not draft:
        best = np.argsort(-q.numpy()[::3], -1)[:, :2]
        tok[1::3], tok[2::3] = best[:, 0], best[:, 1]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    path = torch.empty(batch, 3, dtype=torch.int32, device="cuda")
    length, nxt = torch.empty(batch, dtype=torch.int32, device="cuda"), torch.empty(batch, dtype=torch.int32, device="cuda")
    S.s4kv_verify_tree(dev(tok), dev(parents), dev(cu), p.cuda(), q.cuda() if draft else None, dev(u), path, length, nxt)
    torch.cuda.synchronize()
    ref = verify_reference(tok, parents, cu, p.double().numpy(), q.double().numpy() if draft else None, u, 3)
    for got, want in zip((path, length, nxt), ref):
        assert np.array_equal(got.cpu().numpy(), want)


def test_batch_of_several_waves_of_clusters():
    """400 rows of 128256 entries: clusters of 4 in three waves."""
    import torch
    import int4_kivi_quantized_s4kv_b200 as S
    rng = np.random.default_rng(1)
    B, V = 400, 128256
    p = rng.random((B, V), dtype=np.float32) ** 8
    p /= p.sum(-1, keepdims=True)
    tok, parents, cu, u = np.zeros(B, np.int32), np.full(B, -1, np.int32), np.arange(B + 1, dtype=np.int32), rng.random(B, dtype=np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    path, length, nxt = (torch.empty(x, dtype=torch.int32, device="cuda") for x in ((B, 1), (B,), (B,)))
    S.s4kv_verify_tree(dev(tok), dev(parents), dev(cu), dev(p), None, dev(u), path, length, nxt)
    torch.cuda.synchronize()
    for got, want in zip((path, length, nxt), verify_reference(tok, parents, cu, p, None, u, 1)):
        assert np.array_equal(got.cpu().numpy(), want)
