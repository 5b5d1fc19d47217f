"""References of the speculative-decoding calls in 64 bits: plain numpy over
the oracle's dequantized pages, written from the definitions."""
from __future__ import annotations

import numpy as np

from int4_kivi_quantized_s4kv_b200 import workloads as W

PAGE = 16


def random_parents(rng, n, newest):
    """Node i hangs off one of the `newest` nodes before it, node 0 off the cache (0: every node does)."""
    if n == 0:
        return np.zeros(0, np.int32)
    i = np.arange(n)
    back = rng.integers(1, newest + 1, size=n) if newest else n + 1
    return np.where(i == 0, -1, np.maximum(i - back, 0 if newest else -1)).astype(np.int32)


class SpecCache:
    """The same cache on the GPU and in the oracle, holding `lens` tokens, with `room` more pages a sequence."""

    def __init__(self, lens, heads, bits=4, seed=0, room=0, key_scale=None, gpu=True):
        import oracle
        self.lens = np.asarray(lens, np.int32)
        self.H, self.bits, B = heads, bits, len(lens)
        rng = np.random.default_rng(seed)
        self.max_pages = int(max(1, max((int(L) + PAGE - 1) // PAGE for L in lens) + room))
        pages = B * self.max_pages + 2
        self.bt = rng.permutation(pages)[:B * self.max_pages].reshape(B, self.max_pages).astype(np.int32)
        if key_scale is None:
            key_scale = np.ones((heads, 128))
            key_scale[:, rng.integers(0, 128, 3)] = 8.0
        self.key_scale = key_scale
        self.k = [(rng.standard_normal((int(L), heads, 128)) * key_scale).astype(np.float16) for L in lens]
        self.v = [rng.standard_normal((int(L), heads, 128)).astype(np.float16) for L in lens]
        self.oc = oracle.OracleCache(pages, heads, B, bits=bits)
        self.gpu = None
        if gpu:
            import int4_kivi_quantized_s4kv_b200 as S
            self.S = S
            self.gpu = S.S4KVCache(pages, heads, B, bits=bits)
            self.bt_dev = self.dev(self.bt)
            self.lens_dev = self.dev(self.lens)
        if self.lens.sum():
            cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
            k, v = np.concatenate(self.k), np.concatenate(self.v)
            sm = W.slot_mapping(self.bt, [np.arange(int(L)) for L in lens])
            assert self.oc.append(k, v, sm, cu, self.lens, self.bt) == 0
            if gpu:
                self.S.s4kv_append(self.gpu, self.dev(k), self.dev(v), self.dev(sm), self.dev(cu), self.lens_dev,
                                   self.bt_dev, int(self.lens.max()))

    def dev(self, a):
        import torch
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def cached(self, b):
        """Keys and values of sequence b's cached tokens, float64 [L][heads][128], and how far a quantized key
        is above its zero point (0 for residual rows)."""
        L = int(self.lens[b])
        k, v, up = [], [], []
        for j in range(L // PAGE):
            pk, pv = self.oc.dequant_page(int(self.bt[b, j]))  # [heads][16][128]
            pk, pv = np.asarray(pk, np.float64), np.asarray(pv, np.float64)
            k.append(pk.transpose(1, 0, 2))
            v.append(pv.transpose(1, 0, 2))
            up.append((pk - pk.min(1, keepdims=True)).transpose(1, 0, 2))
        r = L % PAGE
        z = np.zeros((0, self.H, 128))
        k.append(self.k[b][L - r:].astype(np.float64) if r else z)
        v.append(self.v[b][L - r:].astype(np.float64) if r else z)
        up.append(np.zeros((r, self.H, 128)))
        return np.concatenate(k), np.concatenate(v), np.concatenate(up)


def tree_reference(c, q, k, v, cu, parents, sm_scale=128 ** -0.5):
    """(out, bound): the attention in float64, and how far an fp16 result may be from it.

    bound: the output's rounding, 2^-11 |out|; the values' rounding to fp16, 2^-11 sum w|v|; and the logits'
    error d, which changes a weight by at most a factor e^(+-2d) (its own and the sum's): 2 d sum w|v|.  d:
    a quantized key is carried as an fp16 product code * scale plus its remainder in 3 significant bits, against a
    query in as many, so what is lost of each is 2 * 2^-14 of the product, at least 2^-15; sums in fp32 add
    2^-20 of what is summed.  Weights are carried to 2^-20."""
    heads = c.H
    G = q.shape[1] // heads
    out = np.full(q.shape, np.nan)
    bound = np.full(q.shape, np.nan)
    for b in range(len(c.lens)):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if hi <= lo:
            continue
        m = hi - lo
        ck, cv, up = c.cached(b)
        see = np.zeros((m, m), bool)
        for i in range(m):
            a = i
            while a >= 0:
                see[i, a] = True
                a = int(parents[lo + a])
        kk = np.concatenate([ck, k[lo:hi].astype(np.float64)])
        vv = np.concatenate([cv, v[lo:hi].astype(np.float64)])
        lost = np.concatenate([up * 2.0 ** -13 + 2.0 ** -15, np.zeros((m, heads, 128))]) \
            + (np.abs(kk) * 2 + np.concatenate([up, np.zeros((m, heads, 128))])) * 2.0 ** -20 + 2.0 ** -24
        mask = np.concatenate([np.ones((m, len(ck)), bool), see], 1)
        for h in range(heads):
            qq = q[lo:hi, h * G:(h + 1) * G].astype(np.float64)
            s = np.einsum("mgd,td->mgt", qq, kk[:, h]) * sm_scale
            s = np.where(mask[:, None, :], s, -np.inf)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            d = np.einsum("mgd,td->mgt", np.abs(qq), lost[:, h]) * sm_scale
            d = np.where(mask[:, None, :], d, 0).max(-1)[..., None]
            o = w @ vv[:, h]
            a = w @ np.abs(vv[:, h])
            out[lo:hi, h * G:(h + 1) * G] = o
            bound[lo:hi, h * G:(h + 1) * G] = 2.0 ** -11 * np.abs(o) + (2.0 ** -11 + 2 * d + 2.0 ** -19) * a + 2.0 ** -24
    return out, bound


def verify_reference(tokens, parents, cu, target, draft, uniforms, max_nodes):
    """(path, path_len, next_token) from the definition, in float64."""
    B = len(cu) - 1
    path = np.full((B, max_nodes), -1, np.int32)
    length, nxt = np.zeros(B, np.int32), np.full(B, -1, np.int32)

    def row(rows, i):
        x = rows[i].astype(np.float64)
        return np.where(x > 0, x, 0.0)

    for b in range(B):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if hi <= lo:
            continue
        cur, got = 0, [0]
        V = target.shape[1]
        while True:
            left, mass, taken = row(target, lo + cur), 1.0, False
            for c in range(cur + 1, hi - lo):
                x = int(tokens[lo + c])
                if int(parents[lo + c]) != cur or not 0 <= x < V:
                    continue
                Q = row(draft, lo + cur) if draft is not None else None
                if float(uniforms[lo + c]) * mass * (Q[x] if Q is not None else 1.0) < left[x]:
                    got.append(c)
                    cur, taken = c, True
                    break
                if Q is not None:
                    left = np.maximum(left - mass * Q, 0.0)
                    mass = left.sum()
                else:
                    mass -= left[x]
                    left[x] = 0.0
            if not taken:
                break
        path[b, :len(got)] = got
        length[b] = len(got)
        if not left.sum() > 0:
            left = row(target, lo + cur)
        total = left.sum()
        if not (total > 0 and np.isfinite(total)):
            continue
        over = np.nonzero(np.cumsum(left) > float(uniforms[lo]) * total)[0]
        nxt[b] = over[0] if len(over) else np.nonzero(left > 0)[0][-1]
    return path, length, nxt
