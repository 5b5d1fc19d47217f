"""A case of tree attention in which only the remainders of the keys' fp16 rounding count, and the arithmetic by which
the kernel carries them, restated."""
from __future__ import annotations

import numpy as np

from int4_kivi_quantized_s4kv_b200 import workloads as W
from spec_helpers import SpecCache

TOKENS, ROWS = 48, 64
SM_SCALE = 128 ** -0.5


def filled(keys, values, bits=4, gpu=True):
    """A cache of one sequence that holds these keys and values [tokens][heads][128]."""
    n, heads, _ = keys.shape
    c = SpecCache([0], heads, bits, room=n // 16 + 1, key_scale=np.ones((heads, 128)), gpu=gpu)
    c.k, c.v, c.lens = [keys.astype(np.float16)], [values.astype(np.float16)], np.array([n], np.int32)
    at = W.slot_mapping(c.bt, [np.arange(n)])
    cu = np.array([0, n], np.int32)
    assert c.oc.append(c.k[0], c.v[0], at, cu, c.lens, c.bt) == 0
    if gpu:
        c.lens_dev = c.dev(c.lens)
        c.S.s4kv_append(c.gpu, c.dev(c.k[0]), c.dev(c.v[0]), c.dev(at), c.dev(cu), c.lens_dev, c.bt_dev, n)
    return c


def remainder_case(bits, gpu):
    """(cache, q, exact logits [rows][tokens], what the remainders are of each [rows][tokens], emulation).

    The queries are orthogonal to all dequantized keys, up to their rounding, and large: the logits are near 0 while
    what fp16 loses of each key moves them visibly.  Token t's value is level at channel t and 0 elsewhere (exact in any
    code width), so the outputs are the weights.  emulation(f): the logits with each key's remainder times f, cut and
    rounded as the kernel's e5m2 operands are."""
    import torch
    rng = np.random.default_rng(50 + bits)
    keys = (16 * rng.standard_normal((TOKENS, 1, 128))).astype(np.float16)
    level = (2 ** bits - 1) / 2 ** bits
    values = np.zeros((TOKENS, 1, 128))
    values[np.arange(TOKENS), 0, np.arange(TOKENS)] = level
    c = filled(keys, values, bits, gpu)
    full, val, _ = (x[:, 0] for x in c.cached(0))
    assert np.array_equal(val, values[:, 0])
    # the quantizer's formula: codes, scales and zero points of each page
    pages = keys[:, 0].reshape(-1, 16, 128).astype(np.float32)
    mn, mx = pages.min(1, keepdims=True), pages.max(1, keepdims=True)
    s = (mx - mn) / np.float32(2 ** bits - 1)
    code = np.clip(np.rint((pages - mn) / s), 0, 2 ** bits - 1).astype(np.float64)
    scale = s.astype(np.float16).astype(np.float64)
    dequantized = (code.astype(np.float32) * scale.astype(np.float32) + mn).astype(np.float64)
    assert np.array_equal(dequantized.reshape(-1, 128), full)
    quarter = (code / 4 * scale).reshape(-1, 128)
    hi = quarter.astype(np.float16).astype(np.float64)
    rem = (quarter - hi).astype(np.float16)
    assert np.array_equal(rem.astype(np.float64), quarter - hi)
    cut = (rem.view(np.uint16) & 0xFF00).view(np.float16).astype(np.float64)
    r = rng.standard_normal((ROWS, 128))
    basis, _ = np.linalg.qr(full.T)
    r -= r @ basis @ basis.T
    q = (90 * r).astype(np.float16)
    q64 = q.astype(np.float64)
    q8 = torch.from_numpy(q).to(torch.float8_e5m2).double().numpy()
    zero = (dequantized - code * scale).reshape(-1, 128)  # (with the fp32 rounding of the sum)
    parts = SM_SCALE * 4 * np.sqrt((q64 ** 2) @ (quarter - hi).T ** 2)

    def emulation(f):
        return SM_SCALE * (4 * (q64 @ hi.T + f * (q8 @ cut.T)) + q64 @ zero.T)

    return c, q.reshape(ROWS, 1, 128), q64 @ full.T * SM_SCALE, parts, emulation


def remainder_error(logits, exact, parts):
    """How much of the remainders the logits miss: 1 without them, 2 with the wrong sign.

    A remainder is cut to 3 significant bits (a loss below 1/4 of it) against a query rounded to as many (1/8): at most
    1 - 3/4 * 7/8 = 0.344 of each product, whose signs are random, so that their squares add up: at most 0.344.  The sums
    in fp32 and the outputs' rounding are 0.03 of them here (2^-20 of 2e4, 2^-10 of 1, against 0.4)."""
    return float(np.sqrt(((logits - exact) ** 2).mean() / (parts ** 2).mean()))


REMAINDER_BOUND = 0.344 + 0.03
