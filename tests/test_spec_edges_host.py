"""Calls of speculative decoding that are refused before anything is launched, and the statistics of the tests of its
numerics, without a GPU."""
import ctypes

import pytest

from tree_helpers import REMAINDER_BOUND, remainder_case, remainder_error


@pytest.fixture(scope="module")
def S():
    from int4_kivi_quantized_s4kv_b200 import build
    build.build()
    import int4_kivi_quantized_s4kv_b200 as S
    return S


FAR = 1 << 20  # between two arrays; the addresses are never dereferenced


def verify_with(S, **kw):
    """s4kv_verify_tree of 4 sequences of 3 nodes with arrays far apart but for `kw`."""
    names = ("tok", "par", "cu", "t", "d", "u", "path", "ln", "nxt")
    a = {x: FAR * (i + 1) for i, x in enumerate(names)}
    a.update({x: f(a) for x, f in kw.items()})
    P = ctypes.c_void_p
    return S.lib().s4kv_verify_tree(P(a["tok"]), P(a["par"]), P(a["cu"]), 12, 4, 3, P(a["t"]), 100, P(a["d"]), 100, 0, 100,
                                    P(a["u"]), P(a["path"]), P(a["ln"]), P(a["nxt"]), None, P(0))


def test_verify_refuses_results_in_its_inputs(S):
    """Other sequences' CTAs still read what the first to finish would overwrite."""
    sizes = {"tok": 48, "par": 48, "u": 48, "cu": 20}
    for x, size in sizes.items():
        for out, own in (("path", 48), ("ln", 16), ("nxt", 16)):
            for at in (0, size - 4, -(own - 4)):
                assert verify_with(S, **{out: lambda a, x=x, at=at: a[x] + at}) == S.ERR_INVALID_ARG, (x, out, at)
    for x, y, size in (("ln", "nxt", 16), ("path", "ln", 48), ("path", "nxt", 48)):
        for at in (0, size - 4, -12):
            assert verify_with(S, **{y: lambda a, x=x, at=at: a[x] + at}) == S.ERR_INVALID_ARG, (x, y, at)


def test_tree_attention_refuses_results_in_its_inputs(S):
    names = ("q", "k", "v", "cu", "par", "sl", "bt", "out", "ws")
    P = ctypes.c_void_p
    c = S.s4kv_cache_t(FAR * 20, FAR * 21, FAR * 22, None, 10, 2, 4, 128, 16)

    def call(out):  # 4 nodes of 2 kv heads and 8 query heads
        a = {x: FAR * (i + 1) for i, x in enumerate(names)}
        a["out"] = out(a)
        return S.lib().s4kv_tree_attention(ctypes.byref(c), P(a["q"]), P(a["k"]), P(a["v"]), 8, 4, P(a["cu"]), P(a["par"]),
                                           P(a["sl"]), P(a["bt"]), 1, 1, 4, 0.1, P(a["out"]), P(a["ws"]), 0, P(0))

    for x, size in (("k", 2048), ("v", 2048), ("q", 8192)):
        for at in (size - 16, 16, -(8192 - 16)) + ((0,) if x != "q" else ()):
            assert call(lambda a, x=x, at=at: a[x] + at) == S.ERR_INVALID_ARG, (x, at)
    # next to them, or the queries' own place: refused for the workspace alone, of no bytes (without a device: for that)
    for out in (lambda a: a["q"], lambda a: a["k"] + 2048, lambda a: a["v"] - 8192, lambda a: a["q"] + 8192):
        assert call(out) in (S.ERR_WORKSPACE, S.ERR_CUDA)


def test_append_path_refuses_new_lengths_in_its_inputs(S):
    names = ("k", "v", "cu", "path", "ln", "sl", "bt")
    a = {x: FAR * (i + 1) for i, x in enumerate(names)}
    P = ctypes.c_void_p
    c = S.s4kv_cache_t(FAR * 20, FAR * 21, FAR * 22, None, 10, 2, 4, 128, 16)
    for x, size in (("cu", 20), ("path", 48), ("ln", 16), ("sl", 16), ("bt", 32)):
        for at in (0, size - 4, -12):
            got = S.lib().s4kv_append_path(ctypes.byref(c), P(a["k"]), P(a["v"]), 12, P(a["cu"]), P(a["path"]), P(a["ln"]), 3,
                                           P(a["sl"]), P(a["bt"]), 4, 2, P(a[x] + at), P(0))
            assert got == S.ERR_INVALID_ARG, (x, at)


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_the_measure_of_the_keys_remainders_tells_them_from_none(oracle_mod, bits):
    """The kernel's arithmetic passes; without the remainders, with half, twice or minus them it does not."""
    _, _, exact, parts, emulation = remainder_case(bits, False)
    assert remainder_error(emulation(1), exact, parts) <= REMAINDER_BOUND
    for wrong in (0, 0.5, 2, -1):
        assert remainder_error(emulation(wrong), exact, parts) > REMAINDER_BOUND, wrong


class Elsewhere:
    """A tensor's type, shape and address on a device that this machine need not have."""

    def __init__(self, t, device):
        self.t, self.device, self.dtype, self.shape = t, device, t.dtype, t.shape

    def get_device(self):
        return self.device

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("moved", range(8))
def test_wrappers_refuse_tensors_on_two_devices(S, moved):
    import torch
    i32 = lambda *x: torch.zeros(*x, dtype=torch.int32)  # noqa: E731
    f16 = lambda *x: torch.zeros(*x, dtype=torch.float16)  # noqa: E731
    cache = S.S4KVCache(4, 1, 1, device="cpu")
    cache.pool = Elsewhere(cache.pool, 0)
    at = lambda ts: [Elsewhere(t, 1 if i == moved else 0) for i, t in enumerate(ts)]  # noqa: E731
    q, k, v, cu, par, sl, bt, out = at([f16(2, 4, 128), f16(2, 1, 128), f16(2, 1, 128), i32(2), i32(2), i32(1), i32(1, 3), f16(2, 4, 128)])
    with pytest.raises(ValueError, match="all tensors must be on CUDA device 0"):
        S.s4kv_tree_attention(cache, q, k, v, cu, par, sl, bt, out, 2, Elsewhere(torch.zeros(16, dtype=torch.uint8), 0))
    k, v, cu, path, ln, sl, bt, new = at([f16(2, 1, 128), f16(2, 1, 128), i32(2), i32(1, 2), i32(1), i32(1), i32(1, 3), i32(1)])
    with pytest.raises(ValueError, match="all tensors must be on CUDA device 0"):
        S.s4kv_append_path(cache, k, v, cu, path, ln, sl, bt, new)
    if moved:  # the first one names the device
        t, tok, par, cu, q, u, path, ln = at([torch.zeros(2, 5), i32(2), i32(2), i32(2), torch.zeros(2, 5), torch.zeros(2), i32(1, 2), i32(1)])
        with pytest.raises(ValueError, match="all tensors must be on CUDA device 0"):
            S.s4kv_verify_tree(tok, par, cu, t, q, u, path, ln, Elsewhere(i32(1), 0))
