"""Cases of one speculative-decoding step over the paged quantized KV cache.

Three operators, as a serving loop runs them one after the other:

  tree    attention of a tree of drafted tokens over the cache (s4kv_tree_attention)
  verify  acceptance of drafted tokens against the target's probabilities (s4kv_verify_tree)
  commit  append of the accepted path's keys and values to the cache (s4kv_append_path),
          read back as the values its pages stand for (s4kv_dequant_pages)

``own`` false: the plain forms, elementary torch operations in 32 bits (64 for
the verification's sums).  ``own`` true: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DIM, PAGE, GROUP = 128, 16, 32


# ------------------------------------------------------------------ cases --

def _tree(name, batch, hq, hkv, lo, hi, n_lo, n_hi, bits=4, keys="outliers"):
    return {"name": name, "op": "tree", "batch": batch, "hq": hq, "hkv": hkv, "ctx_lo": lo, "ctx_hi": hi,
            "n_lo": n_lo, "n_hi": n_hi, "bits": bits, "keys": keys}


def _verify(name, batch, vocab, n_lo, n_hi, branch, draft, dtype="float32"):
    return {"name": name, "op": "verify", "batch": batch, "vocab": vocab, "n_lo": n_lo, "n_hi": n_hi,
            "branch": branch, "draft": draft, "dtype": dtype}


def _commit(name, batch, hkv, n_lo, n_hi, depth, bits=4):
    return {"name": name, "op": "commit", "batch": batch, "hkv": hkv, "n_lo": n_lo, "n_hi": n_hi,
            "depth": depth, "bits": bits}


def listed():
    return [
        # the smallest call: two short sequences, one kv head, three drafted tokens each
        _tree("tree-tiny", 2, 4, 1, 37, 50, 3, 3),
        # one interactive user with a long context: one sequence has to fill the card
        _tree("tree-single-32k", 1, 32, 8, 32768, 32768, 16, 16, keys="lognormal"),
        # an ordinary serving batch: ragged contexts, ragged small trees, group of 7 query heads
        _tree("tree-ragged-g7", 64, 28, 4, 512, 4096, 3, 9),
        # a large batch at 8K context: bound by the cache's bytes
        _tree("tree-8k-batch64", 64, 32, 8, 8192, 8192, 16, 16, keys="lognormal"),
        # a wide tree of 64 nodes, group of 8, long context: bound by the tensor cores
        _tree("tree-wide-32k", 8, 64, 8, 32768, 32768, 64, 64),
        # 8-bit pages, mixed contexts
        _tree("tree-int8", 16, 24, 8, 128, 4095, 5, 12, bits=8),
        # one user, a chain of four drafted tokens, full draft rows
        _verify("verify-single", 1, 32000, 5, 5, 1, True),
        # a batch of chains with full draft rows over a large vocabulary
        _verify("verify-chain-batch64", 64, 128256, 5, 8, 1, True),
        # trees of the draft's best tokens (no draft rows), bf16 probabilities
        _verify("verify-tree-bf16", 48, 128256, 12, 16, 3, False, "bfloat16"),
        # trees with several draws from one draft row each (every rejection changes what is left), fp16
        _verify("verify-tree-draft", 16, 32000, 9, 12, 3, True, "float16"),
        # one user's accepted path
        _commit("commit-single", 1, 8, 8, 8, 4),
        # a large batch's accepted paths: a third of the sequences complete a page
        _commit("commit-batch128", 128, 8, 16, 16, 8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "verify", "commit"))
    if op == "tree":
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.randint(1, 8)
        ctx = _log_int(rng, 16, 32768)
        n = _log_int(rng, 1, 64)
        # no more than half of the largest listed case's work
        most = 4 * 64 * 64 * 32768 / (hq * n * ctx)
        batch = min(_log_int(rng, 1, 64), max(1, int(most)), max(1, int(2e6 / (ctx * hkv)) * 2))
        c = _tree("", batch, hq, hkv, rng.randint(max(1, ctx // 3), ctx), ctx, rng.randint(max(1, n // 2), n), n,
                  rng.choice((4, 4, 4, 8, 2)), rng.choice(("outliers", "lognormal")))
    elif op == "verify":
        vocab = _log_int(rng, 1000, 128256)
        branch = rng.choice((1, 1, 2, 3))
        n = rng.randint(2, 12)
        c = _verify("", _log_int(rng, 1, 48), vocab, rng.randint(2, n), n, branch, rng.random() < 0.6,
                    rng.choice(("float32", "float32", "bfloat16", "float16")))
    else:
        n = rng.randint(2, 48)
        c = _commit("", _log_int(rng, 1, 128), rng.choice((1, 2, 4, 8)), rng.randint(2, n), n,
                    rng.randint(1, min(n, 12)), rng.choice((4, 4, 8, 2)))
    del c["name"]
    return c


def work(case):
    B = case["batch"]
    n = (case["n_lo"] + case["n_hi"]) / 2
    if case["op"] == "tree":
        L = (case["ctx_lo"] + case["ctx_hi"]) / 2
        pages = max(0.0, (L - 7.5) / PAGE)  # a context ends inside a page, half full on average
        if case["ctx_lo"] == case["ctx_hi"]:
            pages = case["ctx_lo"] // PAGE
        by = B * case["hkv"] * (pages * _block(case["bits"]) + (L - PAGE * pages) * 512 + n * 512)
        by += B * n * case["hq"] * DIM * 2 * 2
        return {"bytes": by, "flops": 4.0 * DIM * case["hq"] * B * n * (L + n / 2)}
    if case["op"] == "verify":
        # the row that the last token is drawn from, and the draft's row for it (nearly every walk
        # ends by a rejection); the tokens that are only tested cost a few bytes each
        es = torch.finfo(getattr(torch, case["dtype"])).bits // 8
        return {"bytes": float(B * case["vocab"] * es * (2 if case["draft"] else 1)),
                "flops": 3.0 * B * case["vocab"]}
    m = (1 + case["depth"]) / 2  # tokens a path
    done = m / PAGE              # pages that a path completes
    by = B * case["hkv"] * (m * 512 * 2 + done * (PAGE * 512 + _block(case["bits"])))
    return {"bytes": by, "flops": B * case["hkv"] * done * PAGE * DIM * 2 * 6.0}


# ----------------------------------------------------------------- layout --

def _block(bits):
    return 2 * PAGE * DIM * bits // 8 + 768


def _places(bits, device):
    """Where the code of (token, channel) stands in its region's stream of codes (lowest bits first):
    ([16, 128] for keys, the same for values)."""
    t = torch.arange(PAGE, device=device)[:, None]
    c = torch.arange(DIM, device=device)[None, :]
    # operand tile, lane, register and half of the tensor-core fragment that holds it
    spots = ((c % 32 // 4, 4 * (t % 8) + c // 32, t // 8 + 2 * (c % 4 // 2), c % 2),
             (2 * (c // 32) + c % 4 // 2, 4 * (c % 32 // 4) + t % 8 // 2, c % 2 + 2 * (t // 8), t % 2))
    out = []
    for tile, lane, reg, half in spots:
        tile, lane, reg, half = torch.broadcast_tensors(tile, lane, reg, half)
        if bits == 4:
            p = 8 * (128 * (tile // 4) + 4 * lane + tile % 4) + reg % 2 + 2 * half + 4 * (reg // 2)
        elif bits == 8:
            p = (tile // 2 * 32 + lane) * 16 + tile % 2 * 8 + 2 * reg + half
        else:
            p = 16 * (4 * lane + tile // 2) + 8 * half + 4 * (tile % 2) + reg
        out.append(p)
    return out


def _meta_places(device):
    c = torch.arange(DIM, device=device)
    t = torch.arange(PAGE, device=device)[:, None]
    g = torch.arange(DIM // GROUP, device=device)[None, :]
    zero_k = 16 * (c % 32 // 4) + 2 * (c // 32) + c % 2 + 8 * (c % 4 // 2)
    scale_v = 16 * (t % 8 // 2) + 8 * (t // 8) + 2 * g + t % 2
    zero_v = g * PAGE + t
    return zero_k, scale_v, zero_v


def _codes(region, places, bits):
    """uint8 [..., bytes] -> the codes [..., 16, 128], as fp32."""
    per = 8 // bits
    shift = torch.arange(0, 8, bits, device=region.device, dtype=torch.uint8)
    s = region if per == 1 else ((region[..., None] >> shift) & ((1 << bits) - 1)).flatten(-2)
    return s[..., places.reshape(-1)].unflatten(-1, (PAGE, DIM)).float()


def _dequant(blocks, bits):
    """uint8 [..., block] -> fp32 keys and values [..., 16, 128]."""
    pk, pv = _places(bits, blocks.device)
    zk, sv, zv = _meta_places(blocks.device)
    n = PAGE * DIM * bits // 8
    meta = blocks[..., 2 * n:].contiguous().view(torch.float16).float()
    k = _codes(blocks[..., :n], pk, bits) * meta[..., None, :DIM] + meta[..., DIM + zk][..., None, :]
    s = meta[..., 2 * DIM + sv].repeat_interleave(GROUP, -1)
    z = meta[..., 2 * DIM + 64 + zv].repeat_interleave(GROUP, -1)
    return k, _codes(blocks[..., n:2 * n], pv, bits) * s + z


def _quantize(k, v, bits):
    """fp16 keys and values [..., 16, 128] -> uint8 [..., block]."""
    top = (1 << bits) - 1
    pk, pv = _places(bits, k.device)
    zk, sv, zv = _meta_places(k.device)

    def group(x, dim):  # the group's axis is `dim`
        lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
        s = (hi - lo) / torch.full_like(lo, top)  # a quotient; by a Python number torch multiplies by its reciprocal
        code = torch.where(s == 0, torch.zeros_like(x), torch.round((x - lo) / s).clamp(0, top))
        return code, s, lo

    def pack(code, places):
        x = torch.empty_like(code.flatten(-2), dtype=torch.uint8)
        x[..., places.reshape(-1)] = code.flatten(-2).to(torch.uint8)
        per = 8 // bits
        if per == 1:
            return x
        w = 1 << torch.arange(0, 8, bits, device=x.device, dtype=torch.int32)
        return (x.unflatten(-1, (-1, per)).int() * w).sum(-1).to(torch.uint8)

    ck, sk, lk = group(k.float(), -2)
    cv, s_v, lv = group(v.float().unflatten(-1, (DIM // GROUP, GROUP)), -1)
    meta = torch.empty(*k.shape[:-2], 2 * DIM + 128, dtype=torch.float16, device=k.device)
    meta[..., :DIM] = sk[..., 0, :].half()
    meta[..., DIM + zk] = lk[..., 0, :].half()
    meta[..., (2 * DIM + sv).reshape(-1)] = s_v[..., 0].half().flatten(-2)
    meta[..., (2 * DIM + 64 + zv).reshape(-1)] = lv[..., 0].half().flatten(-2)
    return torch.cat((pack(ck, pk), pack(cv.flatten(-2), pv), meta.view(torch.uint8)), -1)


# ----------------------------------------------------------------- inputs --

def _gen(seed, *more):
    g = torch.Generator(device="cuda")
    h = int(seed) & 0x7FFFFFFF
    for x in more:
        h = (h * 1000003 + int(x) + 1) & 0x7FFFFFFFFFFF
    g.manual_seed(h)
    return g


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")


def _forest(g, counts, branch):
    """parents of every node: node 0 is a root, node i hangs off a random one of the `branch` newest nodes
    (1: a chain)."""
    out = []
    for n in counts:
        i = torch.arange(n, device="cuda")
        back = _ints(g, 1, branch, n)
        out.append(torch.where(i == 0, -1, (i - back).clamp(min=0)))
    return torch.cat(out).int()


def _key_scale(case, g):
    hkv = case["hkv"]
    if case.get("keys") == "lognormal":  # key channels of very different sizes
        return torch.exp(0.75 * torch.randn(hkv, DIM, generator=g, device="cuda"))
    sc = torch.ones(hkv, DIM, device="cuda")  # or a few large ones
    at = torch.rand(hkv, DIM, generator=g, device="cuda").topk(3, -1).indices
    return sc.scatter_(-1, at, 8.0)


def _cache(case, g, lens, spare):
    """Pool, residual and shuffled page tables of a cache holding `lens` tokens, room for `spare` more."""
    B, H, bits = case["batch"], case["hkv"], case["bits"]
    most = int((lens.max().item() + spare + PAGE - 1) // PAGE)
    pages = B * most + 3
    bt = torch.randperm(pages, generator=g, device="cuda")[:B * most].view(B, most).int()
    pool = torch.zeros(pages, H, _block(bits), dtype=torch.uint8, device="cuda")
    ks = _key_scale(case, g)
    full = lens // PAGE
    at = torch.arange(most, device="cuda")[None, :] < full[:, None]
    ids = bt[at].long()
    step = max(1, (1 << 25) // (H * PAGE * DIM))
    for i in range(0, ids.numel(), step):
        part = ids[i:i + step]
        k = torch.randn(part.numel(), H, PAGE, DIM, generator=g, device="cuda") * ks[:, None, :]
        v = torch.randn(part.numel(), H, PAGE, DIM, generator=g, device="cuda")
        pool[part] = _quantize(k.half(), v.half(), bits)
    res_k = (torch.randn(B, H, PAGE, DIM, generator=g, device="cuda") * ks[:, None, :]).half()
    res_v = torch.randn(B, H, PAGE, DIM, generator=g, device="cuda").half()
    return pool, res_k, res_v, bt, ks


def _handle(case, s):
    """The framework's cache over these contents."""
    import int4_kivi_quantized_s4kv_b200 as S
    c = S.S4KVCache(s["pool"].shape[0], case["hkv"], case["batch"], "cuda", case["bits"])
    c.pool.copy_(s["pool"])
    c.res_k.copy_(s["res_k"])
    c.res_v.copy_(s["res_v"])
    s["pool"], s["res_k"], s["res_v"] = c.pool, c.res_k, c.res_v
    return c


def _counts(case, g):
    """Nodes of each sequence: the whole range, in an order of the seed's."""
    n = case["n_hi"] - torch.arange(case["batch"], device="cuda") % (case["n_hi"] - case["n_lo"] + 1)
    return n[torch.randperm(case["batch"], generator=g, device="cuda")]


def prepare(case, seed):
    g = _gen(seed, sum(map(ord, case["op"])))
    B = case["batch"]
    counts = _counts(case, g)
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0))).int()
    total = int(cu[-1])
    s = {"case": case, "cu": cu, "most": case["n_hi"]}
    if case["op"] == "verify":
        V, dt = case["vocab"], getattr(torch, case["dtype"])
        s["parents"] = _forest(g, counts.tolist(), case["branch"])
        # the draft's distribution of what follows each node, and a target's that is near it
        z = torch.randn(total, V, generator=g, device="cuda").mul_(2.5)
        draft = torch.softmax(z, -1)
        z += torch.randn(total, V, generator=g, device="cuda").mul_(0.6)
        s["target"] = torch.softmax(z, -1).to(dt)
        del z
        base = torch.repeat_interleave(cu[:-1].long(), counts)
        up = (base + s["parents"].clamp(min=0))
        # a node's token: drawn from the row of its parent, or (no draft rows) one of the parent's best
        if case["draft"]:
            tok = torch.multinomial(draft[up], 1, generator=g)[:, 0]
        else:
            rank = torch.arange(total, device="cuda") % case["branch"]
            tok = draft.topk(case["branch"], -1).indices[up, rank]
        s["draft"] = draft.to(dt) if case["draft"] else None
        s["tokens"] = tok.int()
        s["uniforms"] = torch.rand(total, generator=g, device="cuda")
        if own:
            s["path"] = torch.empty(B, s["most"], dtype=torch.int32, device="cuda")
            s["path_len"] = torch.empty(B, dtype=torch.int32, device="cuda")
            s["next"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "tree":
        lens = _ints(g, case["ctx_lo"], case["ctx_hi"], B)
        lens[0] = case["ctx_hi"]
        s["pool"], s["res_k"], s["res_v"], s["bt"], ks = _cache(case, g, lens, 0)
        s["lens"] = lens.int()
        s["parents"] = _forest(g, counts.tolist(), 3)
        s["q"] = torch.randn(total, case["hq"], DIM, generator=g, device="cuda").half()
        s["k"] = (torch.randn(total, case["hkv"], DIM, generator=g, device="cuda") * ks).half()
        s["v"] = torch.randn(total, case["hkv"], DIM, generator=g, device="cuda").half()
        if own:
            import int4_kivi_quantized_s4kv_b200 as S
            s["cache"] = _handle(case, s)
            s["out"] = torch.empty_like(s["q"])
            s["ws"] = S.tree_workspace(case["hq"], case["hkv"], B, s["most"])
        return s
    lens = _ints(g, 1, 79, B)
    s["pool"], s["res_k"], s["res_v"], s["bt"], ks = _cache(case, g, lens, case["depth"] + PAGE)
    s["lens"] = lens.int()
    s["k"] = (torch.randn(total, case["hkv"], DIM, generator=g, device="cuda") * ks).half()
    s["v"] = torch.randn(total, case["hkv"], DIM, generator=g, device="cuda").half()
    # accepted paths: ascending node numbers from node 0, -1 behind the end
    most = torch.minimum(counts, torch.full_like(counts, case["depth"]))
    ln = 1 + (torch.rand(B, generator=g, device="cuda") * most).long().clamp(max=case["depth"] - 1)
    ln = torch.minimum(ln, most)
    r = torch.rand(B, s["most"], generator=g, device="cuda")
    r = torch.where(torch.arange(s["most"], device="cuda")[None, :] < counts[:, None], r, 2.0)
    r[:, 0] = -1
    rank = r.argsort(-1).argsort(-1)
    pick = torch.where(rank < ln[:, None], torch.arange(s["most"], device="cuda")[None, :], 1 << 20).sort(-1).values
    s["path"] = torch.where(pick < (1 << 20), pick, -1).int()
    s["path_len"] = ln.int()
    # the pages that a path may complete
    span = (PAGE - 1 + case["depth"]) // PAGE
    s["span"] = span
    s["pages"] = s["bt"].gather(1, (lens // PAGE)[:, None] + torch.arange(span, device="cuda")[None, :]).reshape(-1).contiguous()
    if own:
        s["cache"] = _handle(case, s)
        s["new_lens"] = torch.empty_like(s["lens"])
        s["pk"] = torch.empty(s["pages"].numel(), case["hkv"], PAGE, DIM, device="cuda")
        s["pv"] = torch.empty_like(s["pk"])
    return s


# -------------------------------------------------------------- the passes --

def run(s):
    if own:
        import int4_kivi_quantized_s4kv_b200 as S
        if s["case"]["op"] == "tree":
            S.s4kv_tree_attention(s["cache"], s["q"], s["k"], s["v"], s["cu"], s["parents"], s["lens"], s["bt"], s["out"],
                                  s["most"], s["ws"])
            return s["out"]
        if s["case"]["op"] == "verify":
            S.s4kv_verify_tree(s["tokens"], s["parents"], s["cu"], s["target"], s["draft"], s["uniforms"],
                               s["path"], s["path_len"], s["next"])
            return {"path": s["path"], "path_len": s["path_len"], "next": s["next"]}
        S.s4kv_append_path(s["cache"], s["k"], s["v"], s["cu"], s["path"], s["path_len"], s["lens"], s["bt"], s["new_lens"])
        S.s4kv_dequant_pages(s["cache"], s["pages"], s["pk"], s["pv"])
        return {"new_lens": s["new_lens"], "res_k": s["res_k"], "res_v": s["res_v"], "pages_k": s["pk"], "pages_v": s["pv"]}
    return {"tree": _run_tree, "verify": _run_verify, "commit": _run_commit}[s["case"]["op"]](s)


def _run_tree(s):
    case = s["case"]
    B, H, n, bits = case["batch"], case["hkv"], s["most"], case["bits"]
    G = case["hq"] // H
    lens, cu = s["lens"].long(), s["cu"].long()
    counts = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    real = i[None, :] < counts[:, None]
    node = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    # keys and values: full pages, residual rows, drafted tokens
    pages = case["ctx_hi"] // PAGE
    kd, vd = _dequant(s["pool"][s["bt"][:, :pages].long()], bits)  # [B, pages, H, 16, 128]
    k = torch.cat((kd.permute(0, 2, 1, 3, 4).flatten(2, 3), s["res_k"].float(), s["k"][node].float().transpose(1, 2)), 2)
    del kd
    v = torch.cat((vd.permute(0, 2, 1, 3, 4).flatten(2, 3), s["res_v"].float(), s["v"][node].float().transpose(1, 2)), 2)
    del vd
    # who sees whom: reach = (self or parent) to the 64th power
    up = torch.where(real, s["parents"][node].long(), -1)
    reach = ((up[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(6):
        reach = (reach @ reach > 0).float()
    full = lens // PAGE * PAGE
    seen = torch.cat((torch.arange(pages * PAGE, device="cuda")[None, :] < full[:, None],
                      torch.arange(PAGE, device="cuda")[None, :] < (lens - full)[:, None]), 1)
    mask = torch.cat((seen[:, None, :].expand(B, n, -1), reach > 0), 2)  # [B, n, keys]
    q = s["q"][node].float().view(B, n, H, G, DIM).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, DIM)
    w = (q @ k.transpose(2, 3)).mul_(DIM ** -0.5).view(B, H, n, G, -1)
    w = w.masked_fill_(~mask[:, None, :, None, :], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    o = (w.view(B, H, n * G, -1) @ v).view(B, H, n, G, DIM) / w.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, H * G, DIM)[real].half()


def _run_verify(s):
    case = s["case"]
    B, n, V = case["batch"], s["most"], case["vocab"]
    cu = s["cu"].long()
    counts = cu[1:] - cu[:-1]
    start = cu[:-1]
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    mass = torch.ones(B, dtype=torch.float64, device="cuda")
    taken = torch.zeros(B, dtype=torch.float64, device="cuda")  # what is subtracted of the draft's row
    gone = torch.zeros(B, n, dtype=torch.bool, device="cuda")   # rejected children of the current node
    path = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    length = torch.ones(B, dtype=torch.long, device="cuda")
    i = torch.arange(n, device="cuda")
    tok = s["tokens"][(start[:, None] + i).clamp(max=s["tokens"].shape[0] - 1)].long()
    for c in range(1, n):  # a node's children come after it, in the order in which they are tried
        at = (start + c).clamp(max=s["tokens"].shape[0] - 1)
        tried = (c < counts) & (s["parents"][at] == cur)
        x = tok[:, c]
        p, u = s["target"][start + cur, x].double(), s["uniforms"][at].double()
        if case["draft"]:
            q = s["draft"][start + cur, x].double()
            left = (p - taken * q).clamp(min=0)
        else:
            q = torch.ones_like(p)
            left = torch.where(((tok == x[:, None]) & gone).any(1), 0.0, p)
        yes = tried & (u * mass * q < left)
        no = tried & ~yes
        if case["draft"]:
            taken = torch.where(no, taken + mass, taken)
            if case["branch"] > 1:
                rest = (s["target"][start + cur].double() - taken[:, None] * s["draft"][start + cur].double()).clamp(min=0).sum(-1)
                mass = torch.where(no, rest, mass)
        else:
            mass = torch.where(no, mass - left, mass)
            gone[:, c] |= no
        path.scatter_(1, torch.where(yes, length, 0)[:, None], torch.where(yes, c, 0).int()[:, None])
        length = length + yes
        cur = torch.where(yes, c, cur)
        mass, taken = torch.where(yes, 1.0, mass), torch.where(yes, 0.0, taken)
        gone &= ~yes[:, None]
    p = s["target"][start + cur].double()
    if case["draft"]:
        r = (p - taken[:, None] * s["draft"][start + cur].double()).clamp(min=0)
    else:
        out = torch.zeros(B, V, dtype=torch.int32, device="cuda").scatter_add_(1, tok, gone.int())
        r = torch.where(out > 0, 0.0, p)
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, p)
    cum = r.cumsum(-1)
    t = s["uniforms"][start].double() * r.sum(-1)
    nxt = (cum <= t[:, None]).sum(-1)
    last = torch.where(r > 0, torch.arange(V, device="cuda"), -1).amax(-1)
    return {"path": path, "path_len": length.int(), "next": torch.minimum(nxt, last).int()}


def _run_commit(s):
    case = s["case"]
    B, H, bits, span = case["batch"], case["hkv"], case["bits"], s["span"]
    lens, ln = s["lens"].long(), s["path_len"].long()
    first = lens // PAGE
    rows = (span + 1) * PAGE  # the pages that a path may complete, and the tail behind them
    j = torch.arange(rows, device="cuda")[None, :]
    off = lens[:, None] % PAGE
    step = (j - off)  # the path's token at this row
    new = (step >= 0) & (step < ln[:, None])
    node = s["path"].long().gather(1, step.clamp(0, s["most"] - 1)).clamp(min=0) + s["cu"][:-1].long()[:, None]
    node = node.clamp(max=s["k"].shape[0] - 1)
    old = j.expand(B, -1) % PAGE

    def rows_of(res, x):
        r = res.transpose(1, 2)  # [B, 16, H, 128]
        kept = r.gather(1, old[:, :, None, None].expand(-1, -1, H, DIM))
        return torch.where(new[:, :, None, None], x[node], kept)  # [B, rows, H, 128]

    k, v = rows_of(s["res_k"], s["k"]), rows_of(s["res_v"], s["v"])
    end = off + ln[:, None]
    done = (torch.arange(span, device="cuda")[None, :] + 1) * PAGE <= end  # [B, span]
    kp = k[:, :span * PAGE].unflatten(1, (span, PAGE)).transpose(2, 3)  # [B, span, H, 16, 128]
    vp = v[:, :span * PAGE].unflatten(1, (span, PAGE)).transpose(2, 3)
    ids = s["pages"].long()
    blocks = torch.where(done.reshape(-1)[:, None, None], _quantize(kp, vp, bits).flatten(0, 1), s["pool"][ids])
    s["pool"][ids] = blocks
    # the tail: the new rows of the page that is left partly filled
    tail = end // PAGE * PAGE
    at = tail + torch.arange(PAGE, device="cuda")[None, :]
    write = new.gather(1, at.clamp(max=rows - 1)) & (at < end)
    pick = at.clamp(max=rows - 1)[:, :, None, None].expand(-1, -1, H, DIM)
    for res, x in ((s["res_k"], k), (s["res_v"], v)):
        res.copy_(torch.where(write[:, :, None, None], x.gather(1, pick), res.transpose(1, 2)).transpose(1, 2))
    pk, pv = _dequant(blocks, bits)
    return {"new_lens": (lens + ln).int(), "res_k": s["res_k"], "res_v": s["res_v"], "pages_k": pk, "pages_v": pv}


# ------------------------------------------------------------- in 64 bits --

def _exact_tables(bits):
    """Byte and shift of the code of every (token, channel), found one by one."""
    tabs = []
    for value in (False, True):
        by, sh = np.zeros((PAGE, DIM), np.int64), np.zeros((PAGE, DIM), np.int64)
        for t in range(PAGE):
            for c in range(DIM):
                if value:
                    m, lane, r, e = 2 * (c // 32) + (c % 4) // 2, 4 * ((c % 32) // 4) + (t % 8) // 2, c % 2 + 2 * (t // 8), t % 2
                else:
                    m, lane, r, e = (c % 32) // 4, 4 * (t % 8) + c // 32, t // 8 + 2 * ((c % 4) // 2), c % 2
                if bits == 8:
                    b = 512 * (m // 2) + 16 * lane + 8 * (m % 2) + 2 * r + e
                    by[t, c], sh[t, c] = b, 0
                elif bits == 4:
                    nib = r % 2 + 2 * e + 4 * (r // 2)
                    by[t, c], sh[t, c] = 512 * (m // 4) + 16 * lane + 4 * (m % 4) + nib // 2, 4 * (nib % 2)
                else:
                    bit = 16 * e + 8 * (m % 2) + 2 * r
                    by[t, c], sh[t, c] = 16 * lane + 4 * (m // 2) + bit // 8, bit % 8
        tabs.append((torch.from_numpy(by).cuda(), torch.from_numpy(sh).cuda()))
    return tabs


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "commit":
        # the residual: rows of the page left partly filled come from the old residual or the path.
        # Pages: their codes are defined by 32-bit arithmetic, there is no value in 64 bits.
        out = [s["res_k"].double(), s["res_v"].double()]
        lens, ln, path, cu = s["lens"].tolist(), s["path_len"].tolist(), s["path"].tolist(), s["cu"].tolist()
        for b in range(case["batch"]):
            for a in range(ln[b]):
                pos = lens[b] + a
                if pos // PAGE == (lens[b] + ln[b]) // PAGE:
                    out[0][b, :, pos % PAGE] = s["k"][cu[b] + path[b][a]].double()
                    out[1][b, :, pos % PAGE] = s["v"][cu[b] + path[b][a]].double()
        return {"new_lens": None, "res_k": out[0], "res_v": out[1], "pages_k": None, "pages_v": None}
    bits, H = case["bits"], case["hkv"]
    G = case["hq"] // H
    (bk, sk), (bv, sv) = _exact_tables(bits)
    n = PAGE * DIM * bits // 8
    lens, cu, parents = s["lens"].tolist(), s["cu"].tolist(), s["parents"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    ch, tk = torch.arange(DIM, device="cuda"), torch.arange(PAGE, device="cuda")
    kz = (ch % 32) // 4 * 16 + ch // 32 * 2 + ch % 2 + (ch % 4) // 2 * 8
    for b in range(case["batch"]):
        lo, hi = cu[b], cu[b + 1]
        m = hi - lo
        full = lens[b] // PAGE
        see = torch.zeros(m, m, dtype=torch.bool)
        for i in range(m):
            a = i
            while a >= 0:
                see[i, a] = True
                a = parents[lo + a]
        see = see.cuda()
        for h in range(H):
            blk = s["pool"][s["bt"][b, :full].long(), h].long()  # [pages, block]
            f = s["pool"][s["bt"][b, :full].long(), h][:, 2 * n:].contiguous().view(torch.float16).double()
            kc = ((blk[:, bk] >> sk) & ((1 << bits) - 1)).double()
            vc = ((blk[:, n + bv] >> sv) & ((1 << bits) - 1)).double()
            k = kc * f[:, None, :DIM] + f[:, None, DIM + kz]
            g = (ch // GROUP)[None, :]
            at = tk[:, None] % 8 // 2 * 16 + tk[:, None] // 8 * 8 + 2 * g + tk[:, None] % 2
            v = vc * f[:, 256 + at] + f[:, 320 + g * PAGE + tk[:, None]]
            r = lens[b] % PAGE
            k = torch.cat((k.reshape(-1, DIM), s["res_k"][b, h, :r].double(), s["k"][lo:hi, h].double()))
            v = torch.cat((v.reshape(-1, DIM), s["res_v"][b, h, :r].double(), s["v"][lo:hi, h].double()))
            x = torch.einsum("nd,kd->nk", s["q"][lo:hi, h * G:(h + 1) * G].double().reshape(-1, DIM), k) / math.sqrt(DIM)
            x = x.view(m, G, -1)
            x[:, :, lens[b]:].masked_fill_(~see[:, None, :], -math.inf)
            out[lo:hi, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return out
