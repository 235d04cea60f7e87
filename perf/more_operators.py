"""Cases of the prompt, draft-tree and block-table operators.

Four groups, next to the library's paged decode, multi-query and append calls:

* prompt attention: whole prompts, packed end to end, attend to their own keys
  and values as the projections left them (causal, grouped heads);
* tree attention: a request's newest tokens are the nodes of a tree of drafted
  tokens; each sees the context and its own ancestors (bf16 and E4M3 caches);
* acceptance: the greedy walk down the tree, and the accepted nodes' rows
  closing up behind the context, in every layer's caches;
* block tables: new tokens get blocks from a pool on the GPU, with a slot and a
  position a row, their rows are written by slot, and blocks go back.

With ``own`` false the operators are computed from elementary torch
operations in fp32 (or integers); with ``own`` true through the library's entry
points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

POOL_HEADER = 4   # int32 words ahead of a pool's list: free blocks, then zeros


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's short prompt: latency counts
        dict(name="prompt_one", op="prompt", batch=1, lo=217, hi=217, q_heads=32, kv_heads=8, dim=128, causal=True,
             out="bf16", lens_seed=1),
        # a prefill batch of uneven prompts
        dict(name="prompt_packed", op="prompt", batch=16, lo=256, hi=4096, q_heads=32, kv_heads=8, dim=128,
             causal=True, out="bf16", lens_seed=2),
        # one long document: arithmetic alone
        dict(name="prompt_long", op="prompt", batch=1, lo=32768, hi=32768, q_heads=32, kv_heads=8, dim=128,
             causal=True, out="bf16", lens_seed=3),
        # small heads without grouping, odd lengths from one token on
        dict(name="prompt_odd", op="prompt", batch=9, lo=1, hi=1500, q_heads=12, kv_heads=12, dim=64, causal=True,
             out="f32", lens_seed=4),
        # one user's draft tree
        dict(name="tree_one", op="tree", kv="bf16", batch=1, lo=777, hi=777, nodes=26, q_heads=32, kv_heads=8, dim=128,
             block=16, lens_seed=5),
        # a decode batch with small trees, the llama8b-shaped batch
        dict(name="tree_batch", op="tree", kv="bf16", batch=64, lo=3584, hi=4096, nodes=16, q_heads=32, kv_heads=8,
             dim=128, block=16, lens_seed=6),
        # a ragged batch over an FP8 cache
        dict(name="tree_ragged_fp8", op="tree", kv="fp8", batch=64, lo=1024, hi=65536, nodes=32, q_heads=32,
             kv_heads=8, dim=128, block=32, lens_seed=7),
        # few requests, wide trees, wide groups: as much arithmetic as memory traffic
        dict(name="tree_wide", op="tree", kv="bf16", batch=8, lo=2048, hi=16384, nodes=61, q_heads=64, kv_heads=8,
             dim=128, block=16, lens_seed=8),
        # one user's accepted path in one layer: latency
        dict(name="accept_one", op="accept", batch=1, lo=777, hi=777, nodes=26, row=2048, layers=1, block=16,
             lens_seed=9),
        # a batch's accepted paths in eight layers
        dict(name="accept_batch", op="accept", batch=64, lo=256, hi=1024, nodes=61, row=2048, layers=8, block=16,
             lens_seed=10),
        # a decode batch's new tokens: tables, one row a request, blocks back
        dict(name="grow_decode", op="grow", kv="bf16", batch=64, lo=3584, hi=4096, new_lo=1, new_hi=1, kv_heads=8,
             dim=128, block=16, lens_seed=11),
        # prompts entering an FP8 cache, some behind a cached prefix
        dict(name="grow_prompt_fp8", op="grow", kv="fp8", batch=33, lo=0, hi=2048, new_lo=16, new_hi=8192, kv_heads=8,
             dim=128, block=32, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    kind = rng.choice(["prompt", "prompt", "tree", "tree", "accept", "grow"])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    block = rng.choice([16, 32])
    if kind == "prompt":
        hi = _log_int(rng, 2, 16384)
        batch = _log_int(rng, 1, max(1, min(64, 65536 // hi)))
        return dict(op="prompt", batch=batch, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, causal=rng.choice([True, True, True, False]),
                    out=rng.choice(["bf16", "bf16", "f32"]), lens_seed=seed)
    if kind == "tree":
        nodes = _log_int(rng, 1, 256)
        hi = nodes + _log_int(rng, 1, 65536)
        batch = _log_int(rng, 1, max(1, min(64, 900000 // hi, 400000000 // (hi * nodes))))
        return dict(op="tree", kv=rng.choice(["bf16", "fp8"]), batch=batch, lo=max(nodes, hi // rng.choice([1, 2, 8])),
                    hi=hi, nodes=nodes, q_heads=q_heads, kv_heads=kv_heads, dim=dim, block=block, lens_seed=seed)
    if kind == "accept":
        nodes = _log_int(rng, 1, 256)
        hi = nodes + _log_int(rng, 1, 2048)
        return dict(op="accept", batch=_log_int(rng, 1, 64), lo=max(nodes, hi // 2), hi=hi, nodes=nodes,
                    row=rng.choice([256, 1024, 1152, 2048]), layers=rng.choice([1, 2, 5]), block=block, lens_seed=seed)
    new_hi = _log_int(rng, 1, 8192)
    return dict(op="grow", kv=rng.choice(["bf16", "fp8"]), batch=_log_int(rng, 1, max(1, min(256, 262144 // new_hi))),
                lo=0, hi=_log_int(rng, 1, 1024), new_lo=max(1, new_hi // rng.choice([1, 4, 64])), new_hi=new_hi,
                kv_heads=kv_heads, dim=dim, block=block, lens_seed=seed)


def _spread(rng, lo, hi, n):
    """n lengths: uniform where the range is narrow, else over the logarithm."""
    if lo == hi:
        return np.full(n, lo, np.int64)
    if hi <= 4 * lo:
        return rng.integers(lo, hi + 1, n)
    x = np.exp(rng.uniform(math.log(max(lo, 0.5)), math.log(hi), n))
    return np.clip(np.rint(x), lo, hi).astype(np.int64)


def _lens(case):
    return _spread(np.random.Generator(np.random.PCG64(case["lens_seed"])), case["lo"], case["hi"], case["batch"])


def _new(case):
    """Rows each request gains in a grow case."""
    rng = np.random.Generator(np.random.PCG64([case["lens_seed"], 1]))
    return _spread(rng, case["new_lo"], case["new_hi"], case["batch"])


def _trees(case):
    """Parents [batch, nodes] of drafted trees: node 0 is the root, wide at first, chains below."""
    rng = np.random.Generator(np.random.PCG64([case["lens_seed"], 2]))
    B, C = case["batch"], case["nodes"]
    parents = np.full((B, C), -1, np.int32)
    for j in range(1, C):
        back = np.minimum(j, rng.geometric(0.15, B))      # among the last few nodes
        parents[:, j] = j - back
    return parents


def _depths(parents):
    depth = np.zeros(parents.shape, np.int64)
    for j in range(1, parents.shape[1]):
        depth[:, j] = np.take_along_axis(depth, parents[:, j:j + 1].astype(np.int64), 1)[:, 0] + 1
    return depth


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _tables(case, lens, gen):
    """Blocks of the pool in random order, as a running server leaves them; a few spare."""
    bs = case["block"]
    need = (lens + bs - 1) // bs
    pool = int(need.sum()) + 5
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    n = torch.from_numpy(need).cuda()
    col = torch.arange(max(1, int(need.max())), device="cuda")
    first = torch.cumsum(n, 0) - n
    idx = (first[:, None] + col[None, :]).clamp_max(pool - 1)
    table = torch.where(col[None, :] < n[:, None], perm[idx], torch.full_like(perm[idx], -1))
    return table.contiguous(), pool


def _normal(shape, gen, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    return {"prompt": _prepare_prompt, "tree": _prepare_tree, "accept": _prepare_accept, "grow": _prepare_grow}[
        case["op"]](dict(case=case), case, gen)


def _prepare_prompt(st, case, gen):
    lens = _lens(case)
    T, Hq, Hkv, D = int(lens.sum()), case["q_heads"], case["kv_heads"], case["dim"]
    # one projection's output: a token's queries, keys and values side by side
    st["qkv"] = _normal((T, Hq + 2 * Hkv, D), gen)
    st["qkv"][:, :Hq] *= 1.5
    st["start"] = _int32(_starts(lens))
    st["scale"] = D ** -0.5
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    st["out"] = torch.empty((T, Hq, D), dtype=dtype, device="cuda")
    st["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    return st


def _prepare_tree(st, case, gen):
    lens = _lens(case)
    B, C, Hq, Hkv, D = (case[k] for k in ("batch", "nodes", "q_heads", "kv_heads", "dim"))
    st["table"], pool = _tables(case, lens, gen)
    st["ctx"], st["max_ctx"] = _int32(lens), int(lens.max())
    st["parents"] = _int32(_trees(case).reshape(-1))
    st["start"] = torch.arange(0, B * C + 1, C, dtype=torch.int32, device="cuda")
    st["scale"] = D ** -0.5
    for n in ("k", "v"):
        st[n] = _normal((pool, case["block"], Hkv, D), gen)
        if case["kv"] == "fp8":
            st[n + "_scale"] = torch.tensor([2.0 ** -(4 + h % 3) for h in range(Hkv)], dtype=torch.float32,
                                            device="cuda")
            st[n] = (st[n] / st[n + "_scale"][:, None]).to(torch.float8_e4m3fn)
    st["q"] = _normal((B * C, Hq, D), gen, scale=1.5)
    st["out"] = torch.empty((B * C, Hq, D), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((B * C, Hq), dtype=torch.float32, device="cuda")
    if own:
        from paged_kv_decode_kf_gb300 import kf
        st["ws"] = kf.make_tree_workspace(B, C, Hq, Hkv, D)
    return st


def _prepare_accept(st, case, gen):
    lens = _lens(case)
    B, C = case["batch"], case["nodes"]
    st["table"], pool = _tables(case, lens, gen)
    st["ctx"] = _int32(lens)
    parents = _trees(case)
    st["depth"] = int(_depths(parents).max())
    st["parents"] = _int32(parents.reshape(-1))
    st["start"] = torch.arange(0, B * C + 1, C, dtype=torch.int32, device="cuda")
    # drafted tokens; the model agrees with a node's first child two times in three
    draft = torch.randint(0, 32000, (B, C), generator=gen, device="cuda", dtype=torch.int32)
    target = torch.randint(0, 32000, (B, C), generator=gen, device="cuda", dtype=torch.int32)
    agree = torch.rand((B, C), generator=gen, device="cuda") < 2 / 3
    child = np.zeros((B, C), np.int64)
    for j in range(C - 1, 0, -1):
        child[np.arange(B), parents[:, j]] = j
    child = torch.from_numpy(child).cuda()
    target = torch.where(agree & (child > 0), draft.gather(1, child), target)
    st["draft"], st["target"] = draft.reshape(-1).contiguous(), target.reshape(-1).contiguous()
    # a row is case["row"] bytes: keys or values of all heads
    st["caches"] = [_normal((pool, case["block"], case["row"] // 2), gen) for _ in range(2 * case["layers"])]
    st["path"] = torch.empty((B, C), dtype=torch.int32, device="cuda")
    st["accepted"], st["next"], st["ctx_out"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
    return st


def _prepare_grow(st, case, gen):
    bs, B = case["block"], case["batch"]
    before, new = _lens(case), _new(case)
    after = before + new
    need = (after + bs - 1) // bs
    held = (before + bs - 1) // bs
    blocks = int(need.sum()) + 7
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    # the cached prefixes' blocks, the rest free
    table = torch.full((B, int(need.max())), -1, dtype=torch.int32, device="cuda")
    n = torch.from_numpy(held).cuda()
    mine = torch.arange(table.shape[1], device="cuda")[None, :] < n[:, None]
    table[mine] = perm[:int(held.sum())]
    free = perm[int(held.sum()):]
    st["pool"] = torch.zeros(POOL_HEADER + blocks, dtype=torch.int32, device="cuda")
    st["pool"][0] = free.numel()
    st["pool"][POOL_HEADER:POOL_HEADER + free.numel()] = free
    st["table"], st["before"], st["start"] = table, _int32(before), _int32(_starts(new))
    st["after"] = torch.empty(B, dtype=torch.int32, device="cuda")
    N, H, D = int(new.sum()), case["kv_heads"], case["dim"]
    st["slots"] = torch.empty(N, dtype=torch.int64, device="cuda")
    st["positions"] = torch.empty(N, dtype=torch.int32, device="cuda")
    for n in ("k", "v"):
        st[n + "_rows"] = _normal((N, H, D), gen)
        st[n] = torch.zeros((blocks, bs, H, D), dtype=torch.bfloat16, device="cuda")
        if case["kv"] == "fp8":
            st[n] = st[n].to(torch.float8_e4m3fn)
            st[n + "_scale"] = torch.tensor([2.0 ** -(4 + h % 3) for h in range(H)], dtype=torch.float32,
                                            device="cuda")
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return {"prompt": _run_prompt, "tree": _run_tree, "accept": _run_accept, "grow": _run_grow}[state["case"]["op"]](
        state)


def _attend(q, k, v, seen, scale):
    """q [n, Hq, D], k and v [m, Hkv, D] in fp32, seen [n, m] or None -> out [n, Hq, D], lse [n, Hq]."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    qg = q.view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
    s = torch.matmul(qg, k.permute(1, 2, 0)).mul_(scale).view(Hkv, G, n, m)
    if seen is not None:
        s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(Hkv, G * n, m), v.transpose(0, 1)).view(Hkv, G, n, D) / total
    lse = (top + torch.log(total))[..., 0]
    return o.permute(2, 0, 1, 3).reshape(n, Hq, D), lse.permute(2, 0, 1).reshape(n, Hq)


def _run_prompt(st):
    case = st["case"]
    lens = _lens(case)
    Hq, Hkv = case["q_heads"], case["kv_heads"]
    q, k, v = st["qkv"].split([Hq, Hkv, Hkv], 1)
    if own:
        from paged_kv_decode_kf_gb300 import kf
        kf.kf_prompt_attention(q, k, v, st["start"], int(lens.max()), st["scale"], causal=case["causal"],
                               out=st["out"], lse_out=st["lse"])
        return st["out"], st["lse"]
    at = 0
    for L in lens.tolist():
        kf32, vf32 = k[at:at + L].float(), v[at:at + L].float()
        for i in range(0, L, 2048):
            n = min(2048, L - i)
            m = i + n if case["causal"] else L
            seen = None
            if case["causal"]:
                seen = torch.arange(m, device="cuda")[None, :] <= torch.arange(i, i + n, device="cuda")[:, None]
            o, lse = _attend(q[at + i:at + i + n].float(), kf32[:m], vf32[:m], seen, st["scale"])
            st["out"][at + i:at + i + n] = o
            st["lse"][at + i:at + i + n] = lse
        at += L
    return st["out"], st["lse"]


def _rows_of(cache, table, b, L):
    """Rows of request b's first L tokens in order."""
    bs = cache.shape[1]
    n = -(-L // bs)
    return cache[table[b, :n].long()].reshape((n * bs,) + tuple(cache.shape[2:]))[:L]


def _ancestors(parents):
    """[B, C, C]: true where node j is node i or an ancestor of it."""
    B, C = parents.shape
    seen = torch.eye(C, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    hop = torch.where(parents < 0, C, parents).long()            # C: above the root
    reach = hop
    for _ in range(C):
        hit = torch.zeros((B, C, C + 1), dtype=torch.bool, device="cuda").scatter_(2, reach[..., None], True)
        if not bool(hit[..., :C].any()):
            break
        seen |= hit[..., :C]
        up = torch.cat([hop, torch.full((B, 1), C, dtype=torch.long, device="cuda")], 1)
        reach = up.gather(1, reach)
    return seen


def _run_tree(st):
    case = st["case"]
    B, C, Hq, Hkv, D = (case[k] for k in ("batch", "nodes", "q_heads", "kv_heads", "dim"))
    if own:
        from paged_kv_decode_kf_gb300 import kf
        if case["kv"] == "fp8":
            kf.kf_tree_attention_fp8(st["q"], st["parents"], st["k"], st["v"], st["k_scale"], st["v_scale"],
                                     st["table"], st["ctx"], st["max_ctx"], st["scale"], st["ws"],
                                     q_start=st["start"], max_query_len=C, out=st["out"], lse_out=st["lse"])
        else:
            kf.kf_tree_attention(st["q"], st["parents"], st["k"], st["v"], st["table"], st["ctx"], st["max_ctx"],
                                 st["scale"], st["ws"], q_start=st["start"], max_query_len=C, out=st["out"],
                                 lse_out=st["lse"])
        return st["out"], st["lse"]
    lens = _lens(case)
    anc = _ancestors(st["parents"].view(B, C))
    for b in range(B):
        L = int(lens[b])
        k, v = (_rows_of(st[n], st["table"], b, L).float() for n in ("k", "v"))
        if case["kv"] == "fp8":
            k, v = k * st["k_scale"][:, None], v * st["v_scale"][:, None]
        seen = torch.cat([torch.ones((C, L - C), dtype=torch.bool, device="cuda"), anc[b]], 1)
        o, lse = _attend(st["q"][b * C:(b + 1) * C].float(), k, v, seen, st["scale"])
        st["out"][b * C:(b + 1) * C] = o
        st["lse"][b * C:(b + 1) * C] = lse
    return st["out"], st["lse"]


def _run_accept(st):
    case = st["case"]
    B, C, bs = case["batch"], case["nodes"], case["block"]
    out = dict(path=st["path"], accepted=st["accepted"], next=st["next"], ctx=st["ctx_out"])
    for i, cache in enumerate(st["caches"]):
        out["cache%d" % i] = cache
    if own:
        from paged_kv_decode_kf_gb300 import kf
        kf.kf_accept_tree(st["parents"], st["draft"], st["target"], st["start"], st["ctx"], C, st["path"],
                          st["accepted"], st["next"], st["ctx_out"])
        for i in range(0, len(st["caches"]), 2):
            kf.kf_commit_tree(st["caches"][i:i + 2], st["table"], st["ctx"], st["start"], st["path"], st["accepted"])
        return out
    parents, draft, target = (st[n].view(B, C).long() for n in ("parents", "draft", "target"))
    node = torch.arange(C, device="cuda").expand(B, C)
    path = torch.full((B, C), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    cur = torch.zeros((B, 1), dtype=torch.int64, device="cuda")
    going = torch.ones((B, 1), dtype=torch.bool, device="cuda")
    count = torch.ones((B, 1), dtype=torch.int64, device="cuda")
    for d in range(1, st["depth"] + 1):
        fits = (parents == cur) & (draft == target.gather(1, cur)) & (node > 0) & going
        child = torch.where(fits, node, C).amin(1, keepdim=True)
        going = child < C
        cur = torch.where(going, child, cur)
        path[:, d:d + 1] = torch.where(going, child, path[:, d:d + 1])
        count += going
    st["path"].copy_(path)
    st["accepted"].copy_(count[:, 0])
    st["next"].copy_(target.gather(1, cur)[:, 0])
    first = st["ctx"].long()[:, None] - C
    st["ctx_out"].copy_((first + count)[:, 0])
    b, i = torch.nonzero(node < count, as_tuple=True)
    src = first[b, 0] + path[b, i]
    dst = first[b, 0] + i
    at_s = st["table"][b, src // bs].long() * bs + src % bs
    at_d = st["table"][b, dst // bs].long() * bs + dst % bs
    for cache in st["caches"]:
        flat = cache.flatten(0, 1)
        flat[at_d] = flat[at_s]
    return out


def _run_grow(st):
    case = st["case"]
    bs = case["block"]
    out = {n: st[n] for n in ("slots", "positions", "after", "k", "v", "table", "pool")}
    if case["kv"] == "fp8":   # what the codes stand for
        out.update(k=st["k"].view(torch.uint8), v=st["v"].view(torch.uint8))
    if own:
        from paged_kv_decode_kf_gb300 import kf
        kf.kf_extend_block_tables(st["pool"], st["table"], st["before"], bs, st["after"], st["slots"],
                                  row_start=st["start"], positions=st["positions"])
        if case["kv"] == "fp8":
            kf.kf_append_rows_fp8(st["k_rows"], st["v_rows"], st["k"], st["v"], st["k_scale"], st["v_scale"],
                                  st["slots"])
        else:
            kf.kf_append_rows(st["k_rows"], st["v_rows"], st["k"], st["v"], st["slots"])
        # (and back, as when the requests are withdrawn: the next pass finds the same pool)
        kf.kf_release_blocks(st["pool"], st["table"], st["after"], bs, context_lens_after=st["before"])
        return out
    N = st["slots"].numel()
    start, before = st["start"].long(), st["before"].long()
    after = before + start[1:] - start[:-1]
    held, need = (before + bs - 1) // bs, (after + bs - 1) // bs
    total = torch.cumsum(need - held, 0)
    free = st["pool"][0].long()
    row = torch.arange(N, device="cuda")
    b = torch.searchsorted(start[1:], row, right=True)
    pos = before[b] + row - start[b]
    lb = pos // bs
    fresh = lb >= held[b]
    pop = free - 1 - (total[b] - need[b] + lb)
    phys = torch.where(fresh, st["pool"][POOL_HEADER + pop.clamp_min(0)], st["table"][b, lb]).long()
    st["slots"].copy_(phys * bs + pos % bs)
    st["positions"].copy_(pos)
    st["after"].copy_(after)
    first = torch.nonzero(fresh & (pos % bs == 0))[:, 0]
    st["table"][b[first], lb[first]] = phys[first].to(torch.int32)
    st["pool"][0] -= total[-1].to(torch.int32)
    for n in ("k", "v"):
        rows = st[n + "_rows"]
        if case["kv"] == "fp8":
            rows = (rows.float() / st[n + "_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            st[n].view(torch.uint8).flatten(0, 1)[st["slots"]] = rows.view(torch.uint8)
        else:
            st[n].flatten(0, 1)[st["slots"]] = rows
    # back to the pool, the last taken first
    col = torch.arange(st["table"].shape[1], device="cuda")[None, :]
    gone = (col >= held[:, None]) & (col < need[:, None])
    blocks = st["table"][gone]
    count = st["pool"][0].long()
    place = count + blocks.numel() - 1 - torch.arange(blocks.numel(), device="cuda")
    st["pool"][POOL_HEADER + place] = blocks
    st["pool"][0] += blocks.numel()
    st["table"][gone] = -1
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    lens = _lens(case).astype(np.float64)
    if case["op"] == "prompt":
        T, Hq, Hkv, D = lens.sum(), case["q_heads"], case["kv_heads"], case["dim"]
        pairs = (lens * (lens + 1) / 2).sum() if case["causal"] else (lens * lens).sum()
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": float(T * ((Hq + 2 * Hkv) * D * 2 + Hq * (D * size + 4))), "flops": float(4 * D * Hq * pairs)}
    if case["op"] == "tree":
        B, C, Hq, Hkv, D = (case[k] for k in ("batch", "nodes", "q_heads", "kv_heads", "dim"))
        depth = _depths(_trees(case)) + 1                        # nodes a node sees, itself among them
        pairs = float(((lens - C) * C).sum() + depth.sum())
        size = 1 if case["kv"] == "fp8" else 2
        return {"bytes": float(lens.sum() * Hkv * D * 2 * size + B * C * (Hq * (D * 4 + 4) + 4)),
                "flops": 4 * D * Hq * pairs}
    if case["op"] == "accept":
        # about three nodes of a request are accepted, the root of them in place already
        B, C = case["batch"], case["nodes"]
        moved = 2.0 * B if C > 2 else 0.0
        return {"bytes": B * C * 16.0 + B * 16 + moved * 2 * case["row"] * 2 * case["layers"], "flops": float(B * C)}
    rows = float(_new(case).sum())
    size = 1 if case["kv"] == "fp8" else 2
    blocks = rows / case["block"]
    data = rows * (case["kv_heads"] * case["dim"] * 2 * (2 + size) + 12) + blocks * 4 * 4 + case["batch"] * 16
    return {"bytes": data, "flops": rows * (case["kv_heads"] * case["dim"] * 2 if size == 1 else 4)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("prompt", "tree") and work(case)["flops"] > 4e12:   # fp64 products run at about a TFLOP/s
        return None
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "tree": _exact_tree, "accept": _exact_accept, "grow": _exact_grow}[case["op"]](
        case, st)


def _exact_prompt(case, st):
    """Head by head, sequence by sequence."""
    lens = _lens(case)
    Hq, Hkv = case["q_heads"], case["kv_heads"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    ends = np.cumsum(lens)
    for L, end in zip(lens.tolist(), ends.tolist()):
        x = st["qkv"][end - L:end].double()
        future = torch.ones((L, L), dtype=torch.bool, device="cuda").triu(1) if case["causal"] else None
        for h in range(Hq):
            g = Hq + h * Hkv // Hq
            s = x[:, h] @ x[:, g].t() * st["scale"]
            if future is not None:
                s = torch.where(future, torch.full_like(s, -math.inf), s)
            lse[end - L:end, h] = torch.logsumexp(s, 1)
            out[end - L:end, h] = torch.softmax(s, 1) @ x[:, g + Hkv]
    return out, lse


def _exact_tree(case, st):
    """Head by head; a node's ancestors by walking up the parents on the host."""
    B, C, Hq, Hkv = (case[k] for k in ("batch", "nodes", "q_heads", "kv_heads"))
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    parents = st["parents"].cpu().numpy().reshape(B, C)
    for b, L in enumerate(_lens(case).tolist()):
        hidden = np.zeros((C, L), bool)
        hidden[:, L - C:] = True
        for i in range(C):
            j = i
            while j >= 0:
                hidden[i, L - C + j] = False
                j = int(parents[b, j])
        hidden = torch.from_numpy(hidden).cuda()
        keys, values = (_rows_of(st[n], st["table"], b, L).double() for n in ("k", "v"))
        for h in range(Hq):
            g = h * Hkv // Hq
            k, v = keys[:, g], values[:, g]
            if case["kv"] == "fp8":
                k, v = k * st["k_scale"][g].double(), v * st["v_scale"][g].double()
            s = st["q"][b * C:(b + 1) * C, h].double() @ k.t() * st["scale"]
            s = torch.where(hidden, torch.full_like(s, -math.inf), s)
            lse[b * C:(b + 1) * C, h] = torch.logsumexp(s, 1)
            out[b * C:(b + 1) * C, h] = torch.softmax(s, 1) @ v
    return out, lse


def _exact_accept(case, st):
    """The walk on the host, then row by row."""
    B, C, bs = case["batch"], case["nodes"], case["block"]
    parents, draft, target = (st[n].cpu().numpy().reshape(B, C) for n in ("parents", "draft", "target"))
    table = st["table"].cpu().numpy().astype(np.int64)
    path = np.full((B, C), -1, np.int32)
    accepted, last, ctx = (np.zeros(B, np.int32) for _ in range(3))
    dst, src = [], []
    for b, L in enumerate(_lens(case).tolist()):
        nodes = [0]
        while True:
            found = [c for c in range(1, C) if parents[b, c] == nodes[-1] and draft[b, c] == target[b, nodes[-1]]]
            if not found:
                break
            nodes.append(found[0])
        path[b, :len(nodes)] = nodes
        accepted[b], last[b], ctx[b] = len(nodes), target[b, nodes[-1]], L - C + len(nodes)
        for i, n in enumerate(nodes):
            for rows, t in ((dst, L - C + i), (src, L - C + n)):
                rows.append(table[b, t // bs] * bs + t % bs)
    out = dict(path=torch.from_numpy(path).cuda(), accepted=torch.from_numpy(accepted).cuda(),
               next=torch.from_numpy(last).cuda(), ctx=torch.from_numpy(ctx).cuda())
    d, s = torch.tensor(dst, device="cuda"), torch.tensor(src, device="cuda")
    for i, cache in enumerate(st["caches"]):
        flat = cache.view(-1, cache.shape[2]).clone()
        flat[d] = cache.view(-1, cache.shape[2])[s]
        out["cache%d" % i] = flat.view(cache.shape).double()
    return out


def _exact_grow(case, st):
    """Block by block on the host: pops, then the same blocks pushed back."""
    bs = case["block"]
    before, new = _lens(case), _new(case)
    pool = st["pool"].cpu().numpy()
    table = st["table"].cpu().numpy()
    free = pool[POOL_HEADER:POOL_HEADER + pool[0]].tolist()
    slots, positions = [], []
    for b in range(case["batch"]):
        blocks = table[b, :-(-int(before[b]) // bs)].tolist()
        for t in range(int(before[b]), int(before[b] + new[b])):
            if t // bs == len(blocks):
                blocks.append(free.pop())
            slots.append(blocks[t // bs] * bs + t % bs)
            positions.append(t)
    at = torch.tensor(slots, device="cuda")
    out = dict(slots=at, positions=_int32(np.array(positions)), after=_int32(before + new), table=st["table"],
               pool=st["pool"])
    for n in ("k", "v"):
        rows = st[n + "_rows"].double()
        flat = st[n].flatten(0, 1)
        if case["kv"] == "fp8":
            rows = rows / st[n + "_scale"].double()[:, None]
            flat.view(torch.uint8)[at] = rows.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            out[n] = st[n].view(torch.uint8)
        else:
            flat[at] = rows.to(torch.bfloat16)
            out[n] = st[n].double()
    return out
