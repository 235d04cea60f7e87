"""Cases of the latent-attention and cache-eviction operators.

Two groups, both over the library's paged cache (block tables, device context
lengths):

* latent attention: one shared row [c_t (R) ; k_rope_t (Dr)] a token; every
  head's key is [W_uk_h c_t ; k_rope_t] and its value W_uv_h c_t. The absorbed
  form (decode, verification of draft tokens) takes queries that hold W_uk
  already and attends to the latent rows themselves, with outputs in the latent
  space; the expanded form (prefill chunks) builds keys and values first.
* eviction: the attention weight each cached token receives is added up
  (`accumulate`), and the tokens with the least are dropped (`evict`).

With ``own`` false the operators are computed from elementary torch
operations in fp32; with ``own`` true through the library's entry points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

ROPE = 64  # rotary part of a latent row


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's first tokens after a short prompt, heads split over GPUs: latency counts
        dict(name="latent_decode_one", op="latent", form="absorbed", batch=1, lo=777, hi=777, heads=16,
             latent=512, nope=128, v=128, queries=1, block=16, lens_seed=1),
        # a full decode batch with every head on this GPU: as much arithmetic as memory traffic
        dict(name="latent_decode_batch", op="latent", form="absorbed", batch=64, lo=3584, hi=4096, heads=128,
             latent=512, nope=128, v=128, queries=1, block=16, lens_seed=2),
        # long agentic contexts of uneven lengths: memory traffic
        dict(name="latent_decode_long", op="latent", form="absorbed", batch=16, lo=8192, hi=262144, heads=32,
             latent=512, nope=128, v=128, queries=1, block=32, lens_seed=3),
        # verification of 4 draft tokens a request, smaller latent
        dict(name="latent_verify", op="latent", form="absorbed", batch=48, lo=3584, hi=4096, heads=20,
             latent=256, nope=64, v=64, queries=4, block=16, lens_seed=4),
        # chunked prefill: 1024 new tokens a request behind 3K-11K cached ones
        dict(name="latent_prefill_chunk", op="latent", form="expanded", batch=4, lo=4096, hi=12288, heads=32,
             latent=512, nope=128, v=128, queries=1024, block=16, lens_seed=5),
        # a few whole prompts of odd lengths (every token a query), smaller latent
        dict(name="latent_prefill_odd", op="latent", form="expanded", batch=3, lo=601, hi=601, heads=12,
             latent=256, nope=64, v=64, queries=601, block=32, lens_seed=6),
        # the weights of one decode step, the llama8b-shaped batch
        dict(name="accumulate_decode", op="accumulate", kv="bf16", batch=64, lo=3584, hi=4096, q_heads=32,
             kv_heads=8, dim=128, queries=1, block=16, lens_seed=7),
        # the same over an FP8 cache and a ragged batch
        dict(name="accumulate_ragged_fp8", op="accumulate", kv="fp8", batch=64, lo=1024, hi=65536, q_heads=32,
             kv_heads=8, dim=128, queries=1, block=32, lens_seed=8),
        # after a prompt: the weights its last 32 queries give
        dict(name="accumulate_window", op="accumulate", kv="bf16", batch=4, lo=4096, hi=12288, q_heads=32,
             kv_heads=8, dim=128, queries=32, block=16, lens_seed=9),
        # the steady state of a bounded cache: one token over the budget in every request
        dict(name="evict_one", op="evict", batch=64, lo=2049, hi=2049, keep=2048, sink=4, recent=256, row=2048,
             caches=2, positions=True, block=16, lens_seed=10),
        # long prompts cut to an eighth
        dict(name="evict_prompt", op="evict", batch=8, lo=65536, hi=131072, keep=12289, sink=4, recent=1024,
             row=2048, caches=2, positions=False, block=32, lens_seed=11),
        # a ragged batch of latent caches, some below the budget
        dict(name="evict_latent", op="evict", batch=33, lo=1024, hi=8192, keep=2500, sink=0, recent=64, row=1152,
             caches=1, positions=True, block=16, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    kind = rng.choice(["decode", "decode", "prefill", "accumulate", "window", "evict"])
    block = rng.choice([16, 32])
    if kind == "decode":
        heads = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 96, 128])
        queries = rng.choice([1, 1, 1, 2, 3, 5, 8])
        hi = _log_int(rng, 1 + queries, 131072)
        batch = _log_int(rng, 1, max(1, min(96, int(1.0e6 * 128 / (hi * heads * queries)), 1500000 // hi)))
        latent, small = rng.choice([(512, 128), (512, 128), (256, 64)])
        return dict(op="latent", form="absorbed", batch=batch, lo=max(queries, hi // rng.choice([1, 2, 8])), hi=hi,
                    heads=heads, latent=latent, nope=small, v=small, queries=queries, block=block, lens_seed=seed)
    if kind == "prefill":
        heads = rng.choice([1, 4, 12, 16, 20, 32])
        queries = _log_int(rng, 17, 1024)
        hi = queries + _log_int(rng, 1, 8192)
        batch = rng.choice([1, 2, 3])
        latent, small = rng.choice([(512, 128), (256, 64)])
        return dict(op="latent", form="expanded", batch=batch, lo=queries, hi=hi, heads=heads, latent=latent,
                    nope=small, v=small, queries=queries, block=block, lens_seed=seed)
    if kind in ("accumulate", "window"):
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 4, 8])
        queries = 1 if kind == "accumulate" else _log_int(rng, 2, 64)
        hi = queries + _log_int(rng, 1, 65536 if queries == 1 else 8192)
        batch = _log_int(rng, 1, max(1, min(64, 30000000 // (hi * queries * q_heads), 900000 // hi)))
        return dict(op="accumulate", kv=rng.choice(["bf16", "fp8"]), batch=batch,
                    lo=max(queries, hi // rng.choice([1, 2, 8])), hi=hi, q_heads=q_heads,
                    kv_heads=kv_heads, dim=rng.choice([64, 128]), queries=queries, block=block, lens_seed=seed)
    hi = _log_int(rng, 33, 131072)
    keep = max(2, int(hi * rng.uniform(0.05, 1.0)))
    return dict(op="evict", batch=_log_int(rng, 1, max(1, min(64, 700000 // hi))), lo=max(1, hi // rng.choice([1, 2, 8])),
                hi=hi, keep=keep, sink=rng.choice([0, min(4, keep // 4)]), recent=rng.randrange(0, keep // 2 + 1),
                row=rng.choice([256, 1024, 1152, 2048]), caches=rng.choice([1, 2]), positions=rng.choice([True, False]),
                block=block, lens_seed=seed)


def _lens(case):
    """Tokens per request: uniform where the range is narrow, else over the logarithm."""
    rng = np.random.Generator(np.random.PCG64(case["lens_seed"]))
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    if lo == hi:
        return np.full(n, lo, np.int64)
    if hi <= 4 * lo:
        return rng.integers(lo, hi + 1, n)
    return np.clip(np.rint(np.exp(rng.uniform(math.log(lo), math.log(hi), n))), lo, hi).astype(np.int64)


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
    col = torch.arange(int(need.max()), device="cuda")
    first = torch.cumsum(n, 0) - n
    idx = (first[:, None] + col[None, :]).clamp_max(pool - 1)
    table = torch.where(col[None, :] < n[:, None], perm[idx], torch.full_like(perm[idx], -1))
    return table.contiguous(), pool


def _normal(shape, gen, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    lens = _lens(case)
    table, pool = _tables(case, lens, gen)
    st = dict(case=case, table=table, ctx=torch.from_numpy(lens.astype(np.int32)).cuda(), max_ctx=int(lens.max()))
    return {"latent": _prepare_latent, "accumulate": _prepare_accumulate, "evict": _prepare_evict}[case["op"]](
        st, case, lens, pool, gen)


def _prepare_latent(st, case, lens, pool, gen):
    B, C, H, R, Dn, Dv = (case[k] for k in ("batch", "queries", "heads", "latent", "nope", "v"))
    st["cache"] = _normal((pool, case["block"], R + ROPE), gen)     # normed latents, rotated keys
    if case["form"] == "absorbed":   # W_uk^T q has sqrt(Dn / R) of q's spread
        st["q"] = _normal((B * C, H, R + ROPE), gen, scale=2.0)
        st["q"][..., :R] *= (Dn / R) ** 0.5
    else:
        st["q"] = _normal((B * C, H, Dn + ROPE), gen, scale=2.0)
        st["w_uk"] = _normal((H, Dn, R), gen, scale=R ** -0.5)
        st["w_uv"] = _normal((H, Dv, R), gen, scale=R ** -0.5)
    st["new"] = _normal((B * C, R + ROPE), gen)                     # the rows this pass appends
    st["scale"] = (Dn + ROPE) ** -0.5
    st["before"] = torch.from_numpy((lens - C).astype(np.int32)).cuda()
    st["start"] = torch.arange(0, B * C + 1, C, dtype=torch.int32, device="cuda")
    st["out"] = torch.empty((B * C, H, R if case["form"] == "absorbed" else Dv), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((B * C, H), dtype=torch.float32, device="cuda")
    if own:
        from paged_kv_decode_kf_gb300 import kf
        if case["form"] == "absorbed":
            st["ws"] = kf.make_latent_workspace(B, C, H, R)
        else:
            st["ws"] = kf.make_latent_expanded_workspace(B, B * C, st["max_ctx"], H, Dn, Dv)
    return st


def _prepare_accumulate(st, case, lens, pool, gen):
    B, C, Hq, Hkv, D = (case[k] for k in ("batch", "queries", "q_heads", "kv_heads", "dim"))
    st["k"] = _normal((pool, case["block"], Hkv, D), gen)
    st["scale"] = D ** -0.5
    if case["kv"] == "fp8":
        st["k_scale"] = torch.tensor([2.0 ** -(4 + h % 3) for h in range(Hkv)], dtype=torch.float32, device="cuda")
        st["k"] = (st["k"] / st["k_scale"][:, None]).to(torch.float8_e4m3fn)
    st["q"] = _normal((B * C, Hq, D), gen, scale=1.5)
    st["start"] = torch.arange(0, B * C + 1, C, dtype=torch.int32, device="cuda")
    st["scores"] = torch.rand((B, st["max_ctx"]), generator=gen, device="cuda")
    st["out"] = torch.zeros((B, st["max_ctx"]), device="cuda")
    # the log-sum-exp of each row, as the attention call before it returns it
    s, hidden = _scores(st)
    lse = torch.logsumexp(s.masked_fill_(hidden[:, None, None], -math.inf), -1)
    st["lse"] = lse.permute(0, 3, 1, 2).reshape(B * C, Hq).contiguous()
    return st


def _prepare_evict(st, case, lens, pool, gen):
    B, M = case["batch"], st["max_ctx"]
    # a row is case["row"] bytes: bf16 keys or values of all heads, or a latent row
    st["caches"] = [_normal((pool, case["block"], case["row"] // 2), gen) for _ in range(case["caches"])]
    # accumulated weights: most tokens little, a few much, some nothing at all
    s = torch.exp(torch.randn((B, M), generator=gen, device="cuda") * 1.5 - 4.0)
    st["scores"] = torch.where(torch.rand((B, M), generator=gen, device="cuda") < 0.05, torch.zeros_like(s), s)
    st["scores_out"] = torch.zeros((B, M), device="cuda")
    st["ctx_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if case["positions"]:
        # earlier evictions left gaps and a mixed order: positions are distinct, below the length seen
        pos = torch.argsort(torch.rand((B, 2 * M), generator=gen, device="cuda"), 1)[:, :M]
        st["positions"] = pos.to(torch.int32).contiguous()
        st["seen"] = torch.full((B,), 2 * M, dtype=torch.int32, device="cuda")
        st["positions_out"] = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    if own:
        from paged_kv_decode_kf_gb300 import kf
        st["ws"] = kf.make_evict_workspace(B, M, case["keep"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _slots(table, t, bs):
    """Row numbers of tokens t [B, n] in the pool seen as one list of rows (padding reads block 0)."""
    return table.gather(1, t // bs).clamp_min(0).long() * bs + t % bs


def _rows(cache, table, n):
    """The first n rows of every request, [B, n, ...]; those past a request's length are masked later."""
    t = torch.arange(n, device="cuda").expand(table.shape[0], n)
    return cache.flatten(0, 1)[_slots(table, t, cache.shape[1])]


def _hidden(ctx, C, n):
    """[B, C, n] true where query j of the last C tokens must not see token t (or there is none)."""
    j = torch.arange(C, device="cuda")[None, :, None]
    return torch.arange(n, device="cuda")[None, None, :] > ctx.long()[:, None, None] - C + j


def run(state):
    return {"latent": _run_latent, "accumulate": _run_accumulate, "evict": _run_evict}[state["case"]["op"]](state)


def _run_latent(st):
    case = st["case"]
    B, C, H, R, Dn, Dv = (case[k] for k in ("batch", "queries", "heads", "latent", "nope", "v"))
    if own:
        from paged_kv_decode_kf_gb300 import kf
        kf.kf_append_latent(st["new"], st["cache"], st["table"], st["before"], row_start=st["start"])
        if case["form"] == "absorbed":
            kf.kf_latent_attention(st["q"], st["cache"], st["table"], st["ctx"], st["max_ctx"], st["scale"], st["ws"],
                                   q_start=st["start"], max_query_len=C, causal=True, out=st["out"],
                                   lse_out=st["lse"])
        else:
            kf.kf_latent_attention_expanded(st["q"], st["cache"], st["w_uk"], st["w_uv"], st["table"], st["ctx"],
                                            st["max_ctx"], st["scale"], st["ws"], q_start=st["start"],
                                            max_query_len=C, causal=True, out=st["out"], lse_out=st["lse"])
        return st["out"], st["lse"]
    M, N = st["max_ctx"], R if case["form"] == "absorbed" else Dn
    t = st["before"].long()[:, None] + torch.arange(C, device="cuda")
    st["cache"].flatten(0, 1)[_slots(st["table"], t, case["block"]).flatten()] = st["new"]
    row = _rows(st["cache"], st["table"], M).float()                       # [B, M, R + 64]
    c, kr = row[..., :R], row[..., R:]
    q = st["q"].float().view(B, C, H, N + ROPE).transpose(1, 2)            # [B, H, C, N + 64]
    if case["form"] == "absorbed":
        s = torch.matmul(q.reshape(B, H * C, R + ROPE), row.transpose(1, 2)).view(B, H, C, M)
    else:
        s = torch.matmul(q[..., :N], torch.einsum("btr,hnr->bhnt", c, st["w_uk"].float()))
        s += torch.matmul(q[..., N:].reshape(B, H * C, ROPE), kr.transpose(1, 2)).view(B, H, C, M)
    s = s.mul_(st["scale"]).masked_fill_(_hidden(st["ctx"], C, M)[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    if case["form"] == "absorbed":
        o = torch.matmul(p.view(B, H * C, M), c).view(B, H, C, R)
    else:
        o = torch.matmul(p, torch.einsum("btr,hvr->bhtv", c, st["w_uv"].float()))
    o = (o / l).transpose(1, 2)
    st["out"].copy_(o.reshape(st["out"].shape))
    st["lse"].copy_((m + torch.log(l))[..., 0].transpose(1, 2).reshape(B * C, H))
    return st["out"], st["lse"]


def _scores(st):
    """Scaled scores [B, Hkv, G, C, M] in fp32 and the mask [B, C, M] of what is not seen."""
    case = st["case"]
    B, C, Hq, Hkv, D = (case[k] for k in ("batch", "queries", "q_heads", "kv_heads", "dim"))
    M = st["max_ctx"]
    k = _rows(st["k"], st["table"], M).float()
    if case["kv"] == "fp8":
        k = k.mul_(st["k_scale"][:, None])
    q = st["q"].float().view(B, C, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(st["scale"]).view(B, Hkv, Hq // Hkv, C, M)
    return s, _hidden(st["ctx"], C, M)


def _run_accumulate(st):
    case = st["case"]
    B, C, Hq, Hkv = (case[k] for k in ("batch", "queries", "q_heads", "kv_heads"))
    if own:
        from paged_kv_decode_kf_gb300 import kf
        extra = dict(q_start=st["start"], max_query_len=C) if C > 1 else {}
        if case["kv"] == "fp8":
            kf.kf_accumulate_attention_fp8(st["q"], st["k"], st["k_scale"], st["table"], st["ctx"], st["max_ctx"],
                                           st["scale"], st["lse"], st["out"], scores_in=st["scores"], **extra)
        else:
            kf.kf_accumulate_attention(st["q"], st["k"], st["table"], st["ctx"], st["max_ctx"], st["scale"],
                                       st["lse"], st["out"], scores_in=st["scores"], **extra)
        return st["out"]
    s, hidden = _scores(st)
    lse = st["lse"].view(B, C, Hkv, Hq // Hkv).permute(0, 2, 3, 1)
    w = s.sub_(lse[..., None]).exp_().masked_fill_(hidden[:, None, None], 0.0).sum((1, 2, 3))
    live = torch.arange(st["max_ctx"], device="cuda") < st["ctx"][:, None]
    st["out"].copy_(torch.where(live, st["scores"] + w, st["out"]))
    return st["out"]


def _run_evict(st):
    case = st["case"]
    keep, sink, recent, bs = case["keep"], case["sink"], case["recent"], case["block"]
    pos_on = case["positions"]
    if own:
        from paged_kv_decode_kf_gb300 import kf
        kf.kf_evict_tokens(st["caches"], st["table"], st["ctx"], st["max_ctx"], st["scores"], keep, sink, recent,
                           st["ctx_out"], st["scores_out"], st["ws"], positions=st.get("positions"),
                           seq_lens=st.get("seen"), positions_out=st.get("positions_out"))
    else:
        M = st["max_ctx"]
        K = min(keep, M)
        t = torch.arange(M, device="cuda").expand(case["batch"], M)
        L = st["ctx"].long()[:, None]
        live = t < L
        pos, seen = (st["positions"], st["seen"].long()[:, None]) if pos_on else (t, L)
        # protected first, then by weight, the lower index first among equals; padding last
        key = torch.where((pos < sink) | (pos >= seen - recent), math.inf, st["scores"])
        order = torch.argsort(torch.where(live, key, -math.inf), dim=1, descending=True, stable=True)
        kept = torch.zeros_like(live).scatter_(1, order[:, :K], True) & live
        # the holes below `keep` take the kept tokens above it, both in order
        dst = torch.nonzero(~kept[:, :K] & (L > keep))
        src = torch.nonzero(kept[:, K:])
        db, dt, st_ = dst[:, 0], dst[:, 1], src[:, 1] + K
        at_d = st["table"][db, dt // bs].long() * bs + dt % bs
        at_s = st["table"][db, st_ // bs].long() * bs + st_ % bs
        for cache in st["caches"]:
            flat = cache.flatten(0, 1)
            flat[at_d] = flat[at_s]
        idx = t[:, :K].clone()
        idx[db, dt] = st_
        fits = t[:, :K] < L
        st["scores_out"][:, :K] = torch.where(fits, st["scores"].gather(1, idx), st["scores_out"][:, :K])
        if pos_on:
            st["positions_out"][:, :K] = torch.where(fits, pos.gather(1, idx), st["positions_out"][:, :K])
        st["ctx_out"].copy_(st["ctx"].clamp_max(keep))
    out = dict(ctx=st["ctx_out"], scores=st["scores_out"])
    for i, cache in enumerate(st["caches"]):
        out["cache%d" % i] = cache
    if pos_on:
        out["positions"] = st["positions_out"]
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    lens = _lens(case)
    tokens = int(lens.sum())
    if case["op"] == "latent":
        B, C, H, R, Dn, Dv = (case[k] for k in ("batch", "queries", "heads", "latent", "nope", "v"))
        rows = B * C
        # (query, token) pairs under the causal mask
        pairs = float((lens * C).sum() - B * C * (C - 1) / 2)
        # the appended rows are read where they are given and written; attention may read them there too
        data = tokens * (R + ROPE) * 2 + rows * (R + ROPE) * 2
        if case["form"] == "absorbed":
            data += rows * H * ((2 * R + ROPE) * 2 + 4)
            flops = 2.0 * pairs * H * (2 * R + ROPE)
        else:
            data += rows * H * ((Dn + ROPE + Dv) * 2 + 4) + H * R * (Dn + Dv) * 2
            flops = 2.0 * pairs * H * (Dn + ROPE + Dv) + 2.0 * tokens * H * R * (Dn + Dv)
        return {"bytes": data, "flops": flops}
    if case["op"] == "accumulate":
        C, Hq, Hkv, D = (case[k] for k in ("queries", "q_heads", "kv_heads", "dim"))
        pairs = float((lens * C).sum() - case["batch"] * C * (C - 1) / 2)
        return {"bytes": tokens * (Hkv * D * (1 if case["kv"] == "fp8" else 2) + 8) + case["batch"] * C * Hq * (D * 2 + 4),
                "flops": 2.0 * pairs * Hq * D}
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    moved = 0.0
    for L in lens:
        if L > keep:
            free = max(1, L - sink - recent)
            share = max(0, keep - sink - recent) / free          # of the unprotected tokens, kept
            if case["positions"]:                                 # protected ones lie anywhere
                moved += (L - keep) * keep / L
            else:                                                 # the last `recent` ones lie at the end
                moved += min(recent, L - keep) + max(0, L - keep - recent) * share
    per = 4 * (2 if case["positions"] else 1)
    kept = float(np.minimum(lens, keep).sum())
    return {"bytes": tokens * per + kept * per + moved * 2 * case["row"] * case["caches"], "flops": float(tokens)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    lens = _lens(case)
    if case["op"] == "latent":
        # fp64 products run at about a TFLOP/s
        if work(case)["flops"] > 8e12:
            return None
        return _exact_latent(case, prepare(case, seed), lens)
    if case["op"] == "accumulate":
        return _exact_accumulate(case, prepare(case, seed), lens)
    return _exact_evict(case, prepare(case, seed), lens)


def _token_rows(cache, table, b, L):
    """Rows of request b's first L tokens in order, block by block."""
    bs = cache.shape[1]
    n = -(-L // bs)
    return cache[table[b, :n].long()].reshape((n * bs,) + tuple(cache.shape[2:]))[:L]


def _exact_latent(case, st, lens):
    """Head by head from the definition: keys and values of one head, then its softmax."""
    B, C, H, R, Dn = (case[k] for k in ("batch", "queries", "heads", "latent", "nope"))
    absorbed = case["form"] == "absorbed"
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((B * C, H), dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(lens[b])
        row = _token_rows(st["cache"], st["table"], b, L).double()
        row[L - C:] = st["new"][b * C:(b + 1) * C].double()
        last = torch.arange(C, device="cuda") + (L - C)           # the newest token query j sees
        seen = torch.arange(L, device="cuda")[None, :] <= last[:, None]
        for h in range(H):
            q = st["q"][b * C:(b + 1) * C, h].double()
            if absorbed:
                key, value = row, row[:, :R]
            else:
                key = torch.cat([row[:, :R] @ st["w_uk"][h].double().t(), row[:, R:]], 1)
                value = row[:, :R] @ st["w_uv"][h].double().t()
            s = q @ key.t() * st["scale"]
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            lse[b * C:(b + 1) * C, h] = torch.logsumexp(s, 1)
            out[b * C:(b + 1) * C, h] = torch.softmax(s, 1) @ value
    return out, lse


def _exact_accumulate(case, st, lens):
    C, Hq, Hkv, D = (case[k] for k in ("queries", "q_heads", "kv_heads", "dim"))
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        L = int(lens[b])
        k = _token_rows(st["k"], st["table"], b, L).double()
        if case["kv"] == "fp8":
            k = k * st["k_scale"].double()[None, :, None]
        last = torch.arange(C, device="cuda") + (L - C)
        seen = torch.arange(L, device="cuda")[:, None] <= last[None, :]
        total = st["scores"][b, :L].double()
        for h in range(Hq):
            s = k[:, h // (Hq // Hkv)] @ st["q"][b * C:(b + 1) * C, h].double().t() * st["scale"]
            w = torch.exp(s - st["lse"][b * C:(b + 1) * C, h].double()[None, :])
            total = total + torch.where(seen, w, torch.zeros_like(w)).sum(1)
        out[b, :L] = total
    return out


def _exact_evict(case, st, lens):
    """Ranks on the host: (protected first, larger score, lower index)."""
    keep, sink, recent, bs = case["keep"], case["sink"], case["recent"], case["block"]
    scores = st["scores"].double().cpu().numpy()
    out_s = np.zeros_like(scores)
    out_c = torch.zeros(case["batch"], dtype=torch.int32)
    pos_on = case["positions"]
    if pos_on:
        positions = st["positions"].cpu().numpy()
        out_p = np.zeros_like(positions)
        seen = st["seen"].cpu().numpy()
    table = st["table"].cpu().numpy().astype(np.int64)
    for b in range(case["batch"]):
        L = int(lens[b])
        n = min(L, keep)
        at = np.arange(n)
        if L > keep:
            pos = positions[b, :L].astype(np.int64) if pos_on else np.arange(L)
            end = int(seen[b]) if pos_on else L
            prot = (pos < sink) | (pos >= end - recent)
            rank = np.lexsort((np.arange(L), -scores[b, :L], ~prot))
            chosen = np.sort(rank[:keep])
            holes = np.setdiff1d(np.arange(keep), chosen)
            tails = chosen[chosen >= keep]
            at[holes] = tails
            d = torch.from_numpy(table[b, holes // bs] * bs + holes % bs).cuda()
            s = torch.from_numpy(table[b, tails // bs] * bs + tails % bs).cuda()
            for cache in st["caches"]:
                cache.view(-1, cache.shape[2]).index_copy_(0, d, cache.view(-1, cache.shape[2])[s])
        out_s[b, :n] = scores[b, at]
        out_c[b] = n
        if pos_on:
            out_p[b, :n] = positions[b, at]
    out = dict(ctx=out_c.cuda(), scores=torch.from_numpy(out_s).cuda())
    for i, cache in enumerate(st["caches"]):
        out["cache%d" % i] = cache.double()
    if pos_on:
        out["positions"] = torch.from_numpy(out_p).cuda()
    return out
