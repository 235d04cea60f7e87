"""Plain 64-bit implementations of the latent-attention and eviction calls, and
seeded inputs for their tests. numpy on the host; shares nothing with the CUDA
path but the layouts."""
from __future__ import annotations

import math

import numpy as np
import torch

ROPE = 64


def paged(lens, bs, width, gen, spare=3, extra_cols=1, dtype=torch.bfloat16):
    """A pool of random rows, tables in random order (-1 past a request's blocks)."""
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + spare
    perm = torch.randperm(nb, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(max(need, default=0), 1) + extra_cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    width = (width,) if isinstance(width, int) else tuple(width)
    return torch.randn((nb, bs) + width, generator=gen).to(dtype), table


def rows_of(cache, table, b, n):
    """Request b's first n rows, float64."""
    bs = cache.shape[1]
    out = [cache[int(table[b, t // bs]), t % bs].double() for t in range(n)]
    return torch.stack(out).numpy() if out else np.zeros((0,) + tuple(cache.shape[2:]))


def attention(q, keys, values, scale, visible):
    """q [H, KD], keys [H or 1, T, KD], values [H or 1, T, VD]: out [H, VD], lse [H],
    sum of weight x |value| [H, VD] and max over tokens of sum |q k| scale [H]."""
    H, T = q.shape[0], keys.shape[1]
    VD = values.shape[2]
    if visible <= 0 or T == 0:
        return np.zeros((H, VD)), np.full(H, -np.inf), np.zeros((H, VD)), np.zeros(H)
    k = np.broadcast_to(keys[:, :visible], (H, visible, keys.shape[2]))
    v = np.broadcast_to(values[:, :visible], (H, visible, VD))
    s = np.einsum("hd,htd->ht", q, k) * scale
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    l = w.sum(1, keepdims=True)
    p = w / l
    mag = (np.einsum("hd,htd->ht", np.abs(q), np.abs(k)) * abs(scale)).max(1)
    return (np.einsum("ht,htv->hv", p, v), (m + np.log(l))[:, 0], np.einsum("ht,htv->hv", p, np.abs(v)), mag)


def latent(q, q_start, cache, table, lens, scale, causal, w_uk=None, w_uv=None):
    """Reference outputs for every query row: out, lse, weight x |value|, max |q k|
    (rows that no request owns hold NaN)."""
    R = cache.shape[2] - ROPE
    nq, H, KD = q.shape
    VD = R if w_uv is None else w_uv.shape[1]
    out = np.full((nq, H, VD), np.nan)
    lse = np.full((nq, H), np.nan)
    mag_o = np.full((nq, H, VD), np.nan)
    mag_s = np.full((nq, H), np.nan)
    qd = q.double().numpy()
    for b, L in enumerate(lens):
        q0, q1 = int(q_start[b]), int(q_start[b + 1])
        row = rows_of(cache, table, b, int(L))
        if row.shape[0] == 0:
            row = np.zeros((0, R + ROPE))
        c, kr = row[:, :R], row[:, R:]
        if w_uk is None:
            keys, values = row[None], c[None]
        else:
            kn = np.einsum("hnr,tr->htn", w_uk.double().numpy(), c)
            keys = np.concatenate([kn, np.broadcast_to(kr[None], (H,) + kr.shape)], 2)
            values = np.einsum("hvr,tr->htv", w_uv.double().numpy(), c)
        for j in range(q1 - q0):
            seen = int(L) - (q1 - q0) + j + 1 if causal else int(L)
            r = attention(qd[q0 + j], keys, values, scale, seen)
            out[q0 + j], lse[q0 + j], mag_o[q0 + j], mag_s[q0 + j] = r
    return out, lse, mag_o, mag_s


def accumulate(q, q_start, k_cache, table, lens, scale, causal, lse, scores_in, stride, k_scale=None):
    """(scores [B, stride] with NaN where nothing is written, sum of the weights)."""
    nq, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    out = np.full((len(lens), stride), np.nan)
    add = np.zeros((len(lens), stride))
    qd, ld = q.double().numpy(), lse.double().numpy()
    for b, L in enumerate(lens):
        q0, q1 = int(q_start[b]), int(q_start[b + 1])
        k = rows_of(k_cache, table, b, int(L))
        if k_scale is not None:
            k = k * k_scale.double().numpy()[None, :, None]
        tot = np.zeros(int(L))
        for j in range(q1 - q0):
            seen = max(0, min(int(L), int(L) - (q1 - q0) + j + 1 if causal else int(L)))
            for h in range(Hq):
                if ld[q0 + j, h] == -np.inf or seen == 0:
                    continue
                tot[:seen] += np.exp(k[:seen, h // G] @ qd[q0 + j, h] * scale - ld[q0 + j, h])
        add[b, :int(L)] = tot
        out[b, :int(L)] = tot + (0.0 if scores_in is None else scores_in[b, :int(L)].double().numpy())
    return out, add


def evict(lens, scores, keep, sink, recent, positions=None, seq_lens=None):
    """Per request: (new length, source index of every kept slot)."""
    res = []
    for b, L in enumerate(lens):
        L = int(L)
        n = min(L, keep)
        at = np.arange(n)
        if L > keep:
            s = scores[b, :L].numpy().astype(np.float64)
            pos = np.arange(L) if positions is None else positions[b, :L].numpy().astype(np.int64)
            end = L if positions is None else int(seq_lens[b])
            rank = sorted(range(L), key=lambda t: (not (pos[t] < sink or pos[t] >= end - recent),
                                                   math.isnan(s[t]), -s[t] if not math.isnan(s[t]) else 0.0, t))
            kept = sorted(rank[:keep])
            chosen = set(kept)
            holes = [t for t in range(keep) if t not in chosen]
            movers = [t for t in kept if t >= keep]
            assert len(holes) == len(movers)
            at[holes] = movers
        res.append((n, at))
    return res
