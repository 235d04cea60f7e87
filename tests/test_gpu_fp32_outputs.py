"""What an fp32 output keeps: sums over long contexts, and the weights' last bits.

Bounds, all relative to sum p |v|; a unit is 2^-23.
Tensor cores cut their fp32 sum off at every step of 16 tokens, by a unit of the sum at most. Four
tiles of 128 tokens are 32 steps, of one product for every piece of the weights (bf16 caches three,
E4M3 two); the sum rises from nothing, so the steps' units are half as large as the last one on average
where all terms are alike, which these inputs see to (values in [1, 2], scores close together). Sums set aside
are added in fp32, half a unit a time, and the weights' own sum likewise: a tile's 128 in 32 additions
of two, then tile by tile. Parts of a run, joined by weights e^(lse - M): an lse is rounded to half a
unit of itself, |lse| <= 16 here, and a part's weight is off by as much, which moves the output by the
parts' difference (values' sums over thousands of tokens: 2 % of each other). Scores: 4 d half units of the
sum of their terms' sizes, twice (the row's and the sum's), as in prompt_tree_ref."""
import numpy as np
import pytest
import torch

import prompt_tree_ref as ref

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -23


@pytest.fixture(scope="module")
def kf():
    from paged_kv_decode_kf_gb300 import kf
    kf.kf_get_device_error()
    return kf


@pytest.mark.parametrize("d,nodes,hkv", [(64, 3, 4), (128, 3, 4), (128, 50, 2), (64, 64, 2)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_tree_sums_over_long_contexts(kf, d, nodes, hkv, fp8):
    """So many requests over one cached context of 40000 tokens that an SM walks a request from end
    to end; few rows (two streams of alternating tiles) and more than 128 (two query tiles)."""
    g = torch.Generator(device="cuda").manual_seed(31)
    L, bs, B, hq = 40000 + nodes, 32, 400 // hkv, 4 * hkv
    blocks = -(-L // bs)
    k = torch.randn((blocks, bs, hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    v = (torch.rand((blocks, bs, hkv, d), generator=g, device="cuda") + 1).to(torch.bfloat16)
    q = (torch.randn((B * nodes, hq, d), generator=g, device="cuda") * 0.01).to(torch.bfloat16)
    # (every request's last block, where its nodes are, could be its own; the same one will do: nothing is written)
    table = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).repeat(B, 1)
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda").repeat(B)
    ctx = torch.full((B,), L, dtype=torch.int32, device="cuda")
    start = torch.arange(0, B * nodes + 1, nodes, dtype=torch.int32, device="cuda")
    ws = kf.make_tree_workspace(B, nodes, hq, hkv, d)
    more = dict(q_start=start, max_query_len=nodes, out_dtype=torch.float32)
    if fp8:
        k, v = (x.to(torch.float8_e4m3fn) for x in (k, v))
        scale = [torch.full((hkv,), 1.0, device="cuda")] * 2
        out, _ = kf.kf_tree_attention_fp8(q, parents, k, v, *scale, table, ctx, L, d ** -0.5, ws, **more)
    else:
        out, _ = kf.kf_tree_attention(q, parents, k, v, table, ctx, L, d ** -0.5, ws, **more)
    assert kf.kf_get_device_error() == 0
    rows = lambda x, h: x[table[0].long()].flatten(0, 1)[:L, h:h + 1].double()
    worst = 0.0
    for b in (0, 7, B // 2, B - 1):
        for h in range(hkv):
            seen = torch.ones((nodes, L), dtype=torch.bool, device="cuda").tril(L - nodes)
            qb = q[b * nodes:(b + 1) * nodes, 4 * h:4 * h + 4].double()
            o, lse, spread, mag = ref.attend(qb, rows(k, h), rows(v, h), seen, d ** -0.5)
            assert float(lse.max()) <= 16
            moved = ref.small_q(qb, rows(k, h), d ** -0.5) if fp8 else 0.0
            pieces = 2 if fp8 else 3
            # 32 steps a piece, half a unit each on average of a rising sum, and the sum's first steps whole
            bound = (32 * pieces / 2 + pieces) * UNIT + (L / 512 + L / 128 + 32 + 4) * UNIT / 2 + 16 * UNIT / 2 * 0.02
            bound = bound + 2 * (4 * d * UNIT / 2 * mag + moved)
            err = (out[b * nodes:(b + 1) * nodes, 4 * h:4 * h + 4].double() - o).abs() / (spread * bound)[..., None]
            worst = max(worst, float(err.max()))
    print("worst %.3f of the bound, %.3g" % (worst, float(bound.max())))
    assert worst <= 1


@pytest.mark.parametrize("hq,hkv,d,nodes", [(8, 2, 128, 9), (8, 2, 64, 70), (8, 1, 128, 33), (4, 4, 64, 1)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_tree_sums_follow_the_maximum(kf, hq, hkv, d, nodes, fp8, scale):
    """Requests of every length around the tiles that are summed together, maxima that rise by
    little, by more than fp32 holds and not at all, a request of NaN between, an output and a
    workspace that held NaN before; all of them one behind the other in an SM's run, and alone,
    cut over many."""
    g = torch.Generator(device="cuda").manual_seed(17)
    bs = 16
    lens = [nodes + n for n in (4500, 1100, 1700, 511, 513, 1023, 1152, 2300, 130, 0)]
    nan_at = 1
    need = [-(-n // bs) for n in lens]
    first = np.concatenate([[0], np.cumsum(need)])
    k, v = (torch.randn((int(first[-1]) * bs, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lens):
        at, rows = torch.arange(n, device="cuda"), slice(first[b] * bs, first[b] * bs + n)
        by = {0: at / 400.0, 2: torch.where(at < 900, 0.01, 30.0), 3: torch.where(at < 100, 20.0, 0.01),
              7: at / 40.0, nan_at: at * float("nan")}.get(b)
        if by is not None:
            k[rows] = (k[rows] * by[:, None, None]).clamp(-400, 400).to(torch.bfloat16)
    q = (torch.randn((len(lens) * nodes, hq, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda")
    k, v = (x.view(-1, bs, hkv, d) for x in (k, v))
    ones = [torch.full((hkv,), 1.0, device="cuda")] * 2
    if fp8:
        k, v = (x.to(torch.float8_e4m3fn) for x in (k, v))

    def run(requests, ctas_full):
        """`ctas_full`: as often over as fills the SMs, so that runs hold whole requests."""
        reps = -(-200 // (len(requests) * hkv)) if ctas_full else 1
        who = requests * reps
        table = np.full((len(who), max(need)), -1, np.int32)
        for i, b in enumerate(who):
            table[i, :need[b]] = np.arange(first[b], first[b + 1])
        rows = torch.cat([torch.arange(b * nodes, (b + 1) * nodes) for b in who]).cuda()
        ws = kf.make_tree_workspace(len(who), nodes, hq, hkv, d)
        ws.view(torch.float32)[:] = float("nan")
        out = torch.full((len(rows), hq, d), float("nan"), device="cuda")
        ctx = torch.tensor([lens[b] for b in who], dtype=torch.int32, device="cuda")
        start = torch.arange(0, len(rows) + 1, nodes, dtype=torch.int32, device="cuda")
        args = (torch.from_numpy(table).cuda(), ctx, max(lens), scale, ws)
        more = dict(q_start=start, max_query_len=nodes, out=out)
        call = (lambda: kf.kf_tree_attention_fp8(q[rows], parents.repeat(len(who)), k, v, *ones, *args, **more)) if fp8 \
            else (lambda: kf.kf_tree_attention(q[rows], parents.repeat(len(who)), k, v, *args, **more))
        _, lse = call()
        for i, b in enumerate(who):
            at = slice(i * nodes, (i + 1) * nodes)
            if b == nan_at:
                assert torch.isnan(out[at]).all()
                continue
            if i >= 2 * len(requests) and i < len(who) - len(requests):
                continue
            kb, vb = (x[first[b]:first[b + 1]].flatten(0, 1)[:lens[b]].double() for x in (k, v))
            qb = q[b * nodes:(b + 1) * nodes].double()
            seen = torch.ones((nodes, lens[b]), dtype=torch.bool, device="cuda").tril(lens[b] - nodes)
            ref.check(out[at], lse[at], ref.attend(qb, kb, vb, seen, scale), lens[b], d, ref.FP16 if fp8 else ref.BF16,
                      "%s %s" % (requests, b), ref.small_q(qb, kb, scale) if fp8 else 0.0)

    every = list(range(len(lens)))
    run(every, False)
    run(every, True)
    run([0], False)
    run([2], False)
    run([7, nan_at, 3], True)
    assert kf.kf_get_device_error() == 0
