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


def weight_bound(pieces):
    """How far w / (1 + w) may be off, relatively, w = 2^x of a score known exactly, -4 <= x < 0:
    ex2.approx 2^-22; x, by the factor's rounding and its own, two half units of 4; what the pieces
    leave of w, a unit (two of fp16) or nothing; a step for each piece, a unit; the sum of weights, its
    inverse, the product and the output's rounding, half a unit each. Two pieces of bf16 would be off
    by up to 2^-17."""
    return 2 * UNIT + np.log(2) * 4 * UNIT + UNIT + pieces * UNIT + 4 * UNIT / 2


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


def exact_scores(n, hq, d, seed, e4m3):
    """q and k of one component each, whose product is a score of -4 <= scale * log2(e) * s < 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.zeros((n, hq, d), device="cuda") for _ in range(2))
    q[..., 5] = torch.rand((n, hq), generator=g, device="cuda") + 1
    k[..., 5] = -torch.rand((n, hq), generator=g, device="cuda") * 1.8 - 0.05
    if e4m3:
        k = k.to(torch.float8_e4m3fn).float()
    return q.to(torch.bfloat16), k.to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lead", [0, 77])
def test_prompt_weights_keep_their_bits(kf, d, lead):
    """Sequences of two tokens (behind `lead` ones of score 0 and value 0 that weigh nothing like as much
    where there are any): the second row's output is a weight's."""
    n, h, scale = 3000, 2, float(np.float32(0.7))
    q, k = exact_scores(n, h, d, 41, False)
    g = torch.Generator(device="cuda").manual_seed(42)
    v = (torch.rand((n, h, d), generator=g, device="cuda") + 1).to(torch.bfloat16)
    m = lead + 2
    x = torch.zeros((n, m, 3 * h, d), dtype=torch.bfloat16, device="cuda")
    x[:, -1, :h], x[:, -1, h:2 * h], x[:, -1, 2 * h:] = q, k, v
    if lead:          # far below: 2^-40 and less
        x[:, 1:-1, h:2 * h, 5] = -40.0
    x = x.view(n * m, 3 * h, d)
    start = torch.arange(0, n * m + 1, m, dtype=torch.int32, device="cuda")
    out, _ = kf.kf_prompt_attention(x[:, :h], x[:, h:2 * h], x[:, 2 * h:], start, m, scale, out_dtype=torch.float32)
    w = torch.exp(scale * (q.double() * k.double()).sum(-1))
    rest = lead * torch.exp(scale * -40.0 * q[..., 5].double()) if lead else 0.0
    want = (w / (1 + w + rest))[..., None] * v.double()
    err = ((out.view(n, m, h, d)[:, -1].double() - want).abs() / want).max()
    assert err <= weight_bound(3) + (UNIT if lead else 0), float(err)
    assert kf.kf_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_weights_keep_their_bits(kf, d, fp8):
    """One node behind a context of one token of score 0 and value 0."""
    n, h, bs, scale = 3000, 2, 16, float(np.float32(0.7))
    q, k = exact_scores(n, h, d, 43, fp8)
    v = torch.ones_like(k)
    kc, vc = (torch.zeros((n, bs, h, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[:, 1], vc[:, 1] = k, v
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    ctx = torch.full((n,), 2, dtype=torch.int32, device="cuda")
    parents = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    ws = kf.make_tree_workspace(n, 1, h, h, d)
    if fp8:
        kc, vc = (x.to(torch.float8_e4m3fn) for x in (kc, vc))
        ones = torch.ones(h, device="cuda")
        out, _ = kf.kf_tree_attention_fp8(q, parents, kc, vc, ones, ones, table, ctx, 2, scale, ws,
                                          out_dtype=torch.float32)
    else:
        out, _ = kf.kf_tree_attention(q, parents, kc, vc, table, ctx, 2, scale, ws, out_dtype=torch.float32)
    w = torch.exp(scale * (q.double() * k.double()).sum(-1))
    want = (w / (1 + w))[..., None]
    err = ((out.double() - want).abs() / want).max()
    assert err <= weight_bound(2 if fp8 else 3), float(err)
    assert kf.kf_get_device_error() == 0


@pytest.mark.parametrize("lens,hq,hkv,d", [([1000, 300, 1261], 12, 12, 64), ([1000, 300, 1261], 8, 2, 128),
                                           ([6000], 4, 2, 64), ([6000], 4, 1, 128)])
def test_prompts_as_near_as_documented(kf, lens, hq, hkv, d):
    """The error's size over all rows, relative to the output's. Of the 32 steps between two sums set
    aside each cuts off half a unit on average of a sum that grows by its root (2/3 of the last on
    average): 10.7 units, 0.72 of it as sums lie between powers of two: 8. Scores lose two units the same way
    (8 steps or 4), times a size of 1.5: 3. The root of the squares' sum: 8.5 units, 1.02e-6. The three
    pieces in one sum would be 24 (1.1e-6 and more was measured), sums not set aside more."""
    g = torch.Generator(device="cuda").manual_seed(44)
    T = sum(lens)
    x = torch.randn((T, hq + 2 * hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    x[:, :hq] *= 1.5
    q, k, v = x.split([hq, hkv, hkv], 1)
    ends = np.cumsum(lens)
    start = torch.tensor([0] + ends.tolist(), dtype=torch.int32, device="cuda")
    out, _ = kf.kf_prompt_attention(q, k, v, start, max(lens), d ** -0.5, out_dtype=torch.float32)
    off = size = 0.0
    for n, e in zip(lens, ends):
        for r in range(0, n, 1500):
            m = min(n, r + 1500)
            seen = torch.ones((m, m), dtype=torch.bool, device="cuda").tril()[r:]
            o = ref.attend(q[e - n + r:e - n + m].double(), k[e - n:e - n + m].double(), v[e - n:e - n + m].double(), seen,
                           d ** -0.5)[0]
            off += float(((out[e - n + r:e - n + m].double() - o) ** 2).sum())
            size += float((o ** 2).sum())
    assert (off / size) ** 0.5 <= 8.5 * UNIT, (off / size) ** 0.5


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d,nodes,L", [(128, 16, 1000), (128, 16, 20000), (64, 40, 20000)])
def test_trees_as_near_as_documented(kf, d, nodes, L, fp8):
    """As above; all pieces go into one sum, so that 96 steps (64) lie between two sums set aside: 24
    units (16); the scores' 3; parts are joined by e^(lse - M), |lse| up to 16: a unit of 16 in a part's
    weight at most, half a unit on average of two parts: 8. Their root: 25.5 units, 3.0e-6 (18.2, 2.2e-6)."""
    g = torch.Generator(device="cuda").manual_seed(45)
    hq, hkv, bs, B = 8, 2, 32, 100
    blocks = -(-L // bs)
    k, v = (torch.randn((blocks, bs, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    scales = [torch.full((hkv,), 1 / 16, device="cuda")] * 2
    if fp8:
        k, v = ((x.float() * 16).to(torch.float8_e4m3fn) for x in (k, v))
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = (torch.randn((B * nodes, hq, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda").repeat(B)
    ctx = torch.full((B,), L, dtype=torch.int32, device="cuda")
    start = torch.arange(0, B * nodes + 1, nodes, dtype=torch.int32, device="cuda")
    ws = kf.make_tree_workspace(B, nodes, hq, hkv, d)
    more = dict(q_start=start, max_query_len=nodes, out_dtype=torch.float32)
    if fp8:
        out, _ = kf.kf_tree_attention_fp8(q, parents, k, v, *scales, table, ctx, L, d ** -0.5, ws, **more)
    else:
        out, _ = kf.kf_tree_attention(q, parents, k, v, table, ctx, L, d ** -0.5, ws, **more)
    kk, vv = (x.flatten(0, 1)[:L].double() / (16 if fp8 else 1) for x in (k, v))
    off = size = 0.0
    for b in (0, 13, B - 1):
        rows = slice(b * nodes, (b + 1) * nodes)
        seen = torch.ones((nodes, L), dtype=torch.bool, device="cuda").tril(L - nodes)
        o = ref.attend(q[rows].double(), kk, vv, seen, d ** -0.5)[0]
        off += float(((out[rows].double() - o) ** 2).sum())
        size += float((o ** 2).sum())
    assert (off / size) ** 0.5 <= (18.2 if fp8 else 25.5) * UNIT, (off / size) ** 0.5
    assert kf.kf_get_device_error() == 0


def test_tree_sums_captured_and_on_streams(kf):
    """Sums set aside lie in the call's workspace: replayed graphs with other lengths, and four streams
    with a workspace each, give the bits of a call alone."""
    g = torch.Generator(device="cuda").manual_seed(46)
    hq, hkv, d, bs, C, L = 8, 2, 128, 16, 20, 6000
    B, blocks = 90, 6000 // 16
    k, v = (torch.randn((blocks, bs, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = (torch.randn((B * C, hq, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    parents = torch.arange(-1, C - 1, dtype=torch.int32, device="cuda").repeat(B)
    start = torch.arange(0, B * C + 1, C, dtype=torch.int32, device="cuda")
    lens = [torch.randint(C, L, (B,), generator=g, device="cuda", dtype=torch.int32) for _ in range(4)]
    spaces = [kf.make_tree_workspace(B, C, hq, hkv, d) for _ in range(4)]

    def call(ctx, ws, out=None, lse=None):
        return kf.kf_tree_attention(q, parents, k, v, table, ctx, L, d ** -0.5, ws, q_start=start, max_query_len=C,
                                    out=out, lse_out=lse, out_dtype=torch.float32)

    want = [call(n, spaces[0]) for n in lens]
    ctx, out, lse = lens[0].clone(), torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ctx, spaces[0], out, lse)
    for n, (o, l) in zip(lens, want):
        ctx.copy_(n)
        graph.replay()
        assert torch.equal(out, o) and torch.equal(lse, l)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s, ws, n in zip(streams, spaces, lens):
            with torch.cuda.stream(s):
                got.append(call(n, ws))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1])
    assert kf.kf_get_device_error() == 0
