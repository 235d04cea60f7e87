"""Accumulated attention weight and eviction against plain implementations, and
a run of them behind the library's decode step.

Accumulate, tolerance: a score is an fp32 sum of at most 128 exact products, off
by at most 128 * 2^-24 * sum |q k| scale (sum |q k| scale < 12 here), which moves
a weight by less than 1e-4 of itself; adding to scores_in rounds once more.
Eviction is exact.
"""
import numpy as np
import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kf():
    import __graft_entry__ as g
    g.build()
    from paged_kv_decode_kf_gb300 import kf
    assert kf.kf_get_device_error() == 0
    return kf


@pytest.fixture(autouse=True)
def no_device_error(kf):
    yield
    assert kf.kf_get_device_error() == 0, "a kernel raised a device error"


def _acc_inputs(lens, counts, hq, hkv, D, bs, fp8, seed, gap=0):
    g = torch.Generator().manual_seed(seed)
    cache, table = ref.paged(lens, bs, (hkv, D), g)
    k_scale = None
    if fp8:
        k_scale = torch.tensor([2.0 ** -(4 + h % 3) for h in range(hkv)])
        cache = (cache.float() / k_scale[:, None]).to(torch.float8_e4m3fn)
    start = torch.tensor(np.concatenate([[gap], gap + np.cumsum(counts)]), dtype=torch.int32)
    nq = int(start[-1]) + gap
    q = torch.randn(nq, hq, D, generator=g).to(torch.bfloat16)
    # any lse will do: near the true one for rows, -inf for a few (rows that saw nothing)
    lse = torch.log(torch.tensor([float(max(n, 1)) for n, c in zip(lens, counts) for _ in range(c)])) + 0.5
    full = torch.full((nq, hq), 3.0)
    full[gap:gap + len(lse)] = lse[:, None] + 0.3 * torch.randn(len(lse), hq, generator=g)
    scores = torch.rand(len(lens), max(max(lens), 1) + 3, generator=g)
    return cache, table, k_scale, start, q, full, scores


def _run_acc(kf, a, lens, counts, causal, use_in=True, alias=False, q_start=True, stream=None):
    cache, table, k_scale, start, q, lse, scores = a
    D = q.shape[2]
    out = torch.full(scores.shape, -5.0, device="cuda")
    sin = scores.cuda() if use_in else None
    if alias:
        out = sin
    kw = dict(scores_in=sin, causal=causal, max_query_len=max(max(counts), 1), stream=stream,
              q_start=start.cuda() if q_start else None)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    args = (table.cuda(), ctx, max(max(lens), 1), D ** -0.5, lse.cuda(), out)
    if k_scale is None:
        kf.kf_accumulate_attention(q.cuda(), cache.cuda(), *args, **kw)
    else:
        kf.kf_accumulate_attention_fp8(q.cuda(), cache.cuda(), k_scale.cuda(), *args, **kw)
    torch.cuda.synchronize()
    want, add = ref.accumulate(q, start, cache, table, lens, D ** -0.5, causal, lse, scores if use_in else None,
                               scores.shape[1], k_scale)
    got = out.cpu().double().numpy()
    live = ~np.isnan(want)
    rest = scores.double().numpy() if alias else np.full(got.shape, -5.0)
    assert np.array_equal(got[~live], rest[~live]), "entries past the context"
    err = np.abs(got - want)[live]
    assert np.all(err <= (1e-4 * add + 2.0 ** -23 * np.abs(want))[live] + 1e-30), err.max()
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,D,bs", [(8, 2, 128, 16), (4, 4, 64, 32), (16, 2, 128, 32), (6, 3, 64, 16),
                                         (32, 8, 128, 16)])
def test_accumulate_decode(kf, fp8, hq, hkv, D, bs):
    lens = [1, 15, 16, 17, 0, 200, 333]
    a = _acc_inputs(lens, [1] * 7, hq, hkv, D, bs, fp8, seed=hq + D)
    _run_acc(kf, a, lens, [1] * 7, True)
    _run_acc(kf, a, lens, [1] * 7, True, use_in=False, q_start=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (3, 3, 64), (16, 2, 64)])
def test_accumulate_windows(kf, fp8, causal, hq, hkv, D):
    lens, counts = [40, 7, 65, 0, 130, 12], [33, 7, 2, 0, 9, 0]
    a = _acc_inputs(lens, counts, hq, hkv, D, 16, fp8, seed=5 + hq, gap=2)
    _run_acc(kf, a, lens, counts, causal)
    _run_acc(kf, a, lens, counts, causal, alias=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_accumulate_long_windows_and_few_tokens(kf, fp8):
    """Several groups of 128 columns, more queries than tokens, many requests."""
    lens, counts = [150, 3, 129, 20], [70, 9, 1, 20]
    a = _acc_inputs(lens, counts, 16, 2, 128, 16, fp8, seed=91)
    _run_acc(kf, a, lens, counts, True)
    lens, counts = [(7 * i) % 40 for i in range(400)], [i % 3 for i in range(400)]
    a = _acc_inputs(lens, counts, 8, 1, 64, 32, fp8, seed=92)
    _run_acc(kf, a, lens, counts, True)
    lens = [(11 * i) % 40 for i in range(400)]
    a = _acc_inputs(lens, [1] * 400, 8, 1, 64, 32, fp8, seed=93)
    _run_acc(kf, a, lens, [1] * 400, True)


def test_accumulate_no_queries(kf):
    """No query at all: the scores come through."""
    lens, counts = [30, 5], [0, 0]
    a = _acc_inputs(lens, counts, 8, 2, 128, 16, False, seed=94)
    _run_acc(kf, a, lens, counts, True)


def test_accumulate_rows_without_weight_and_masked_nan(kf):
    lens, counts = [50, 20], [3, 1]
    a = list(_acc_inputs(lens, counts, 8, 2, 128, 16, False, seed=77))
    a[5][1, 3:] = -float("inf")
    a[0][int(a[1][0, 3]), 2:] = float("nan")      # past request 0's 50 tokens
    _run_acc(kf, tuple(a), lens, counts, True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts", [[1, 1], [3, 40]])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 2)])
def test_accumulate_nan_queries_without_weight(kf, fp8, counts, hq, hkv):
    """A query that holds NaN adds nothing where its lse is -inf."""
    lens = [150, 90]
    a = _acc_inputs(lens, counts, hq, hkv, 128, 16, fp8, seed=79)
    a[4][0, 1] = float("nan")
    a[5][0, 1] = -float("inf")
    a[4][-1, hq - 1] = float("nan")
    a[5][-1, hq - 1] = -float("inf")
    _run_acc(kf, a, lens, counts, True)
    _run_acc(kf, a, lens, counts, False)


@pytest.mark.parametrize("counts", [[1, 1], [3, 2], [20, 40]])
@pytest.mark.parametrize("hq", [2, 8, 16])
def test_accumulate_infinite_keys(kf, counts, hq):
    """Tokens whose scores are all -inf (an infinite number in the key) get nothing."""
    lens = [150, 90]
    a = _acc_inputs(lens, counts, hq, 2, 64, 16, False, seed=80)
    a[4][..., 5] = -a[4][..., 5].abs() - 1
    for b, t in ((0, 0), (0, 70), (0, 149), (1, 33)):
        a[0][int(a[1][b, t // 16]), t % 16, :, 5] = float("inf")
    _run_acc(kf, a, lens, counts, True)
    _run_acc(kf, a, lens, counts, False)


def test_accumulate_equal_bits_and_errors(kf):
    lens, counts = [300, 100], [1, 1]
    a = list(_acc_inputs(lens, counts, 32, 8, 128, 16, False, seed=78))
    one = _run_acc(kf, tuple(a), lens, counts, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    two = _run_acc(kf, tuple(a), lens, counts, True, stream=s)
    assert torch.equal(one, two)
    bad = a[1].clone()
    bad[0, 1] = 10 ** 6
    kf.kf_accumulate_attention(a[4].cuda(), a[0].cuda(), bad.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 300,
                               0.1, a[5].cuda(), one)
    assert kf.kf_get_device_error() == kf.KF_DEVERR_BLOCK_ID
    kf.kf_accumulate_attention(a[4].cuda(), a[0].cuda(), a[1].cuda(),
                               torch.tensor([-1, 301], dtype=torch.int32).cuda(), 300, 0.1, a[5].cuda(), one)
    # request 1's table has no blocks past its 100 tokens: those entries are -1
    assert kf.kf_get_device_error() == kf.KF_DEVERR_CONTEXT_LEN | kf.KF_DEVERR_MAX_CONTEXT | kf.KF_DEVERR_BLOCK_ID


# ----------------------------------------------------------------------------
# eviction
# ----------------------------------------------------------------------------

def _evict_case(kf, lens, keep, sink, recent, width, n_caches, with_pos, seed, dtype=torch.bfloat16, alias=False,
                scores=None, bs=16):
    g = torch.Generator().manual_seed(seed)
    _, table = ref.paged(lens, bs, 8, g)
    nb = int(table.max()) + 4
    caches = [torch.randint(0, 255, (nb, bs, width), generator=g, dtype=torch.uint8) for _ in range(n_caches)]
    B, M = len(lens), max(max(lens), 1) + 2
    if scores is None:
        scores = torch.rand(B, M, generator=g)
        scores[torch.rand(B, M, generator=g) < 0.3] = 0.25          # ties
    pos = seq = None
    if with_pos:
        pos = torch.stack([torch.randperm(2 * M, generator=g)[:M] for _ in range(B)]).to(torch.int32)
        seq = torch.full((B,), 2 * M, dtype=torch.int32)
    want = ref.evict(lens, scores, keep, sink, recent, pos, seq)
    d = [c.cuda() for c in caches]
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    sc = scores.cuda()
    s_out = sc if alias else torch.full((B, M), -9.0, device="cuda")
    c_out = ctx if alias else torch.full((B,), -9, dtype=torch.int32, device="cuda")
    p_in = None if pos is None else pos.cuda()
    p_out = None if pos is None else (p_in if alias else torch.full((B, M), -9, dtype=torch.int32, device="cuda"))
    ws = kf.make_evict_workspace(B, M, keep)
    ws.fill_(0xff)
    kf.kf_evict_tokens(d, table.cuda(), ctx, M, sc, keep, sink, recent, c_out, s_out, ws, positions=p_in,
                       seq_lens=None if seq is None else seq.cuda(), positions_out=p_out)
    torch.cuda.synchronize()
    for b, (n, at) in enumerate(want):
        assert int(c_out[b]) == n
        assert np.array_equal(s_out[b, :n].cpu().numpy().view(np.int32), scores[b].numpy()[at].view(np.int32)), b
        if not alias:
            assert torch.all(s_out[b, n:] == -9.0)
        if pos is not None:
            assert np.array_equal(p_out[b, :n].cpu().numpy(), pos[b].numpy()[at])
        for c in caches:
            src = c.clone()
            for i in range(n):
                if at[i] != i:
                    c[int(table[b, i // bs]), i % bs] = src[int(table[b, at[i] // bs]), at[i] % bs]
    for c, x in zip(caches, d):
        assert torch.equal(c, x.cpu())


@pytest.mark.parametrize("with_pos", [False, True])
@pytest.mark.parametrize("alias", [False, True])
def test_evict_ragged(kf, with_pos, alias):
    _evict_case(kf, [1, 30, 31, 32, 64, 100, 0, 257], 31, 4, 8, 1152, 1, with_pos, 1, alias=alias)
    _evict_case(kf, [1500, 2047, 3], 1025, 0, 0, 256, 2, with_pos, 2, alias=alias, bs=32)


@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 0, 1), (1, 1, 0), (50, 25, 25), (199, 0, 199), (199, 199, 0)])
def test_evict_budgets(kf, keep, sink, recent):
    _evict_case(kf, [200, 199, 198, 1], keep, sink, recent, 64, 2, False, 3)
    _evict_case(kf, [200, 199, 198, 1], keep, sink, recent, 64, 2, True, 4)


def test_evict_one_of_many(kf):
    _evict_case(kf, [2049] * 3 + [2048], 2048, 4, 256, 2048, 2, True, 5)


def test_evict_long(kf):
    _evict_case(kf, [70001, 5], 9001, 4, 1000, 16, 1, False, 6)


def test_evict_wide_and_few_moves(kf):
    """A cluster a request that moves its rows itself, and keys beyond shared memory."""
    _evict_case(kf, [9000, 8991, 8990, 100], 8990, 4, 100, 64, 2, True, 10)
    _evict_case(kf, [400001], 399990, 0, 5, 16, 1, False, 11)
    _evict_case(kf, [400001], 1000, 4, 5, 16, 1, False, 12)
    _evict_case(kf, [20000, 300, 12289], 5000, 4, 50, 32, 1, True, 15)


def test_evict_many_requests(kf):
    _evict_case(kf, [20 + i % 50 for i in range(300)], 40, 2, 8, 32, 1, True, 13)


def test_evict_graph(kf):
    """A captured call follows new scores."""
    g = torch.Generator().manual_seed(14)
    cache, table = ref.paged([100, 60], 16, 8, g)
    d, t = cache.cuda(), table.cuda()
    ctx = torch.tensor([100, 60], dtype=torch.int32, device="cuda")
    out_ctx = torch.zeros_like(ctx)
    sc = torch.rand(2, 100, device="cuda")
    so = torch.zeros_like(sc)
    ws = kf.make_evict_workspace(2, 100, 30)

    def step():
        kf.kf_evict_tokens([d], t, ctx, 100, sc, 30, 1, 4, out_ctx, so, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        d.copy_(cache)
        sc.copy_(torch.rand(2, 100))
        graph.replay()
        torch.cuda.synchronize()
        for b, (n, at) in enumerate(ref.evict([100, 60], sc.cpu(), 30, 1, 4)):
            assert np.array_equal(ref.rows_of(d.cpu(), table, b, n), ref.rows_of(cache, table, b, int(ctx[b]))[at])
            assert np.array_equal(so[b, :n].cpu().numpy(), sc[b].cpu().numpy()[at])


def test_evict_special_scores(kf):
    """All equal, signed zeros, infinities, NaN, negative ones."""
    s = torch.zeros(6, 102)
    s[1, ::2] = -0.0
    s[2] = torch.linspace(-1, 1, 102)
    s[3, 10:20] = float("inf")
    s[3, 30:40] = -float("inf")
    s[3, 35:50] = float("nan")
    s[4] = float("nan")
    s[5] = torch.finfo(torch.float32).min
    s[5, 60] = -float("inf")
    _evict_case(kf, [100] * 6, 40, 2, 5, 32, 1, False, 7, scores=s)
    _evict_case(kf, [100] * 6, 95, 0, 0, 32, 1, False, 8, scores=s)


def test_evict_bad_inputs_are_reported(kf):
    g = torch.Generator().manual_seed(9)
    cache, table = ref.paged([40, 40], 16, 8, g)
    bad = table.clone()
    bad[0] = -1
    d = cache.cuda()
    ctx_out = torch.zeros(2, dtype=torch.int32, device="cuda")
    sc = torch.rand(2, 40, device="cuda")
    ws = kf.make_evict_workspace(2, 40, 10)

    def call(t, lens):
        kf.kf_evict_tokens([d], t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 40, sc, 10, 0, 0, ctx_out,
                           torch.empty_like(sc), ws)
        torch.cuda.synchronize()
        return kf.kf_get_device_error()
    before = d.clone()
    assert call(bad, [40, 5]) == kf.KF_DEVERR_BLOCK_ID
    assert torch.equal(before, d)
    assert call(table, [-1, 5]) == kf.KF_DEVERR_CONTEXT_LEN
    assert call(table, [5, 41]) == kf.KF_DEVERR_MAX_CONTEXT
    assert call(table, [5, 10 ** 6]) == kf.KF_DEVERR_CONTEXT_LEN | kf.KF_DEVERR_MAX_CONTEXT


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------

def test_decode_with_a_bounded_cache(kf):
    """Steps of append + attention + accumulate + evict as a server with a bounded
    cache runs them, every step against the plain forms on the cache's contents."""
    torch.manual_seed(0)
    B, hq, hkv, D, bs, keep = 3, 8, 2, 128, 16, 40
    lens = torch.tensor([38, 40, 12], dtype=torch.int32)
    seq = torch.tensor([90, 200, 12], dtype=torch.int32)
    nb, cols = 16, 4
    table = torch.randperm(nb)[:B * cols].view(B, cols).to(torch.int32).cuda()
    k = torch.randn(nb, bs, hkv, D, device="cuda").to(torch.bfloat16)
    v = torch.randn(nb, bs, hkv, D, device="cuda").to(torch.bfloat16)
    scores = torch.rand(B, 64, device="cuda")
    pos = torch.stack([torch.randperm(int(s))[:64] if int(s) >= 64 else
                       torch.cat([torch.arange(int(s)), torch.zeros(64 - int(s))]) for s in seq]).to(torch.int32).cuda()
    ctx = lens.cuda()
    seen = seq.cuda()
    ws = kf.make_workspace(B, hq, hkv, D, 2)
    ews = kf.make_evict_workspace(B, 64, keep)
    scale = D ** -0.5
    for step in range(6):
        q = torch.randn(B, hq, D, device="cuda").to(torch.bfloat16)
        kn = torch.randn(B, hkv, D, device="cuda").to(torch.bfloat16)
        vn = torch.randn(B, hkv, D, device="cuda").to(torch.bfloat16)
        out, lse = kf.kf_decode_step(q, kn, vn, k, v, table, ctx, 64, scale, 2, ws)
        rows = torch.arange(B, device="cuda")
        pos[rows, ctx.long()] = seen          # the new token's position, and no weight yet
        scores[rows, ctx.long()] = 0.0
        ctx += 1
        seen += 1
        before = (ctx.cpu(), scores.cpu(), pos.cpu(), k.cpu(), v.cpu(), seen.cpu())
        kf.kf_accumulate_attention(q, k, table, ctx, 64, scale, lse, scores, scores_in=scores)
        want, add = ref.accumulate(q.cpu(), torch.arange(B + 1), k.cpu(), table.cpu(), before[0], scale, True,
                                   lse.cpu(), before[1], 64)
        for b in range(B):
            L = int(before[0][b])
            got = scores[b, :L].double().cpu().numpy()
            assert np.all(np.abs(got - want[b, :L]) <= 1e-4 * add[b, :L] + 2.0 ** -22 * want[b, :L])
            assert abs(add[b, :L].sum() - hq) < 1e-3      # the weights of a row sum to one
        acc = scores.cpu()
        kf.kf_evict_tokens([k, v], table, ctx, 64, scores, keep, 2, 8, ctx, scores, ews, positions=pos, seq_lens=seen,
                           positions_out=pos)
        torch.cuda.synchronize()
        plan = ref.evict(before[0], acc, keep, 2, 8, before[2], before[5])
        for b, (n, at) in enumerate(plan):
            assert int(ctx[b]) == n
            for cache, old in ((k, before[3]), (v, before[4])):
                a = ref.rows_of(old, table.cpu(), b, int(before[0][b]))[at]
                assert np.array_equal(ref.rows_of(cache.cpu(), table.cpu(), b, n), a)
            assert np.array_equal(pos[b, :n].cpu().numpy(), before[2][b].numpy()[at])
            p = set(pos[b, :n].tolist())
            newest = set(range(int(before[5][b]) - 8, int(before[5][b])))
            assert newest & set(before[2][b, :int(before[0][b])].tolist()) <= p   # those cached stay
