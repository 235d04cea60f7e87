"""Latent attention (append, absorbed form, expanded form) against plain 64-bit
implementations.

Tolerances, element by element, with A = sum_t p_t |v_t| of the element (from
the reference) and bf16's half step 2^-8 (fp16: 2^-11):
 * absorbed: every softmax weight is rounded to bf16 once, so the sum is off by
   at most 2^-8 A; scores are fp32 sums of at most 576 exact products, whose
   rounding moves a weight by less than 1e-4 at these magnitudes
   (576 * 2^-24 * sum |q k| scale, sum |q k| scale < 40 here: < 1.4e-3 at the very
   worst, met only if every rounding error had one sign; 2e-4 is taken);
 * expanded: keys as pairs of bf16 numbers (the second rounds the first one's
   remainder, so 2^-16 of the key) move a score by at most 2^-16 sum |q k| scale
   = 2^-16 S, so a normalised weight by 2 * 2^-16 S; values and weights rounded
   to fp16 add 2 * 2^-11; the same 2e-4 for fp32 sums;
 * a bf16 output adds 2^-8 |out|.
lse: 2^-16 S (expanded) plus the library's 1e-4 relative.
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


class Case:
    """Inputs on the host and the device; queries of request b: counts[b] tokens."""

    def __init__(self, lens, counts, heads, R, bs=16, width=None, seed=0, qscale=1.0, gap=0, w=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.R, self.bs = list(lens), heads, R, bs
        self.cache, self.table = ref.paged(lens, bs, R + ref.ROPE, g)
        starts = np.concatenate([[gap], gap + np.cumsum(counts)])
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        nq = int(starts[-1]) + gap
        wid = (R if w is None else w) + ref.ROPE
        self.q = (torch.randn(nq, heads, wid, generator=g) * qscale).to(torch.bfloat16)
        self.scale = wid ** -0.5
        self.max_ctx, self.max_q = max(max(lens), 1), max(max(counts), 1)
        self.w_uk = self.w_uv = None
        if w is not None:
            self.w_uk = (torch.randn(heads, w, R, generator=g) * R ** -0.5).to(torch.bfloat16)
            self.w_uv = (torch.randn(heads, w, R, generator=g) * R ** -0.5).to(torch.bfloat16)

    def dev(self):
        ctx = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self.q.cuda(), self.cache.cuda(), self.table.cuda(), ctx, self.q_start.cuda()

    def run(self, kf, causal=True, out_dtype=torch.float32, ws=None, q_start=True, stream=None):
        q, cache, table, ctx, qs = self.dev()
        vd = self.R if self.w_uv is None else self.w_uv.shape[1]
        out = torch.full((q.shape[0], self.heads, vd), 77.0, dtype=out_dtype, device="cuda")
        lse = torch.full((q.shape[0], self.heads), 77.0, device="cuda")
        kw = dict(q_start=qs if q_start else None, max_query_len=self.max_q, causal=causal, out=out, lse_out=lse,
                  stream=stream)
        B = len(self.lens)
        if self.w_uk is None:
            ws = ws if ws is not None else kf.make_latent_workspace(B, self.max_q, self.heads, self.R)
            ws.fill_(0xff)   # any contents will do
            kf.kf_latent_attention(q, cache, table, ctx, self.max_ctx, self.scale, ws, **kw)
        else:
            ws = ws if ws is not None else kf.make_latent_expanded_workspace(B, q.shape[0], self.max_ctx, self.heads,
                                                                            vd, vd)
            ws.fill_(0xff)
            kf.kf_latent_attention_expanded(q, cache, self.w_uk.cuda(), self.w_uv.cuda(), table, ctx, self.max_ctx,
                                            self.scale, ws, **kw)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def check(self, out, lse, causal=True):
        o, l, mag, s = ref.latent(self.q, self.q_start, self.cache, self.table, self.lens, self.scale, causal,
                                  self.w_uk, self.w_uv)
        owned = ~np.isnan(l)
        g, gl = out.double().numpy(), lse.double().numpy()
        assert np.all(g[~owned[:, 0]] == 77.0) and np.all(gl[~owned] == 77.0), "rows that no request owns"
        if self.w_uk is None:
            tol = (2.0 ** -8 + 2e-4) * mag
            tol_l = 0.0
        else:
            tol = (2 * 2.0 ** -16 * s[..., None] + 2 * 2.0 ** -11 + 2e-4) * mag
            tol_l = 2.0 ** -16 * s
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(o)
        m = owned[:, 0]
        err = np.abs(g - o)[m]
        assert np.all(np.isfinite(g[m]))
        assert np.all(err <= tol[m] + 1e-30), (err - tol[m]).max()
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(gl) & owned, empty & owned)
        ok = owned & ~empty
        dl = np.abs(gl - np.where(ok, l, 0.0))
        lim = tol_l + 1e-4 * np.maximum(1.0, np.abs(l))
        assert np.all(dl[ok] <= (lim if np.ndim(lim) else np.full(l.shape, lim))[ok]), dl[ok].max()


# ----------------------------------------------------------------------------
# append
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("R,bs", [(512, 16), (256, 32)])
def test_append_one_row(kf, R, bs):
    g = torch.Generator().manual_seed(3)
    lens = [0, 1, bs - 1, bs, 3 * bs + 5]
    cache, table = ref.paged([n + 1 for n in lens], bs, R + 64, g)
    new = torch.randn(len(lens), R + 64, generator=g).to(torch.bfloat16)
    d = cache.cuda()
    kf.kf_append_latent(new.cuda(), d, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    want = cache.clone()
    for b, n in enumerate(lens):
        want[int(table[b, n // bs]), n % bs] = new[b]
    assert torch.equal(d.cpu().view(torch.int16), want.view(torch.int16))


def test_append_many_rows(kf):
    g = torch.Generator().manual_seed(4)
    lens, counts, bs, R = [0, 5, 16, 31, 2], [40, 0, 1, 3, 17], 16, 512
    cache, table = ref.paged([a + c for a, c in zip(lens, counts)], bs, R + 64, g)
    start = np.concatenate([[2], 2 + np.cumsum(counts)])
    new = torch.randn(int(start[-1]) + 3, R + 64, generator=g).to(torch.bfloat16)
    d = cache.cuda()
    kf.kf_append_latent(new.cuda(), d, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        row_start=torch.tensor(start, dtype=torch.int32).cuda())
    want = cache.clone()
    for b in range(len(lens)):
        for j in range(counts[b]):
            p = lens[b] + j
            want[int(table[b, p // bs]), p % bs] = new[int(start[b]) + j]
    assert torch.equal(d.cpu().view(torch.int16), want.view(torch.int16))


def test_append_bad_places_write_nothing(kf):
    g = torch.Generator().manual_seed(5)
    cache, table = ref.paged([20, 20, 20], 16, 576, g)
    bad = table.clone()
    bad[0, 0] = cache.shape[0]            # a block outside the pool
    bad[1, 0] = -1
    d = cache.cuda()
    before = torch.tensor([3, 4, table.shape[1] * 16], dtype=torch.int32)   # the last: past its table
    kf.kf_append_latent(torch.zeros(3, 576, dtype=torch.bfloat16).cuda(), d, bad.cuda(), before.cuda())
    torch.cuda.synchronize()
    assert kf.kf_get_device_error() == kf.KF_DEVERR_BLOCK_ID | kf.KF_DEVERR_APPEND_POS
    assert torch.equal(d.cpu().view(torch.int16), cache.view(torch.int16))


# ----------------------------------------------------------------------------
# absorbed form
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("heads", [1, 5, 16, 20, 64, 65, 128])
@pytest.mark.parametrize("R,bs", [(512, 16), (512, 32), (256, 16)])
def test_absorbed_decode(kf, heads, R, bs):
    c = Case([1, 2, 63, 64, 65, 200, 0, 129], [1] * 8, heads, R, bs, seed=heads + R)
    out, lse = c.run(kf)
    c.check(out, lse)


def test_absorbed_bf16_out_and_no_q_start(kf):
    c = Case([77, 300, 1], [1, 1, 1], 16, 512, seed=7)
    out, lse = c.run(kf, out_dtype=torch.bfloat16, q_start=False)
    c.check(out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,R", [(16, 512), (20, 256), (128, 512), (3, 512)])
def test_absorbed_several_queries(kf, causal, heads, R):
    c = Case([4, 70, 9, 130, 64, 5], [4, 3, 9, 1, 0, 5], heads, R, seed=11 + heads)
    out, lse = c.run(kf, causal=causal)
    c.check(out, lse, causal)


def test_absorbed_long_and_ragged(kf):
    """Runs that cross requests, requests cut over many CTAs, and one-token ones."""
    c = Case([5000, 1, 17, 3001, 0, 640], [1] * 6, 16, 512, bs=32, seed=13, qscale=2.0)
    out, lse = c.run(kf)
    c.check(out, lse)


def test_absorbed_rows_that_no_request_owns(kf):
    c = Case([33, 90], [2, 1], 16, 512, seed=17, gap=2)
    out, lse = c.run(kf)
    c.check(out, lse)


def test_absorbed_large_scores_and_masked_nan(kf):
    """Scores of several hundred (one token takes all the weight), NaN and infinite
    rows in the unused part of the last block."""
    c = Case([70, 33], [1, 1], 16, 512, seed=19, qscale=60.0)
    for b, n in enumerate(c.lens):
        blk = int(c.table[b, (n - 1) // 16])
        c.cache[blk, n % 16:] = float("nan")
        c.cache[blk, 15] = float("inf")
    out, lse = c.run(kf)
    o, l, mag, s = ref.latent(c.q, c.q_start, c.cache, c.table, c.lens, c.scale, True)
    # scores of size s are fp32 sums: each off by at most 576 * 2^-24 s
    ds = 576 * 2.0 ** -24 * s
    tol = (2.0 ** -8 + 2 * (np.exp(ds) - 1)[..., None]) * mag + 1e-6
    assert np.all(np.abs(out.double().numpy() - o) <= tol)
    assert np.all(np.abs(lse.double().numpy() - l) <= ds + 1e-4 * np.abs(l))


def test_absorbed_split_equals_itself_and_streams(kf):
    """Equal calls give equal bits, on a side stream too, with a dirty workspace."""
    c = Case([900, 40, 2000], [1, 1, 1], 32, 512, seed=23)
    a = c.run(kf)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = c.run(kf)
    d = c.run(kf, stream=torch.cuda.current_stream().cuda_stream)
    for x in (b, d):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_absorbed_graph(kf):
    """A captured step follows new contents of its buffers."""
    c = Case([100, 31, 64], [1, 1, 1], 16, 512, seed=29)
    q, cache, table, ctx, qs = c.dev()
    ws = kf.make_latent_workspace(3, 1, 16, 512)
    out = torch.zeros(3, 16, 512, device="cuda")
    lse = torch.zeros(3, 16, device="cuda")
    new = torch.randn(3, 576, device="cuda").to(torch.bfloat16)
    before = ctx - 1

    def step():
        kf.kf_append_latent(new, cache, table, before)
        kf.kf_latent_attention(q, cache, table, ctx, c.max_ctx, c.scale, ws, out=out, lse_out=lse)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        new.copy_(torch.randn(3, 576).to(torch.bfloat16))
        q.copy_(torch.randn(q.shape).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        c.q, c.cache = q.cpu(), cache.cpu()
        c.check(out.cpu(), lse.cpu())


def test_absorbed_graph_after_copies_and_a_joined_stream(kf):
    """The call directly behind copies, from the device and from pinned memory, and
    behind an event of another stream: captured, it still waits for all of them."""
    c = Case([100, 31, 640], [1, 1, 1], 16, 512, seed=30)
    q, cache, table, ctx, qs = c.dev()
    ws = kf.make_latent_workspace(3, 1, 16, 512)
    out = torch.zeros(3, 16, 512, device="cuda")
    lse = torch.zeros(3, 16, device="cuda")
    src, rows = torch.empty_like(q), torch.empty_like(cache)
    pinned = torch.empty(q.shape, dtype=q.dtype).pin_memory()
    side = torch.cuda.Stream()

    def step(kind):
        if kind == "device":
            q.copy_(src)
        elif kind == "pinned":
            q.copy_(pinned, non_blocking=True)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                cache.copy_(rows)
            torch.cuda.current_stream().wait_stream(side)
        kf.kf_latent_attention(q, cache, table, ctx, c.max_ctx, c.scale, ws, out=out, lse_out=lse)

    for kind in ("device", "pinned", "joined"):
        rows.copy_(cache)
        src.copy_(q)
        pinned.copy_(q)
        step(kind)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(kind)
        for seed in (1, 2):
            gen = torch.Generator().manual_seed(seed)
            new = torch.randn(q.shape, generator=gen).to(torch.bfloat16)
            src.copy_(new)
            pinned.copy_(new)
            rows.copy_(torch.randn(cache.shape, generator=gen).to(torch.bfloat16))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            c.q, c.cache = q.cpu(), cache.cpu()
            c.check(out.cpu(), lse.cpu())


@pytest.mark.parametrize("R", [512, 256])
def test_absorbed_more_queries_than_tokens(kf, R):
    """C > L, causal: the first C - L queries see nothing."""
    c = Case([2, 70, 0], [5, 3, 2], 20, R, seed=33)
    out, lse = c.run(kf)
    c.check(out, lse)
    assert np.all(np.isneginf(lse[:3].numpy())) and float(out[:3].abs().max()) == 0.0


@pytest.mark.parametrize("R", [512, 256])
def test_absorbed_many_small_requests(kf, R):
    """More requests than threads search for the runs."""
    lens = [(7 * i) % 50 for i in range(700)]
    c = Case(lens, [1] * 700, 2, R, seed=35)
    out, lse = c.run(kf)
    c.check(out, lse)


@pytest.mark.parametrize("lens", [[40, 50], [3000, 50]])
def test_absorbed_nan_query_stays_its_own(kf, lens):
    c = Case(lens, [1, 1], 16, 512, seed=37)
    clean, clean_lse = c.run(kf)
    c.q[0, 3, 5] = float("nan")
    out, lse = c.run(kf)
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
    keep = torch.ones(2, 16, dtype=torch.bool)
    keep[0, 3] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])


def test_absorbed_negative_and_zero_scale(kf):
    for scale in (-0.04, 0.0):
        c = Case([90, 33], [2, 1], 16, 512, seed=39)
        c.scale = scale
        out, lse = c.run(kf)
        c.check(out, lse)


def test_absorbed_device_errors(kf):
    c = Case([40, 50, 60], [1, 1, 1], 16, 512, seed=31)
    good = c.run(kf)[0]
    c.table[1, 0] = c.cache.shape[0] + 5
    out = c.run(kf)[0]
    assert kf.kf_get_device_error() == kf.KF_DEVERR_BLOCK_ID
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    c.table[1, 0] = 0
    c.lens[1] = c.table.shape[1] * 16 + 1
    c.run(kf)
    assert kf.kf_get_device_error() & kf.KF_DEVERR_CONTEXT_LEN
    c.lens[1] = -3
    c.run(kf)
    assert kf.kf_get_device_error() & kf.KF_DEVERR_CONTEXT_LEN
    c.lens[1] = 50
    c.max_ctx = 45
    c.run(kf)
    assert kf.kf_get_device_error() & kf.KF_DEVERR_MAX_CONTEXT


# ----------------------------------------------------------------------------
# expanded form
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,R,w,bs", [(3, 512, 128, 16), (2, 256, 64, 32), (1, 512, 64, 32)])
def test_expanded(kf, causal, heads, R, w, bs):
    c = Case([150, 40, 1, 0, 129, 300], [150, 7, 1, 0, 128, 33], heads, R, bs, seed=41 + heads, w=w)
    out, lse = c.run(kf, causal=causal)
    c.check(out, lse, causal)


def test_expanded_more_queries_than_a_tile(kf):
    c = Case([700, 257], [300, 257], 2, 256, 16, seed=43, w=64)
    out, lse = c.run(kf, out_dtype=torch.bfloat16)
    c.check(out, lse)


def test_expanded_one_query_a_request_and_gaps(kf):
    c = Case([33, 600], [1, 1], 2, 512, 16, seed=45, w=128, gap=3)
    out, lse = c.run(kf)
    c.check(out, lse)


def test_expanded_masked_nan(kf):
    c = Case([70, 33], [3, 33], 2, 512, 16, seed=47, w=128)
    for b, n in enumerate(c.lens):
        c.cache[int(c.table[b, (n - 1) // 16]), n % 16:] = float("nan")
    clean = Case([70, 33], [3, 33], 2, 512, 16, seed=47, w=128)
    out, lse = c.run(kf)
    clean.check(out, lse)


def test_expanded_more_queries_than_tokens(kf):
    c = Case([2, 70, 0], [140, 3, 2], 2, 256, 16, seed=53, w=64)
    out, lse = c.run(kf)
    c.check(out, lse)


def test_expanded_many_small_requests(kf):
    """More requests than the blocks sort, and a batch that they do."""
    for n in (330, 40):
        c = Case([1 + (5 * i) % 20 for i in range(n)], [1] * n, 1, 256, 16, seed=55, w=64)
        out, lse = c.run(kf)
        c.check(out, lse)


def test_expanded_nan_query_and_scales(kf):
    c = Case([60, 50], [30, 7], 2, 512, 16, seed=57, w=128)
    clean, clean_lse = c.run(kf)
    c.q[4, 1, 5] = float("nan")
    out, lse = c.run(kf)
    assert torch.isnan(out[4, 1]).all() and torch.isnan(lse[4, 1])
    keep = torch.ones(37, 2, dtype=torch.bool)
    keep[4, 1] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    for scale in (-0.05, 0.0):
        c = Case([60, 50], [30, 7], 2, 512, 16, seed=57, w=128)
        c.scale = scale
        out, lse = c.run(kf)
        c.check(out, lse)


def test_expanded_graph(kf):
    """A captured call follows new contents of its buffers."""
    c = Case([100, 70], [40, 70], 2, 256, 16, seed=59, w=64)
    q, cache, table, ctx, qs = c.dev()
    wk, wv = c.w_uk.cuda(), c.w_uv.cuda()
    ws = kf.make_latent_expanded_workspace(2, q.shape[0], 100, 2, 64, 64)
    out = torch.zeros(q.shape[0], 2, 64, device="cuda")
    lse = torch.zeros(q.shape[0], 2, device="cuda")

    def step():
        kf.kf_latent_attention_expanded(q, cache, wk, wv, table, ctx, 100, c.scale, ws, q_start=qs, max_query_len=70,
                                        out=out, lse_out=lse)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        cache.copy_(torch.randn(cache.shape).to(torch.bfloat16))
        q.copy_(torch.randn(q.shape).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        c.q, c.cache = q.cpu(), cache.cpu()
        c.check(out.cpu(), lse.cpu())


def test_loose_host_bounds(kf):
    """Host bounds far above the real ones cost nothing but the expanded workspace."""
    for w in (None, 128):
        c = Case([70, 9], [3, 2], 4, 512, seed=61, w=w)
        c.max_q = 2 ** 31 - 1
        if w is None:
            c.max_ctx = 2 ** 31 - 1
        c.check(*c.run(kf))


def test_expanded_agrees_with_absorbed(kf):
    """One batch through both forms, projections by plain products."""
    c = Case([90, 200], [5, 20], 8, 512, 16, seed=49, w=128)
    out, lse = c.run(kf)
    q, cache, table, ctx, qs = c.dev()
    wk, wv = c.w_uk.cuda().float(), c.w_uv.cuda().float()
    ql = torch.cat([torch.einsum("jhn,hnr->jhr", q[..., :128].float(), wk), q[..., 128:].float()], 2)
    ws = kf.make_latent_workspace(2, 20, 8, 512)
    o, l = kf.kf_latent_attention(ql.to(torch.bfloat16), cache, table, ctx, 200, c.scale, ws, q_start=qs,
                                  max_query_len=20, out_dtype=torch.float32)
    o = torch.einsum("jhr,hvr->jhv", o, wv).cpu()
    # the absorbed queries are rounded to bf16 here: off by 2^-8 of each product
    _, _, mag, s = ref.latent(c.q, c.q_start, c.cache, c.table, c.lens, c.scale, True, c.w_uk, c.w_uv)
    assert np.all(np.abs(lse.double().numpy() - l.cpu().double().numpy()) <= 2.0 ** -8 * s * 4 + 1e-3)
    err = (o - out).norm() / out.norm()
    assert float(err) < 3 * 2.0 ** -8


def test_expanded_out_of_range_is_reported(kf):
    c = Case([40], [40], 1, 256, 16, seed=51, w=64)
    c.w_uv.fill_(500.0)
    c.cache.fill_(8.0)          # 256 * 8 * 500 is far above fp16's largest number
    c.run(kf)
    assert kf.kf_get_device_error() == kf.KF_DEVERR_RANGE


def test_calls_on_several_streams_at_once(kf):
    """Calls that share inputs but no workspace, on four streams together, give the bits
    that each gives alone."""
    g = torch.Generator().manual_seed(71)
    lens = [700, 33, 1500, 260]
    one = Case(lens, [1] * 4, 128, 512, seed=72)
    q1, cache, table, ctx, qs1 = one.dev()
    many = Case(lens, [200, 33, 300, 7], 4, 512, seed=72, w=128)
    q2, cache2, table2, ctx2, qs2 = many.dev()
    uk, uv = many.w_uk.cuda(), many.w_uv.cuda()
    q3 = torch.randn(4 * 24, 16, 128, generator=g).to(torch.bfloat16).cuda()
    qs3 = torch.arange(0, 4 * 24 + 1, 24, dtype=torch.int32).cuda()
    k = torch.randn(int(table.max()) + 1, 16, 2, 128, generator=g).to(torch.bfloat16).cuda()
    lse3 = torch.full((4 * 24, 16), 6.0, device="cuda")
    scores = torch.rand(4, 1500, generator=g).cuda()
    rows = torch.randint(0, 255, (int(table.max()) + 1, 16, 2048), generator=g, dtype=torch.uint8).cuda()
    kept = torch.empty(4, dtype=torch.int32, device="cuda")
    outs = {n: t.cuda() for n, t in (
        ("absorbed", torch.zeros(4, 128, 512)), ("absorbed lse", torch.zeros(4, 128)),
        ("expanded", torch.zeros(q2.shape[0], 4, 128)), ("expanded lse", torch.zeros(q2.shape[0], 4)),
        ("weights", torch.zeros(4, 1500)), ("kept scores", torch.zeros(4, 1500)))}
    w1 = kf.make_latent_workspace(4, 1, 128, 512)
    w2 = kf.make_latent_expanded_workspace(4, q2.shape[0], 1500, 4, 128, 128)
    w4 = kf.make_evict_workspace(4, 1500, 250)
    calls = (
        lambda: kf.kf_latent_attention(q1, cache, table, ctx, 1500, one.scale, w1, out=outs["absorbed"],
                                       lse_out=outs["absorbed lse"]),
        lambda: kf.kf_latent_attention_expanded(q2, cache2, uk, uv, table2, ctx2, 1500, many.scale, w2, q_start=qs2,
                                                max_query_len=300, out=outs["expanded"],
                                                lse_out=outs["expanded lse"]),
        lambda: kf.kf_accumulate_attention(q3, k, table, ctx, 1500, 128 ** -0.5, lse3, outs["weights"], q_start=qs3,
                                           max_query_len=24),
        # (no source is a destination: the same call again moves the same rows)
        lambda: kf.kf_evict_tokens([rows], table, ctx, 1500, scores, 250, 4, 32, kept, outs["kept scores"], w4),
    )
    for call in calls:
        call()
    torch.cuda.synchronize()
    alone = {n: t.clone() for n, t in outs.items()}
    rows_alone = rows.clone()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for t in outs.values():
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for s, call in zip(streams, calls):
                with torch.cuda.stream(s):
                    call()
        torch.cuda.synchronize()
        for n, t in outs.items():
            assert torch.equal(t, alone[n]), n
        assert torch.equal(rows, rows_alone)
