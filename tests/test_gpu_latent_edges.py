"""Latent attention where its kernels' parts meet: maxima that move at the last
tile, host bounds above the real sizes, weights and values far below the largest,
row ranges that are none. Inputs, references and tolerances as in test_gpu_latent."""
import numpy as np
import pytest
import torch

import latent_ref as ref
from test_gpu_latent import Case, kf, no_device_error  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# absorbed form: the last tile raises every row's maximum
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("R,heads", [(512, 64), (512, 128), (256, 128)])
def test_absorbed_maximum_in_the_last_tile(kf, R, heads):
    """O^T is rescaled right before the epilogue, in every unit and every row; many
    times the same bits. (The last tile's tokens score some 15 powers of two above the
    rest, so that a factor taken from another place shows at once.)"""
    tile = 32 if R == 512 else 64
    lens = [200 + 7 * i for i in range(40)]
    c = Case(lens, [1] * 40, heads, R, seed=201 + heads)
    c.q[..., R] = 8.0
    lift = 10.5 / (8.0 * c.scale)
    for b, n in enumerate(lens):
        for t in range(n):
            c.cache[int(c.table[b, t // 16]), t % 16, R] = lift if t >= (n - 1) // tile * tile else 0.0
    first = c.run(kf)
    c.check(*first)
    q, cache, table, ctx, _ = c.dev()
    ws = kf.make_latent_workspace(40, 1, heads, R)
    want_out, want_lse = first[0].cuda(), first[1].cuda()
    out, lse = torch.empty_like(want_out), torch.empty_like(want_lse)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        kf.kf_latent_attention(q, cache, table, ctx, c.max_ctx, c.scale, ws, out=out, lse_out=lse)
        wrong += (out != want_out).sum() + (lse != want_lse).sum()
    assert int(wrong) == 0


# ----------------------------------------------------------------------------
# append: ranges that are none
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("start", [[0, 5, 3, 8], [-2, 3, 5, 8], [0, 2, 5, 9], [4, 4, 3, 3], [0, 8, 9, 8]])
def test_append_ranges_that_do_not_ascend_or_leave_the_rows(kf, start):
    """Reported, and what is written lies where some request's range puts it."""
    g = torch.Generator().manual_seed(211)
    lens = [3, 20, 0]
    cache, table = ref.paged([n + 12 for n in lens], 16, 576, g)
    new = torch.randn(8, 576, generator=g).to(torch.bfloat16)
    d = cache.cuda()
    kf.kf_append_latent(new.cuda(), d, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        row_start=torch.tensor(start, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert kf.kf_get_device_error() == kf.KF_DEVERR_CONTEXT_LEN
    got, allowed = d.cpu().view(torch.int16), {}
    for b, n in enumerate(lens):
        for r in range(max(start[b], 0), min(start[b + 1], 8)):
            p = n + r - start[b]
            allowed[int(table[b, p // 16]), p % 16] = new[r].view(torch.int16)
    old = cache.view(torch.int16)
    for blk, slot in np.argwhere((got != old).any(2).numpy()):
        assert torch.equal(got[blk, slot], allowed[int(blk), int(slot)])


def test_append_ranges_in_order_are_no_error(kf):
    """Many requests (more than a block's threads), some without rows."""
    g = torch.Generator().manual_seed(212)
    counts = [i % 3 for i in range(700)]
    cache, table = ref.paged([c + 1 for c in counts], 16, 320, g)
    start = np.concatenate([[0], np.cumsum(counts)])
    new = torch.randn(int(start[-1]), 320, generator=g).to(torch.bfloat16)
    d = cache.cuda()
    kf.kf_append_latent(new.cuda(), d, table.cuda(), torch.ones(700, dtype=torch.int32).cuda(),
                        row_start=torch.tensor(start, dtype=torch.int32).cuda())
    for b, c in enumerate(counts):
        for j in range(c):
            cache[int(table[b, 0]), 1 + j] = new[int(start[b]) + j]
    assert torch.equal(d.cpu().view(torch.int16), cache.view(torch.int16))


# ----------------------------------------------------------------------------
# expanded form: weights and values far below the largest
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dominant", [0.0, -1.0])
@pytest.mark.parametrize("w,at", [(64, 0), (64, 140000), (128, (1 << 18) - 1)])
def test_expanded_many_small_weights(kf, w, at, dominant):
    """One token of weight 1 and 2^18 - 1 others 17.4 nats below it, 0.7 % of the sum
    together; the one's value is 0, or the others' negated.

    Bound. The small weights are 2^-25.1 of the largest and 2^7 times that in fp16, whose
    step 2^-24 is 2^-5.9 of them: each is off by 2^-6.9 of itself at most; a value by
    2^-11. The product's fp32 sum takes 16 products at a time; each may lose up to one
    fp32 step, 2^-23, of the sum so far. Where all values are alike the sum grows evenly,
    its mean half of its end: N 2^-24 = 2^-6 of the result. Where the large token comes
    first, the sum is 1 throughout: N 2^-23 = 2^-5 of |value|, more than the others' share,
    and the test shows the lse and that nothing else goes wrong. l takes 2^12 sums of 64,
    each off by half a step, 2^-24: 2^-12, twice."""
    n, R = 1 << 18, 256
    g = torch.Generator().manual_seed(221)
    c = Case([n], [1], 1, R, 32, seed=222, w=w)
    c.q.zero_()
    c.q[..., w] = 1.0
    u = torch.randn(R, generator=g).to(torch.bfloat16)
    c.cache[...] = torch.cat([u, torch.zeros(64, dtype=torch.bfloat16)])
    blk = int(c.table[0, at // 32])
    c.cache[blk, at % 32, :R] = dominant * u
    c.cache[blk, at % 32, R] = 1.0
    c.scale = 17.4
    out, lse = c.run(kf)
    # by the definition: all other tokens share one key and one value
    v = c.w_uv[0].double().numpy() @ u.double().numpy()
    rest = (n - 1) * np.exp(-17.4)
    want = v * (rest + dominant) / (rest + 1.0)
    tol = (2.0 ** -6.9 + 2.0 ** -6) * rest + 2.0 ** -11 * (rest + abs(dominant)) + 2 * 2.0 ** -12 * (rest + abs(dominant))
    if dominant:
        tol += 2.0 ** -5
    err = np.abs(out[0, 0].double().numpy() - want)
    assert np.all(err <= tol * np.abs(v)), (err / np.abs(v)).max()
    assert abs(float(lse[0, 0]) - (17.4 + np.log1p(rest))) <= 1e-4 * 17.4


@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -16, 2.0 ** -22])
def test_expanded_small_values(kf, size):
    """Values below fp16's least normal number: off by 2^-25 at most, whatever their size."""
    c = Case([70, 300], [9, 40], 2, 256, 16, seed=231, w=64)
    c.w_uv = (c.w_uv.float() * size).to(torch.bfloat16)
    out, lse = c.run(kf)
    o, l, mag, s = ref.latent(c.q, c.q_start, c.cache, c.table, c.lens, c.scale, True, c.w_uk, c.w_uv)
    tol = (2 * 2.0 ** -16 * s[..., None] + 2 * 2.0 ** -11 + 2e-4) * mag + 2.0 ** -25
    assert np.all(np.abs(out.double().numpy() - o) <= tol)
    assert np.all(np.abs(lse.double().numpy() - l) <= 2.0 ** -16 * s + 1e-4 * np.maximum(1.0, np.abs(l)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("R,w,bs", [(256, 128, 16), (256, 128, 32), (512, 64, 16)])
def test_expanded_every_width_of_latent_and_head(kf, causal, R, w, bs):
    c = Case([150, 40, 1, 0, 129, 300], [150, 7, 1, 0, 128, 33], 3, R, bs, seed=241 + w, w=w)
    out, lse = c.run(kf, causal=causal)
    c.check(out, lse, causal)


# ----------------------------------------------------------------------------
# host bounds above the real sizes
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("R,heads", [(512, 20), (512, 64), (256, 20)])
def test_absorbed_work_is_cut_by_the_real_query_counts(kf, R, heads):
    """A bound of several draft tokens where requests bring one: the bits of the exact
    bound, so the same runs on the same CTAs."""
    lens = [900 + 37 * i for i in range(64)]
    c = Case(lens, [1] * 64, heads, R, seed=251 + heads)
    want = c.run(kf)
    c.check(*want)
    for bound in (4, 64, 2 ** 31 - 1):
        c.max_q = bound
        got = c.run(kf)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), bound
        got = c.run(kf, q_start=False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), bound


@pytest.mark.parametrize("counts", [[3] * 9, [1, 4, 1, 1, 4, 1, 0, 1, 2], [4] * 8 + [1], [2, 2, 2, 1, 2, 2, 2, 2, 2],
                                    [4, 0, 0, 0, 0, 0, 0, 0, 0]])
@pytest.mark.parametrize("R,heads", [(512, 40), (256, 64)])
def test_absorbed_odd_and_even_units(kf, R, heads, counts):
    """Requests of one, two, three and more units in one batch, cut over CTAs."""
    lens = [700, 33, 1500, 64, 5, 260, 90, 2100, 31]
    c = Case(lens, counts, heads, R, seed=261 + sum(counts))
    out, lse = c.run(kf)
    c.check(out, lse)
    c.max_q = 9
    out, lse = c.run(kf, causal=False)
    c.check(out, lse, False)


@pytest.mark.parametrize("R,heads", [(512, 40), (256, 64)])
def test_absorbed_graph_follows_query_counts(kf, R, heads):
    """A call captured with one set of query counts, replayed with others: requests of
    one, two and three units, with and without rows that no request owns."""
    lens = [700, 33, 1500, 64, 5, 260, 90]
    first = Case(lens, [4] * 7, heads, R, seed=271)
    q, cache, table, ctx, qs = first.dev()
    ws = kf.make_latent_workspace(7, 5, heads, R)
    for bound, captured in ((4, [4] * 7), (5, [1] * 7)):      # every query a request's; and not
        out = torch.empty(28, heads, R, device="cuda")
        lse = torch.empty(28, heads, device="cuda")
        qs.copy_(torch.tensor(np.concatenate([[0], np.cumsum(captured)]), dtype=torch.int32))

        def step():
            kf.kf_latent_attention(q, cache, table, ctx, 1500, first.scale, ws, q_start=qs, max_query_len=bound,
                                   out=out, lse_out=lse)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for counts in ([1] * 7, [4] * 7, [2, 2, 2, 2, 2, 2, 1], [1, 3, 0, 4, 4, 4, 1], [0] * 7):
            first.q_start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
            qs.copy_(first.q_start)
            out.fill_(77.0)
            lse.fill_(77.0)
            graph.replay()
            torch.cuda.synchronize()
            first.check(out.cpu(), lse.cpu())


@pytest.mark.parametrize("R", [512, 256])
@pytest.mark.parametrize("lens,counts,heads,gap,bound", [
    ([40], [1], 40, 2, 4), ([64], [3], 64, 0, 3), ([1], [1], 128, 0, 1), ([65], [2], 128, 1, 9), ([0], [2], 128, 0, 2),
    ([30, 0], [1, 0], 64, 3, 7), ([200], [9], 128, 0, 9)])
def test_absorbed_few_pairs(kf, R, lens, counts, heads, gap, bound):
    """One pair of CTAs or two, with units for one CTA of a pair or for both."""
    c = Case(lens, counts, heads, R, seed=281 + heads, gap=gap)
    c.max_q = bound
    out, lse = c.run(kf)
    c.check(out, lse)
