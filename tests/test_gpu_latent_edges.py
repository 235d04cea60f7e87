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
