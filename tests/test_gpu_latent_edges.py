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
