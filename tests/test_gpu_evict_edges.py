"""Accumulated weights and eviction at sizes that test_gpu_evict does not reach."""
import numpy as np
import pytest
import torch

from test_gpu_evict import _acc_inputs, _evict_case, _run_acc, kf, no_device_error  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("with_pos", [False, True])
@pytest.mark.parametrize("keep", [399990, 1000])
def test_evict_keys_beyond_shared_memory(kf, alias, with_pos, keep):
    """Keys computed again in every pass, in place and with positions, beside short
    requests; few moves and many."""
    _evict_case(kf, [400001, 30, 1200], keep, 4, 5, 16, 1, with_pos, 21, alias=alias)


@pytest.mark.parametrize("hq,hkv,D", [(20, 10, 128), (9, 9, 64), (48, 24, 64), (16, 16, 128)])
@pytest.mark.parametrize("fp8", [False, True])
def test_accumulate_windows_of_many_heads(kf, fp8, hq, hkv, D):
    """More KV heads than a block has warps: heads take turns."""
    lens, counts = [140, 7, 65, 300], [33, 7, 12, 0]
    a = _acc_inputs(lens, counts, hq, hkv, D, 16, fp8, seed=31 + hq)
    _run_acc(kf, a, lens, counts, True)
    _run_acc(kf, a, lens, counts, False)


@pytest.mark.parametrize("fp8", [False, True])
def test_accumulate_one_query_whatever_the_bound(kf, fp8):
    """Without q_start every request has one query, whatever max_query_len says: the same
    bits."""
    lens = [500, 33, 1200, 0, 1]
    cache, table, k_scale, start, q, lse, scores = _acc_inputs(lens, [1] * 5, 16, 4, 128, 16, fp8, seed=41)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    outs = []
    for bound in (1, 5, 64):
        out = torch.full(scores.shape, -5.0, device="cuda")
        args = (table.cuda(), ctx, 1200, 128 ** -0.5, lse.cuda(), out)
        kw = dict(scores_in=scores.cuda(), max_query_len=bound)
        if fp8:
            kf.kf_accumulate_attention_fp8(q.cuda(), cache.cuda(), k_scale.cuda(), *args, **kw)
        else:
            kf.kf_accumulate_attention(q.cuda(), cache.cuda(), *args, **kw)
        outs.append(out.cpu().numpy())
    for out in outs[1:]:
        assert np.array_equal(out, outs[0])
