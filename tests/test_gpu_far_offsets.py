"""Prompts, draft trees and rows whose offsets pass 32 bits: the bits that the same rows give in
small arrays."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kf():
    from paged_kv_decode_kf_gb300 import kf
    kf.kf_get_device_error()
    return kf


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d,hkv", [(128, 8), (64, 3)])
def test_caches_past_32_bits(kf, fp8, d, hkv):
    """The first, the middle and the last blocks of caches of more than 2^32 numbers."""
    g = torch.Generator(device="cuda").manual_seed(3)
    bs, hq, C = 16, 4 * hkv, 21
    nb = 2 ** 32 // (bs * hkv * d) + 50
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    lens = [70, 150]
    L = sum(lens)
    blocks = [0, nb - 1, nb // 2, nb - 2, nb // 2 + 1, nb - 40, 1, nb - 3, nb - 7, 2, nb - 9, nb // 2 - 5, nb - 20, 3, nb - 30]
    need = [-(-n // bs) for n in lens]
    table = np.full((2, 12), -1, np.int64)
    table[0, :need[0]], table[1, :need[1]] = blocks[:need[0]], blocks[need[0]:need[0] + need[1]]
    small = np.where(table >= 0, [[blocks.index(x) if x >= 0 else 0 for x in r] for r in table.tolist()], -1)
    k, v = (torch.randn((L, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = (torch.randn((2 * C, hq, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    parents = i32(np.concatenate([[-1], np.arange(C - 1) // 2] * 2))
    scale = [torch.full((hkv,), 2.0 ** -5, device="cuda")] * 2
    ctx, start = i32(lens), i32([0, C, 2 * C])
    path = torch.full((2, C), -1, dtype=torch.int32, device="cuda")
    path[:, :5] = i32([0, 2, 6, 13, 20])
    ws = kf.make_tree_workspace(2, C, hq, hkv, d)
    got = []
    for n, t in ((nb, table), (len(blocks), small)):
        kc, vc = (torch.empty((n, bs, hkv, d), dtype=dt, device="cuda") for _ in range(2))
        slots = torch.tensor([int(t[b, i // bs]) * bs + i % bs for b in range(2) for i in range(lens[b])], device="cuda")
        tab = i32(t)
        if fp8:
            kf.kf_append_rows_fp8(k, v, kc, vc, *scale, slots)
            out, lse = kf.kf_tree_attention_fp8(q, parents, kc, vc, *scale, tab, ctx, 150, 0.1, ws, q_start=start,
                                                max_query_len=C, out_dtype=torch.float32)
        else:
            kf.kf_append_rows(k, v, kc, vc, slots)
            out, lse = kf.kf_tree_attention(q, parents, kc, vc, tab, ctx, 150, 0.1, ws, q_start=start, max_query_len=C,
                                            out_dtype=torch.float32)
        kf.kf_commit_tree([kc, vc], tab, ctx, start, path, i32([5, 5]))
        raw = lambda x: x.view(torch.uint8 if fp8 else torch.int16).flatten(0, 1)[slots].clone()
        got.append((out, lse, raw(kc), raw(vc)))
        assert kf.kf_get_device_error() == 0
        del kc, vc
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # and they are the rows that were written, but for those that moved
    if not fp8:
        want = k.view(torch.int16).clone()
        for first in (70 - C, L - C):
            want[first:first + 5] = k.view(torch.int16)[[first + j for j in (0, 2, 6, 13, 20)]]
        assert torch.equal(got[0][2], want)


def test_pools_and_slots_past_32_bits(kf):
    """A table entry of some 2^27 blocks of 32 tokens: slots of more than 2^31."""
    nb = 2 ** 27
    pool = torch.zeros(4 + nb, dtype=torch.int32, device="cuda")
    pool[0] = 3
    pool[4:7] = i32([5, nb - 1, nb - 2])
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    ctx, slots = i32([0, 0]), torch.empty(50, dtype=torch.int64, device="cuda")
    kf.kf_extend_block_tables(pool, table, ctx, 32, ctx, slots, row_start=i32([0, 40, 50]))
    want = [(nb - 2) * 32 + i for i in range(32)] + [(nb - 1) * 32 + i for i in range(8)] + [160 + i for i in range(10)]
    assert slots.tolist() == want and table.tolist() == [[nb - 2, nb - 1, -1], [5, -1, -1]]
    kf.kf_release_blocks(pool, table, ctx, 32)
    assert pool[:7].tolist() == [3, 0, 0, 0, 5, nb - 1, nb - 2] and kf.kf_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 8, 8)])
def test_prompts_past_32_bits(kf, dtype, d, hq, hkv):
    """Sequences behind the first 2^32 numbers of q and of the output; tokens 2^24 numbers apart."""
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = [300, 1, 129]
    n = sum(lens)
    q, k, v = (torch.randn((n, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    start = np.concatenate([[0], np.cumsum(lens)])
    want, wlse = kf.kf_prompt_attention(q, k, v, i32(start), 300, 0.1, out_dtype=dtype)
    lead = 2 ** 32 // (hq * d) + 77
    big = []
    for x in (q, k, v):
        b = torch.empty((lead + n,) + x.shape[1:], dtype=x.dtype, device="cuda")
        b[lead:] = x
        big.append(b)
    out, lse = kf.kf_prompt_attention(*big, i32(start + lead), 300, 0.1, out_dtype=dtype)
    assert torch.equal(out[lead:], want) and torch.equal(lse[lead:], wlse)
    del out, lse, big
    step = 2 ** 24
    far = []
    for x in (q, k, v):
        buf = torch.empty(step * (n - 1) + 2 ** 13, dtype=torch.bfloat16, device="cuda")
        y = buf.as_strided(x.shape, (step, d, 1))
        y.copy_(x)
        far.append(y)
    out, lse = kf.kf_prompt_attention(*far, i32(start), 300, 0.1, out_dtype=dtype)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert kf.kf_get_device_error() == 0
