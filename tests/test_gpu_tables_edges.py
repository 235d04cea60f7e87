"""Row ranges that do not ascend: which requests grow, and that no other loses its rows.
Rows wider than one pass of the kernels that write and move them."""
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


def grown(free, lens, starts, num_rows, cols, bs):
    """Request by request on the host. A range that leaves the rows, or starts before the end of an
    earlier one that does not leave them, grows nothing. -> free list, tables, lengths, slots, positions, bad ranges."""
    free, table = list(free), np.full((len(lens), cols), -1, np.int64)
    for b, n in enumerate(lens):
        for lb in range(-(-n // bs)):
            table[b, lb] = free.pop()
    before, taken = table.copy(), list(free)
    slots, pos, after, end, bad = np.full(num_rows, -1, np.int64), np.full(num_rows, -1, np.int64), list(lens), 0, 0
    for b, L in enumerate(lens):
        s, e = int(starts[b]), int(starts[b + 1])
        if not 0 <= s <= e <= num_rows:
            bad += 1
            continue
        ok, end = s >= end, max(end, e)
        if not ok:
            bad += 1
            continue
        for r in range(s, e):
            t = L + r - s
            if t % bs == 0:
                table[b, t // bs] = free.pop()
            slots[r], pos[r] = table[b, t // bs] * bs + t % bs, t
        after[b] = L + e - s
    return before, taken, free, table, after, slots, pos, bad


def extend_and_compare(kf, lens, starts, num_rows, bs=16, cols=8, in_place=False, num_blocks=None):
    nb = num_blocks or sum(-(-n // bs) for n in lens) + num_rows + len(lens)
    ids = np.random.default_rng(len(lens)).permutation(nb).tolist()
    before, list0, free, table, after, slots, pos, bad = grown(ids, lens, starts, num_rows, cols, bs)
    p = np.zeros(4 + nb, np.int32)
    p[0] = len(list0)
    p[4:4 + len(list0)] = list0
    pool, tab, ctx = i32(p), i32(before), i32(lens)
    got_slots = torch.full((num_rows,), -7, dtype=torch.int64, device="cuda")
    got_pos = torch.full((num_rows,), -7, dtype=torch.int32, device="cuda")
    got_after = ctx if in_place else torch.full_like(ctx, -7)
    kf.kf_extend_block_tables(pool, tab, ctx, bs, got_after, got_slots, row_start=i32(starts), positions=got_pos)
    err = kf.kf_get_device_error()
    assert got_slots.tolist() == slots.tolist() and got_pos.tolist() == pos.tolist()
    assert got_after.tolist() == after and np.array_equal(tab.cpu().numpy(), table)
    assert int(pool[0]) == len(free) and (pool[1:4] == 0).all() and pool[4:4 + len(free)].tolist() == free
    assert err == (kf.KF_DEVERR_CONTEXT_LEN if bad else 0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("starts,num_rows", [
    ([0, 9, 2, 4], 4),              # a range past the rows ahead of one that is right
    ([0, 4, 2, 6], 6),              # a range over rows that another has
    ([0, 2, -1, 3, 6], 6),
    ([5, 5, 0, 2, 2, 40, 2, 7], 7),
    ([3, 3, 3, 8], 9),              # rows that nobody has, requests without rows
    ([0, 2 ** 31 - 1, -2 ** 31, 5], 5)])
def test_ranges_that_do_not_ascend(kf, starts, num_rows, in_place):
    extend_and_compare(kf, [15 + 7 * b for b in range(len(starts) - 1)], starts, num_rows, in_place=in_place)


@pytest.mark.parametrize("batch", [511, 513, 1300, 5000])
def test_bad_ranges_among_many(kf, batch):
    """More requests than a block has threads; bad entries first, inside and last in a thread's share."""
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 4, batch)
    starts = np.concatenate([[0], np.cumsum(new)])
    n = int(starts[-1])
    lens = rng.integers(0, 60, batch).tolist()
    extend_and_compare(kf, lens, starts, n, in_place=True)
    for at, what in ((1, n + 5), (batch // 2, -3), (batch // 3, 0), (batch - 1, 2 ** 30), (7, -2 ** 31), (100, int(starts[130]))):
        bad = starts.copy()
        bad[at] = what
        extend_and_compare(kf, lens, bad, n, in_place=at % 2 == 0)
    bad = starts.copy()
    bad[rng.integers(0, batch, 40)] = rng.choice([-1, n + 1, 2 ** 31 - 1], 40)
    extend_and_compare(kf, lens, bad, n)


@pytest.mark.parametrize("hkv,d", [(8, 128), (9, 128), (17, 64), (12, 128), (32, 128), (100, 128)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_rows_of_any_width(kf, hkv, d, fp8):
    """128 vectors of 8 values are a pass of a warp. Slots that are refused leave both caches alone, and
    the other rows are written."""
    g = torch.Generator(device="cuda").manual_seed(hkv)
    n, nb, bs = 61, 5, 16
    k, v = (torch.randn((n, hkv, d), generator=g, device="cuda").mul_(100).to(torch.bfloat16) for _ in range(2))
    ks, vs = (torch.rand(hkv, generator=g, device="cuda") + 0.1 for _ in range(2))
    old = torch.randint(0, 100, (nb, bs, hkv, d), generator=g, device="cuda").to(torch.uint8 if fp8 else torch.bfloat16)
    held = lambda x, s: (x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x
    good = torch.randperm(nb * bs, generator=g, device="cuda")[:n]
    for bad in (None, nb * bs, -2, 2 ** 62, -2 ** 63, -1):
        slots = good.clone()
        if bad is not None:
            slots[7] = slots[n - 1] = bad
        live = slots == good
        kc, vc, wk, wv = (old.clone() for _ in range(4))
        wk.view(nb * bs, hkv, d)[slots[live]] = held(k, ks)[live]
        wv.view(nb * bs, hkv, d)[slots[live]] = held(v, vs)[live]
        if fp8:
            kf.kf_append_rows_fp8(k, v, kc, vc, ks, vs, slots)
        else:
            kf.kf_append_rows(k, v, kc, vc, slots)
        assert torch.equal(kc, wk) and torch.equal(vc, wv), bad
        assert kf.kf_get_device_error() == (0 if bad in (None, -1) else kf.KF_DEVERR_APPEND_POS)


@pytest.mark.parametrize("row_bytes", [16, 2032, 2048, 2064, 4112, 8192, 1 << 16])
@pytest.mark.parametrize("two", [False, True])
def test_commits_of_rows_of_any_width(kf, row_bytes, two):
    """128 vectors of 16 bytes are a pass of a block; a path that turns bad does so for every pass."""
    g = torch.Generator(device="cuda").manual_seed(row_bytes)
    nb, bs = 40, 16
    nodes = [30, 12, 20, 1, 9]
    lens = [60, 12, 100, 33, 20]
    # the second leaves the nodes, the third repeats one
    paths = [[0, 2, 3, 8, 9, 10, 15, 16, 20, 29], [0, 1, 11, 12, 13], [0, 5, 6, 6, 7], [0], [3, 8]]
    kept = [10, 3, 3, 1, 2]
    table = torch.full((5, 8), -1, dtype=torch.int32, device="cuda")
    ids, at = torch.randperm(nb, generator=g, device="cuda").to(torch.int32), 0
    for b, n in enumerate(lens):
        need = -(-n // bs)
        table[b, :need] = ids[at:at + need]
        at += need
    path = torch.full((5, 12), -1, dtype=torch.int32, device="cuda")
    for b, p in enumerate(paths):
        path[b, :len(p)] = i32(p)
    caches = [torch.randint(0, 256, (nb, bs, row_bytes), generator=g, device="cuda").to(torch.uint8)
              for _ in range(1 + two)]
    want = [c.clone() for c in caches]
    slot = lambda b, t: int(table[b, t // bs]) * bs + t % bs
    for c, w in zip(caches, want):
        for b, p in enumerate(paths):
            first = lens[b] - nodes[b]
            for i in range(kept[b]):
                w.view(nb * bs, -1)[slot(b, first + i)] = c.view(nb * bs, -1)[slot(b, first + p[i])]
    start = i32(np.concatenate([[0], np.cumsum(nodes)]))
    kf.kf_commit_tree(caches, table, i32(lens), start, path, i32([len(p) for p in paths]))
    assert kf.kf_get_device_error() == kf.KF_DEVERR_TREE
    for c, w in zip(caches, want):
        assert torch.equal(c, w)
