"""Latent attention and eviction calls: host-side checks and refusals. No GPU
needed: every call here returns before any CUDA work."""
import pytest
import torch


@pytest.fixture(scope="module")
def kf():
    import __graft_entry__ as g
    g.build()
    from paged_kv_decode_kf_gb300 import kf
    return kf


def _append(lib, **kw):
    a = dict(new=16, start=None, cache=16, bt=16, st=4, ctx=16, B=2, n=2, r=512, rope=64, bs=16, nb=8)
    a.update(kw)
    return lib.kf_append_latent(a["new"], a["start"], a["cache"], a["bt"], a["st"], a["ctx"], a["B"], a["n"], a["r"],
                                a["rope"], a["bs"], a["nb"], None)


def test_append_latent_host_checks(kf):
    lib = kf.raw()
    assert _append(lib, B=0, n=0) == kf.KF_OK
    assert _append(lib, start=16, n=0) == kf.KF_OK
    for bad in (dict(new=None), dict(cache=None), dict(bt=None), dict(ctx=None), dict(B=-1), dict(n=-1), dict(n=3),
                dict(st=0), dict(nb=0), dict(cache=8), dict(new=24), dict(start=18, n=5), dict(bs=0)):
        assert _append(lib, **bad) == kf.KF_ERR_INVALID, bad
    for bad in (dict(r=384), dict(rope=32), dict(bs=8), dict(bs=64)):
        assert _append(lib, **bad) == kf.KF_ERR_UNSUPPORTED, bad


def _latent(lib, **kw):
    a = dict(q=16, qs=16, cache=16, bt=16, st=4, ctx=16, causal=1, mc=64, mq=3, B=2, n=6, h=16, r=512, rope=64, bs=16,
             nb=8, scale=0.1, ws=16, wsb=1 << 40, out=16, dt=0, lse=None)
    a.update(kw)
    return lib.kf_latent_attention(a["q"], a["qs"], a["cache"], a["bt"], a["st"], a["ctx"], a["causal"], a["mc"],
                                   a["mq"], a["B"], a["n"], a["h"], a["r"], a["rope"], a["bs"], a["nb"], a["scale"],
                                   a["ws"], a["wsb"], a["out"], a["dt"], a["lse"], None)


def _expanded(lib, **kw):
    a = dict(q=16, qs=16, cache=16, uk=16, uv=16, bt=16, st=4, ctx=16, causal=1, mc=64, mq=3, B=2, n=6, h=16, r=512,
             rope=64, dn=128, dv=128, bs=16, nb=8, scale=0.1, ws=16, wsb=1 << 40, out=16, dt=0, lse=None)
    a.update(kw)
    return lib.kf_latent_attention_expanded(a["q"], a["qs"], a["cache"], a["uk"], a["uv"], a["bt"], a["st"], a["ctx"],
                                            a["causal"], a["mc"], a["mq"], a["B"], a["n"], a["h"], a["r"], a["rope"],
                                            a["dn"], a["dv"], a["bs"], a["nb"], a["scale"], a["ws"], a["wsb"],
                                            a["out"], a["dt"], a["lse"], None)


COMMON_BAD = (dict(q=None), dict(cache=None), dict(bt=None), dict(ctx=None), dict(ws=None), dict(out=None), dict(q=8),
              dict(cache=24), dict(ws=8), dict(out=4), dict(lse=2), dict(qs=18), dict(B=-1), dict(n=-1), dict(mc=-1),
              dict(mq=-1), dict(h=0), dict(st=0), dict(nb=0), dict(scale=float("nan")), dict(scale=float("inf")),
              dict(causal=2), dict(dt=5), dict(qs=None))
COMMON_UNSUPPORTED = (dict(r=384), dict(r=1024), dict(rope=0), dict(rope=32), dict(bs=8), dict(bs=64), dict(h=1025),
                      dict(B=70000), dict(n=1 << 30), dict(nb=1 << 40))


@pytest.mark.parametrize("call", [_latent, _expanded])
def test_latent_attention_host_checks(kf, call):
    lib = kf.raw()
    for ok in (dict(B=0, n=0), dict(n=0), dict(mq=0)):
        assert call(lib, **ok) == kf.KF_OK, ok
    for bad in COMMON_BAD:
        assert call(lib, **bad) == kf.KF_ERR_INVALID, bad
    for bad in COMMON_UNSUPPORTED:
        assert call(lib, **bad) == kf.KF_ERR_UNSUPPORTED, bad


def test_expanded_host_checks(kf):
    lib = kf.raw()
    for bad in (dict(uk=None), dict(uv=None), dict(uk=8), dict(uv=8), dict(dn=0), dict(dv=0)):
        assert _expanded(lib, **bad) == kf.KF_ERR_INVALID, bad
    for bad in (dict(dn=96, dv=96), dict(dn=128, dv=64), dict(dn=64, dv=128), dict(mc=2 ** 30)):
        assert _expanded(lib, **bad) == kf.KF_ERR_UNSUPPORTED, bad
    need = kf.kf_latent_expanded_workspace_size(2, 6, 64, 16, 128, 128)
    assert need >= 2 * 128 * 16 * (128 + 128) * 2
    assert _expanded(lib, wsb=need - 1) == kf.KF_ERR_INVALID
    assert kf.kf_latent_expanded_workspace_size(-1, 6, 64, 16, 128, 128) == 0
    assert kf.kf_latent_expanded_workspace_size(2, 6, 64, 0, 128, 128) == 0


def test_latent_workspace_size_arguments(kf):
    for bad in ((-1, 1, 16, 512), (1, -1, 16, 512), (1, 1, 0, 512), (1, 1, 16, 384)):
        assert kf.kf_latent_workspace_size(*bad) == 0
    if not torch.cuda.is_available():      # it is sized for the current device
        assert kf.kf_latent_workspace_size(4, 1, 16, 512) == 0


def _acc(lib, fp8, **kw):
    a = dict(q=16, qs=16, k=16, ks=16, bt=16, st=4, ctx=16, causal=1, mc=64, mq=3, B=2, n=6, hq=8, hkv=2, d=128, bs=16,
             nb=8, scale=0.1, lse=16, sin=None, out=16, ss=64)
    a.update(kw)
    head = (a["q"], a["qs"], a["k"]) + ((a["ks"],) if fp8 else ())
    return (lib.kf_accumulate_attention_fp8 if fp8 else lib.kf_accumulate_attention)(
        *head, a["bt"], a["st"], a["ctx"], a["causal"], a["mc"], a["mq"], a["B"], a["n"], a["hq"], a["hkv"], a["d"],
        a["bs"], a["nb"], a["scale"], a["lse"], a["sin"], a["out"], a["ss"], None)


@pytest.mark.parametrize("fp8", [False, True])
def test_accumulate_host_checks(kf, fp8):
    lib = kf.raw()
    for ok in (dict(B=0, n=0), dict(mc=0)):
        assert _acc(lib, fp8, **ok) == kf.KF_OK, ok
    for bad in (dict(q=None), dict(k=None), dict(bt=None), dict(ctx=None), dict(lse=None), dict(out=None), dict(q=8),
                dict(k=8), dict(lse=18), dict(sin=18), dict(out=18), dict(B=-1), dict(n=-1), dict(mq=-1), dict(mc=-1),
                dict(ss=63), dict(qs=None), dict(hq=0), dict(hkv=0), dict(d=0), dict(scale=float("inf")),
                dict(causal=-1), dict(st=0), dict(nb=0)) + ((dict(ks=None),) if fp8 else ()):
        assert _acc(lib, fp8, **bad) == kf.KF_ERR_INVALID, bad
    for bad in (dict(d=96), dict(bs=64), dict(hq=6), dict(hq=32, hkv=2), dict(hq=7, hkv=2), dict(B=70000),
                dict(n=1 << 30), dict(nb=1 << 40)):
        assert _acc(lib, fp8, **bad) == kf.KF_ERR_UNSUPPORTED, bad


def _evict(lib, **kw):
    a = dict(a=16, b=None, row=1152, bt=16, st=4, ctx=16, mc=64, B=2, bs=16, nb=8, s=16, so=16, ss=64, p=None, po=None,
             sl=None, keep=32, sink=2, recent=8, co=16, ws=16, wsb=1 << 40)
    a.update(kw)
    return lib.kf_evict_tokens(a["a"], a["b"], a["row"], a["bt"], a["st"], a["ctx"], a["mc"], a["B"], a["bs"], a["nb"],
                               a["s"], a["so"], a["ss"], a["p"], a["po"], a["sl"], a["keep"], a["sink"], a["recent"],
                               a["co"], a["ws"], a["wsb"], None)


def test_evict_host_checks(kf):
    lib = kf.raw()
    assert _evict(lib, B=0) == kf.KF_OK
    for bad in (dict(a=None), dict(bt=None), dict(ctx=None), dict(s=None), dict(so=None), dict(co=None), dict(ws=None),
                dict(a=8), dict(b=8), dict(ws=8), dict(s=18), dict(co=18), dict(B=-1), dict(mc=-1), dict(ss=63),
                dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=20, recent=20), dict(row=0), dict(p=16),
                dict(p=16, po=16), dict(sl=16), dict(po=16, sl=16)):
        assert _evict(lib, **bad) == kf.KF_ERR_INVALID, bad
    for bad in (dict(row=1000), dict(row=1 << 21), dict(bs=8), dict(B=70000)):
        assert _evict(lib, **bad) == kf.KF_ERR_UNSUPPORTED, bad
    need = kf.kf_evict_workspace_size(2, 64, 32)
    assert need >= 2 * 4 + 2 * 2 * 32 * 4
    assert _evict(lib, wsb=need - 1) == kf.KF_ERR_INVALID
    assert kf.kf_evict_workspace_size(2, 64, 0) == 0 and kf.kf_evict_workspace_size(-1, 64, 8) == 0


def test_token_counts_past_31_bits_are_refused(kf):
    """A tile's or a block's stride past the last token stays inside 31 bits."""
    lib, n = kf.raw(), (1 << 30) + 16
    for call in (_latent, _expanded):
        assert call(lib, mc=n, st=n // 16) == kf.KF_ERR_UNSUPPORTED
    for fp8 in (False, True):
        assert _acc(lib, fp8, mc=n, ss=n) == kf.KF_ERR_UNSUPPORTED
    assert _evict(lib, mc=n, ss=n) == kf.KF_ERR_UNSUPPORTED


def test_bindings_refuse_shapes_and_host_tensors(kf):
    bf, i32 = torch.bfloat16, torch.int32
    q = torch.zeros(2, 4, 576, dtype=bf)
    cache = torch.zeros(4, 16, 576, dtype=bf)
    bt, ctx, ws = torch.zeros(2, 2, dtype=i32), torch.ones(2, dtype=i32), torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kf.kf_latent_attention(q, cache, bt, ctx, 16, 0.1, ws)
    with pytest.raises(ValueError, match="CUDA"):
        kf.kf_append_latent(torch.zeros(2, 576, dtype=bf), cache, bt, ctx)
    with pytest.raises(ValueError, match="q must"):
        kf.kf_latent_attention(q[..., :512], cache, bt, ctx, 16, 0.1, ws)
    with pytest.raises(ValueError, match="one query token"):
        kf.kf_latent_attention(torch.zeros(3, 4, 576, dtype=bf), cache, bt, ctx, 16, 0.1, ws)
    with pytest.raises(ValueError, match="latent_cache"):
        kf.kf_latent_attention(q, torch.zeros(4, 16, 2, 64, dtype=bf), bt, ctx, 16, 0.1, ws)
    with pytest.raises(ValueError, match="w_uk"):
        kf.kf_latent_attention_expanded(torch.zeros(2, 4, 192, dtype=bf), cache, torch.zeros(3, 128, 512, dtype=bf),
                                        torch.zeros(4, 128, 512, dtype=bf), bt, ctx, 16, 0.1, ws)
    k = torch.zeros(4, 16, 2, 128, dtype=bf)
    with pytest.raises(ValueError, match="lse"):
        kf.kf_accumulate_attention(torch.zeros(2, 8, 128, dtype=bf), k, bt, ctx, 16, 0.1, torch.zeros(2, 4),
                                   torch.zeros(2, 16))
    with pytest.raises(ValueError, match="one or two"):
        kf.kf_evict_tokens([], bt, ctx, 16, torch.zeros(2, 16), 4, 0, 0, ctx, torch.zeros(2, 16), ws)
    with pytest.raises(ValueError, match="positions"):
        kf.kf_evict_tokens([k], bt, ctx, 16, torch.zeros(2, 16), 4, 0, 0, ctx, torch.zeros(2, 16), ws,
                           positions=torch.zeros(2, 15, dtype=i32))


def test_evict_refuses_caches_that_are_no_list(kf):
    i32 = torch.int32
    kv, ctx, sc = torch.zeros(2, 16, 2, 64), torch.ones(2, dtype=i32), torch.zeros(2, 32)
    args = (torch.zeros(2, 2, dtype=i32), ctx, 32, sc, 8, 0, 0, ctx, sc, torch.zeros(64, dtype=torch.uint8))
    for caches in (kv, [], [kv, kv, kv]):
        with pytest.raises(ValueError, match="one or two"):
            kf.kf_evict_tokens(caches, *args)
    with pytest.raises(ValueError, match="share one"):
        kf.kf_evict_tokens([kv, kv[:1]], *args)
