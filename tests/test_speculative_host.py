"""Host side of the speculative-step operators (no GPU): refusals before
anything is launched, the tree-mask helper, the split plan."""

import ctypes

import pytest
import torch

import spec_reference as R


@pytest.fixture(scope="module")
def K():
    from paged_kv_cache_482_b200 import build as B

    B.build()
    from paged_kv_cache_482_b200 import pagedkv

    pagedkv.lib()
    return pagedkv


def test_norm_rope_abi_refusals(K):
    L = K.lib()
    ok = dict(q=0x10000, qs=4096, qo=0x11000, qos=4096, k=0x20000, ks_=1024, v=0x30000, vs_=1024, qw=0x31000,
              kw=0x32000, eps=1e-6, kc=0x40000, vc=0x50000, sm=0x60000, pos=0x70000, cs=0x80000, mp=4096, style=0,
              N=4, nq=32, nkv=8, d=128, bs=16, nblk=10, dt=0, ks=None, vs=None)

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        return L.pkv_store_kvcache_norm_rope(
            a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks_"], a["v"], a["vs_"], a["qw"], a["kw"], a["eps"],
            a["kc"], a["vc"], a["sm"], a["pos"], a["cs"], a["mp"], a["style"], a["N"], a["nq"], a["nkv"], a["d"],
            a["bs"], a["nblk"], a["dt"], a["ks"], a["vs"], None, None)

    assert call(d=24) == K.PKV_ERR_INVALID_ARG
    assert call(d=48) == K.PKV_ERR_UNSUPPORTED
    assert call(d=1024, qs=1 << 16, qos=1 << 16, ks_=1 << 16, vs_=1 << 16) == K.PKV_ERR_UNSUPPORTED
    assert call(style=2) == K.PKV_ERR_INVALID_ARG
    assert call(qo=None) == K.PKV_ERR_INVALID_ARG
    assert call(qw=None) == K.PKV_ERR_INVALID_ARG
    assert call(kw=None) == K.PKV_ERR_INVALID_ARG
    assert call(kw=0x32008) == K.PKV_ERR_INVALID_ARG
    assert call(ks_=1023) == K.PKV_ERR_INVALID_ARG and call(ks_=1016) == K.PKV_ERR_INVALID_ARG
    assert call(vs_=512) == K.PKV_ERR_INVALID_ARG
    assert call(qs=4095) == K.PKV_ERR_INVALID_ARG and call(qos=2048) == K.PKV_ERR_INVALID_ARG
    assert call(qs=-4096) == K.PKV_ERR_INVALID_ARG
    assert call(nq=2**20, qs=2**27, qos=2**27) == K.PKV_ERR_INVALID_ARG  # more than 2^26 elements a token
    assert call(nkv=2**20, ks_=2**27, vs_=2**27) == K.PKV_ERR_INVALID_ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == K.PKV_ERR_INVALID_ARG
    assert call(mp=0) == K.PKV_ERR_INVALID_ARG
    assert call(cs=0x80008) == K.PKV_ERR_INVALID_ARG
    assert call(dt=1) == K.PKV_ERR_INVALID_ARG and call(dt=3) == K.PKV_ERR_INVALID_ARG
    assert call(pos=None) == K.PKV_ERR_INVALID_ARG
    assert call(N=-1) == K.PKV_ERR_INVALID_ARG
    assert call(N=0) == K.PKV_OK
    assert call(N=0, q=None, qo=None, k=None, v=None, pos=None, cs=None, sm=None) == K.PKV_OK


def test_tree_abi_refusals(K):
    L = K.lib()
    ok = dict(q=0x10000, kc=0x20000, vc=0x30000, bt=0x40000, maxb=8, cu=0x50000, cl=0x60000, mask=0x61000, words=2,
              S=4, T=100, nq=32, nkv=8, d=128, bs=256, nblk=100, scale=0.088, dt=0, ks=None, vs=None, mq=64,
              mc=2048, part=1, ws=None, wsb=0, out=0x70000)

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        return L.pkv_paged_attention_tree(
            a["q"], a["kc"], a["vc"], a["bt"], a["maxb"], a["cu"], a["cl"], a["mask"], a["words"], a["S"], a["T"],
            a["nq"], a["nkv"], a["d"], a["bs"], a["nblk"], a["scale"], a["dt"], a["ks"], a["vs"], a["mq"], a["mc"],
            a["part"], a["ws"], a["wsb"], a["out"], None, None)

    for name in ("q", "kc", "vc", "bt", "cu", "cl", "mask", "out"):
        assert call(**{name: None}) == K.PKV_ERR_INVALID_ARG, name
    assert call(out=0x70008) == K.PKV_ERR_INVALID_ARG
    assert call(d=96) == K.PKV_ERR_UNSUPPORTED
    assert call(nq=24) == K.PKV_ERR_UNSUPPORTED and call(nq=128) == K.PKV_ERR_UNSUPPORTED
    assert call(nq=30) == K.PKV_ERR_INVALID_ARG
    assert call(bs=100) == K.PKV_ERR_INVALID_ARG and call(bs=4, mc=32) == K.PKV_ERR_INVALID_ARG
    assert call(dt=1) == K.PKV_ERR_INVALID_ARG and call(dt=5) == K.PKV_ERR_INVALID_ARG
    for s in (float("nan"), -0.1, 0.0, float("inf")):
        assert call(scale=s) == K.PKV_ERR_INVALID_ARG
    assert call(mq=0) == K.PKV_ERR_INVALID_ARG
    assert call(words=1) == K.PKV_ERR_INVALID_ARG  # 64 drafts need two words
    assert call(words=0) == K.PKV_ERR_INVALID_ARG
    assert call(mc=2049) == K.PKV_ERR_INVALID_ARG  # beyond the table
    assert call(mc=0) == K.PKV_ERR_INVALID_ARG
    assert call(mq=65537, words=4096) == K.PKV_ERR_INVALID_ARG
    assert call(mc=2**31 - 1, maxb=2**24) == K.PKV_ERR_INVALID_ARG
    assert call(part=-1) == K.PKV_ERR_INVALID_ARG and call(part=4097) == K.PKV_ERR_INVALID_ARG
    assert call(part=0) == K.PKV_ERR_WORKSPACE and call(part=2, ws=0x80000, wsb=64) == K.PKV_ERR_WORKSPACE
    assert call(part=2, ws=0x80010, wsb=1 << 30) == K.PKV_ERR_INVALID_ARG  # not 256-byte aligned
    assert call(S=0, part=2, ws=0x80000, wsb=1 << 30) == K.PKV_OK
    assert call(nblk=2**31) == K.PKV_ERR_INVALID_ARG
    # scale pools are copied in 16-byte pieces; scales per head are read one by one
    for bad in (dict(ks=0x80004), dict(vs=0x90008)):
        assert call(dt=2, **{**dict(ks=0x80000, vs=0x90000), **bad}) == K.PKV_ERR_INVALID_ARG
    assert call(S=-1) == K.PKV_ERR_INVALID_ARG and call(T=-1) == K.PKV_ERR_INVALID_ARG
    assert call(S=0) == K.PKV_OK and call(T=0) == K.PKV_OK
    assert call(T=0, q=None, mask=None, out=None) == K.PKV_OK


def test_compact_abi_refusals(K):
    L = K.lib()
    ok = dict(kc=0x20000, vc=0x30000, bt=0x40000, maxb=8, cu=0x50000, cl=0x60000, acc=0x61000, most=4, n=0x62000,
              S=4, nkv=8, d=128, bs=16, nblk=100, dt=0, ks=None, vs=None)

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        return L.pkv_compact_kvcache(a["kc"], a["vc"], a["bt"], a["maxb"], a["cu"], a["cl"], a["acc"], a["most"],
                                     a["n"], a["S"], a["nkv"], a["d"], a["bs"], a["nblk"], a["dt"], a["ks"], a["vs"],
                                     None, None)

    for name in ("kc", "vc", "bt", "cu", "cl", "acc", "n"):
        assert call(**{name: None}) == K.PKV_ERR_INVALID_ARG, name
    for bad in (dict(kc=0x20008), dict(d=12), dict(d=0), dict(most=0), dict(maxb=0), dict(nblk=0), dict(bs=0),
                dict(nkv=0), dict(S=-1), dict(dt=3), dict(dt=2), dict(nblk=2**31), dict(nkv=1 << 20)):
        assert call(**bad) == K.PKV_ERR_INVALID_ARG, bad
    assert call(S=0) == K.PKV_OK
    assert call(S=0, kc=None, acc=None) == K.PKV_OK


def test_load_abi_refusals(K):
    L = K.lib()
    ok = dict(kc=0x20000, vc=0x30000, bt=0x40000, maxb=8, cu=0x50000, st=None, S=4, T=9, nkv=8, d=128, bs=16,
              nblk=100, dt=0, ks=None, vs=None, ko=0x70000, vo=0x80000)

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        return L.pkv_load_kvcache(a["kc"], a["vc"], a["bt"], a["maxb"], a["cu"], a["st"], a["S"], a["T"], a["nkv"],
                                  a["d"], a["bs"], a["nblk"], a["dt"], a["ks"], a["vs"], a["ko"], a["vo"], None, None)

    for name in ("kc", "vc", "bt", "cu", "ko", "vo"):
        assert call(**{name: None}) == K.PKV_ERR_INVALID_ARG, name
    for bad in (dict(kc=0x20008), dict(ko=0x70008), dict(d=12), dict(maxb=0), dict(nblk=0), dict(S=-1), dict(T=-1),
                dict(dt=1), dict(dt=2), dict(dt=3), dict(nblk=2**31), dict(nkv=1 << 20)):
        assert call(**bad) == K.PKV_ERR_INVALID_ARG, bad
    assert call(S=0) == K.PKV_OK and call(T=0) == K.PKV_OK


def _pools(dtype=torch.bfloat16):
    return torch.zeros(6, 2, 16, 64, dtype=dtype), torch.zeros(6, 2, 16, 64, dtype=dtype)


def test_python_refusals(K):
    """Types, shapes and strides are checked before the library is called; what
    passes them is refused for not being on a CUDA device."""
    i32 = dict(dtype=torch.int32)
    kc, vc = _pools()
    bf = dict(dtype=torch.bfloat16)
    k, v, q = torch.zeros(3, 2, 64, **bf), torch.zeros(3, 2, 64, **bf), torch.zeros(3, 4, 64, **bf)
    w, cs = torch.ones(64, **bf), torch.zeros(9, 64)
    sl, pos = torch.zeros(3, **i32), torch.zeros(3, **i32)

    def norm(**kw):
        a = dict(k=k, v=v, k_cache=kc, v_cache=vc, slot_mapping=sl, positions=pos, cos_sin=cs, k_weight=w, eps=1e-6,
                 q=q, q_weight=w)
        a.update(kw)
        return K.store_kvcache_norm_rope(**a)

    with pytest.raises(ValueError, match="CUDA device"):
        norm()
    for bad in (dict(k=k.float()), dict(slot_mapping=sl.long()), dict(cos_sin=cs.double()), dict(k_weight=w[:32])):
        with pytest.raises(TypeError):
            norm(**bad)
    for bad in (dict(k=k[:2]), dict(v=v[:, :1]), dict(q_weight=None), dict(positions=pos[:2]), dict(cos_sin=cs[:, :32]),
                dict(v_cache=vc[:5]), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(q=None, q_out=q), dict(q_out=q[:, :2])):
        with pytest.raises((ValueError, TypeError)):
            norm(**bad)
    k8, v8 = _pools(torch.uint8)
    s = torch.ones(2)
    for bad in (dict(), dict(k_scale=s), dict(k_scale=s, v_scale=torch.ones(6, 2, 16)), dict(k_scale=s, v_scale=s[:1]),
                dict(k_scale=s.double(), v_scale=s)):
        with pytest.raises(ValueError):
            norm(k_cache=k8, v_cache=v8, **bad)

    tab, cu, ctx = torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    mask = torch.zeros(3, 1, **i32)

    def tree(**kw):
        a = dict(q=q, k_cache=kc, v_cache=vc, block_tables=tab, cu_q_lens=cu, context_lens=ctx, tree_mask=mask,
                 scale=0.1, max_q_len=3)
        a.update(kw)
        return K.paged_attention_tree(**a)

    with pytest.raises(ValueError, match="CUDA device"):
        tree()
    for bad in (dict(q=q.half()), dict(tree_mask=mask.long()), dict(tree_mask=mask[:2]), dict(cu_q_lens=cu[:2]),
                dict(block_tables=tab[:1]), dict(q=q[:, :, :32].contiguous()), dict(out=q[:2]),
                dict(q=q.transpose(0, 1)), dict(k_cache=kc.transpose(0, 1)), dict(dev_err=torch.zeros(1)),
                dict(workspace=torch.zeros(4, 4).t())):
        with pytest.raises((ValueError, TypeError)):
            tree(**bad)

    acc, n = torch.zeros(2, 2, **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError, match="CUDA device"):
        K.compact_kvcache(kc, vc, tab, cu, ctx, acc, n)
    with pytest.raises((ValueError, TypeError)):
        K.compact_kvcache(kc, vc, tab, cu, ctx, acc[:1], n)
    with pytest.raises((ValueError, TypeError)):
        K.compact_kvcache(kc, vc, tab, cu, ctx, acc, n.long())
    with pytest.raises(ValueError, match="CUDA device"):
        K.load_kvcache(kc, vc, tab, cu, total_rows=4)
    with pytest.raises(ValueError):
        K.load_kvcache(kc, vc, tab, cu)
    with pytest.raises(ValueError):
        K.load_kvcache(kc, vc, tab, cu, k_out=k)
    with pytest.raises(ValueError):
        K.load_kvcache(kc, vc, tab, cu, k_out=k, v_out=v[:2])


def test_tree_mask_helper(K):
    m, depth = K.tree_mask([-1, 0, 0, 1, -1, 3])
    assert depth.tolist() == [0, 1, 1, 2, 0, 3]
    assert m.shape == (6, 1) and m.dtype == torch.int32
    assert [[j for j in range(6) if m[r, 0] >> j & 1] for r in range(6)] == [[0], [0, 1], [0, 2], [0, 1, 3], [4],
                                                                             [0, 1, 3, 5]]
    m, depth = K.tree_mask(list(range(-1, 69)), words=4)  # a chain over three words
    assert m.shape == (70, 4) and depth.tolist() == list(range(70))
    assert torch.equal(R.sees(m, 70), torch.ones(70, 70).tril().bool())
    assert K.tree_mask([])[0].shape == (0, 1)
    for bad in ([0], [-2], [-1, 1]):
        with pytest.raises(ValueError):
            K.tree_mask(bad)
    with pytest.raises(ValueError):
        K.tree_mask([-1] * 33, words=1)


def test_tree_plan(K):
    """The workspace holds two partials of up to 256 rows for every share."""
    for args in ((1, 32, 8, 128, 256, 8, 512), (64, 32, 8, 128, 16, 32, 32768), (1, 4, 4, 64, 8, 1, 1),
                 (3, 8, 1, 64, 1024, 300, 40000)):
        rows = min(256, args[5] * args[1] // args[2])
        for dt in (K.PKV_CACHE_BF16, K.PKV_CACHE_FP8_E4M3, K.PKV_CACHE_FP8_E4M3_TOKEN):
            for shares in (0, 1, 2, 77, 4096):
                p = K.plan_tree(*args, cache_dtype=dt, shares=shares)
                n = p["shares"]
                assert n == shares if shares else n >= 1
                least = 2 * n * rows * (args[3] + 2) * 4 if n > 1 else 0
                assert least <= p["workspace_bytes"] <= least + 512
    for bad in ((1, 32, 8, 96, 256, 8, 512), (1, 24, 8, 128, 256, 8, 512), (1, 32, 8, 128, 100, 8, 512),
                (1, 32, 8, 128, 256, 0, 512), (1, 32, 8, 128, 256, 8, 0), (-1, 32, 8, 128, 256, 8, 512),
                (1, 32, 8, 128, 256, 8, 512, 0, -1), (1, 32, 8, 128, 256, 8, 512, 0, 4097),
                (1, 32, 8, 128, 256, 8, 512, 3)):
        with pytest.raises(K.PagedKVError):
            K.plan_tree(*bad)
    assert K.lib().pkv_plan_tree(1, 32, 8, 128, 256, 8, 512, 0, 0, ctypes.POINTER(K._TreePlan)()) == \
        K.PKV_ERR_INVALID_ARG


def test_tree_workspace_is_planned_on_the_tensors_device(K, monkeypatch):
    """The number of shares follows the SMs of the device that is current: the workspace of a call on device 1
    made while device 0 is current is planned with device 1 current, as the launch is."""
    import contextlib

    current, planned = [0], []

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    def plan(*args):
        planned.append((current[0], args))
        return dict(shares=3, workspace_bytes=512)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(K, "_on_device", lambda *t: on)
    monkeypatch.setattr(K, "_empty", lambda shape, dtype, index, stream: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(K, "_run", lambda *a: None)
    monkeypatch.setattr(K, "plan_tree", plan)
    kc, vc = _pools()
    i32 = dict(dtype=torch.int32)
    for on in (1, 0):
        K.paged_attention_tree(torch.zeros(3, 4, 64, dtype=torch.bfloat16), kc, vc, torch.zeros(2, 3, **i32),
                               torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(3, 1, **i32), 0.1, 3)
    assert [p[0] for p in planned] == [1, 0] and current == [0]
    assert planned[0][1] == (2, 4, 2, 64, 16, 3, 48, K.PKV_CACHE_BF16, 0)
