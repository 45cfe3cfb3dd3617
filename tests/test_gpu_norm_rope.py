"""Per-head RMSNorm + RoPE + store on the GPU against the 64-bit formula."""

import pytest
import torch

import spec_reference as R
from paged_kv_cache_482_b200 import pagedkv as K
from paged_kv_cache_482_b200 import workloads as W

pytestmark = pytest.mark.gpu

EPS = 1e-6
# binary32 sum of at most 512 squares, square root, two products per factor:
# each of fewer than 2^5 dependent roundings and one approximate reciprocal
# square root (2 units) is within 2^-24 of its value
REL32 = 2.0 ** -18


def make(N, nq, nkv, d, bs, cache, seed, fused=True, spare=3):
    g = torch.Generator().manual_seed(seed)
    width = (nq + 2 * nkv) * d
    qkv = (torch.randn(N, width, generator=g) * torch.exp(torch.randn(N, 1, generator=g))).bfloat16().cuda()
    q, k, v = (x.view(N, x.shape[1] // d, d) for x in qkv.split([nq * d, nkv * d, nkv * d], 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = (1 + 0.3 * torch.randn(2, d, generator=g)).bfloat16().cuda()
    blocks = -(-max(N, 1) // bs) + spare
    slots = torch.randperm(blocks * bs, generator=g)[:N].int().cuda()
    top = 300
    pos = torch.randint(0, top, (N,), generator=g).int().cuda()
    cs = W.rope_cache(top, d).cuda()
    shape = (blocks, nkv, bs, d)
    ks = vs = None
    if cache == "bf16":
        kp = torch.full(shape, W.CANARY_BF16, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        vp = kp.clone()
    else:
        kp = torch.full(shape, W.CANARY_FP8, dtype=torch.uint8, device="cuda")
        vp = kp.clone()
        if cache == "fp8":
            ks, vs = (torch.rand(2, nkv, generator=g) * 0.02 + 0.005).cuda()
        else:
            ks, vs = (torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2))
    return dict(q=q, k=k, v=v, qw=qw, kw=kw, slots=slots, pos=pos, cs=cs, kp=kp, vp=vp, ks=ks, vs=vs)


def call(c, style=0, eps=EPS, err=None, **kw):
    a = dict(q=c["q"], q_weight=c["qw"], style=style, k_scale=c["ks"], v_scale=c["vs"], dev_err=err)
    a.update(kw)
    return K.store_kvcache_norm_rope(c["k"], c["v"], c["kp"], c["vp"], c["slots"], c["pos"], c["cs"], c["kw"], eps, **a)


def check_rows(got, ref, mag, what):
    g = got.double().cpu()
    tol = R.U_BF16 * (ref.abs() + REL32 * mag) + REL32 * mag + 1e-38
    assert bool(((g - ref).abs() <= tol).all()), f"{what}: off by {float(((g - ref).abs() / tol).max()):.3g} tolerances"


def check_store(c, before, style, eps=EPS, live=None):
    """K rows in tolerance, V rows as store_kvcache stores them, all else untouched."""
    N, nkv, d = c["k"].shape
    bs = c["kp"].shape[2]
    slots = c["slots"].cpu().long()
    keep = slots >= 0 if live is None else live
    t = torch.nonzero(keep).flatten()
    blk, off = slots[t] // bs, slots[t] % bs
    ref, mag = R.norm_rope(c["k"], c["kw"], eps, c["pos"], c["cs"], style)
    ref, mag = ref[t], mag[t]
    err = REL32 * mag
    if c["ks"] is None:
        check_rows(c["kp"].cpu()[blk, :, off], ref, mag, "k rows")
    else:
        code = R.e4m3_values(c["kp"])[blk, :, off]
        if c["ks"].dim() == 3:
            s = c["ks"].double().cpu()[blk, :, off]
            by = ref.abs().amax(-1) / 448
            assert bool(((s - by).abs() <= err.amax(-1) / 448 + 2 * R.U_F32 * by + 2.0 ** -126).all()), "k scales"
        else:
            s = c["ks"].double().cpu().expand(len(t), nkv)
        # against the scale that was used; the quotient is off by its rounding and by k's own error
        y = (ref / s[..., None]).clamp(-448, 448)
        tol = R.U_E4M3 * y.abs() + R.E4M3_STEP / 2 + (1 + R.U_E4M3) * (err / s[..., None] + R.U_F32 * y.abs())
        assert bool(((code - y).abs() <= tol).all()), "k codes"
    # v and everything that is not written: as the plain store leaves them
    kp, vp, ks, vs = before
    K.store_kvcache(c["v"].contiguous(), c["v"].contiguous(), kp, vp, torch.where(keep.cuda(), c["slots"], -1).int(),
                    vs, vs)
    assert torch.equal(c["vp"].view(torch.uint8), vp.view(torch.uint8)), "v pool"
    if c["vs"] is not None and c["vs"].dim() == 3:
        assert torch.equal(c["vs"].view(torch.int32), vs.view(torch.int32)), "v scales"
    rest = torch.ones(c["kp"].shape[:3], dtype=torch.bool)
    rest[blk, :, off] = False
    bits = c["kp"].cpu().view(torch.int16 if c["ks"] is None else torch.uint8)
    assert bool((bits[rest] == (W.CANARY_BF16 if c["ks"] is None else W.CANARY_FP8)).all()), "untouched rows"
    if c["ks"] is not None and c["ks"].dim() == 3:
        assert bool(c["ks"].cpu()[rest].isnan().all()), "untouched scales"


def copies(c):
    return tuple(None if c[n] is None else c[n].clone() for n in ("kp", "vp", "ks", "vs"))


CASES = [(N, nq, nkv, d, bs, cache, style)
         for cache in ("bf16", "fp8", "fp8_token") for style in (0, 1)
         for N, nq, nkv, d, bs in ((1, 32, 8, 128, 256), (37, 16, 2, 64, 16), (5, 3, 3, 16, 7))] + \
        [(3, 2, 1, 256, 8, "fp8_token", 0), (2, 1, 1, 512, 8, "bf16", 1), (700, 32, 8, 128, 16, "bf16", 0),
         (701, 16, 8, 128, 256, "fp8_token", 1), (1500, 4, 4, 64, 16, "fp8", 0), (9, 7, 5, 32, 16, "fp8", 1)]


@pytest.mark.parametrize("N,nq,nkv,d,bs,cache,style", CASES)
def test_against_the_formula(N, nq, nkv, d, bs, cache, style):
    c = make(N, nq, nkv, d, bs, cache, seed=N + d)
    before = copies(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, style, err=err)
    assert K.read_device_error(err) == K.PKV_OK
    ref, mag = R.norm_rope(c["q"], c["qw"], EPS, c["pos"], c["cs"], style)
    check_rows(out, ref, mag, "q")
    check_store(c, before, style)


@pytest.mark.parametrize("cache", ["bf16", "fp8_token"])
def test_skipped_slots_bad_positions_and_slots(cache):
    c = make(24, 8, 2, 128, 16, cache, seed=5)
    c["slots"][3] = -1
    c["slots"][11] = c["kp"].shape[0] * 16  # outside the pool
    c["pos"][7], c["pos"][20] = 300, -1     # outside the table
    before = copies(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(c["q"].contiguous(), 7.0)
    call(c, err=err, q_out=q_out)
    assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS
    good = torch.tensor([i not in (7, 20) for i in range(24)])
    assert bool((q_out[~good.cuda()] == 7.0).all())
    ref, mag = R.norm_rope(c["q"], c["qw"], EPS, c["pos"], c["cs"], 0)
    check_rows(q_out[good.cuda()], ref[good], mag[good], "q")
    check_store(c, before, 0, live=torch.tensor([i not in (3, 7, 11, 20) for i in range(24)]))


def test_strided_views_in_place_keys_only_and_contiguous_agree():
    c = make(41, 8, 4, 64, 16, "bf16", seed=6)
    base = copies(c)
    out = call(c)
    kp = c["kp"].clone()
    # contiguous inputs
    d = dict(c, q=c["q"].contiguous(), k=c["k"].contiguous(), v=c["v"].contiguous(), kp=base[0].clone(), vp=base[1].clone())
    assert torch.equal(call(d), out) and torch.equal(d["kp"].view(torch.int16), kp.view(torch.int16))
    # keys only
    e = dict(c, kp=base[0].clone(), vp=base[1].clone())
    assert call(e, q=None, q_weight=None) is None
    assert torch.equal(e["kp"].view(torch.int16), kp.view(torch.int16))
    # q in place, inside the fused projection
    f = dict(c, kp=base[0].clone(), vp=base[1].clone())
    k0, v0 = f["k"].clone(), f["v"].clone()
    got = call(f, q_out=f["q"])
    assert got is f["q"] and torch.equal(f["q"], out)
    assert torch.equal(f["k"], k0) and torch.equal(f["v"], v0)


def test_no_tokens_launches_nothing():
    c = make(0, 8, 4, 64, 16, "bf16", seed=6)
    assert call(c).shape == (0, 8, 64)


def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    for cache in ("bf16", "fp8_token"):
        c = make(12, 4, 2, 128, 16, cache, seed=8, fused=False)
        c["q"][2, 1] = 0
        c["k"][4, 1] = 0
        c["k"][6, 0, 5] = float("nan")
        c["q"][7, 0, 3] = float("inf")
        out = call(c)
        ref, mag = R.norm_rope(c["q"], c["qw"], EPS, c["pos"], c["cs"], 0)
        hit = torch.zeros(12, 4, dtype=torch.bool)
        hit[7, 0] = True
        check_rows(out.cpu()[~hit], ref[~hit], mag[~hit], "q")
        assert bool((out[2, 1] == 0).all()) and bool(out[7, 0].isnan().any())
        bs = 16
        s = c["slots"].cpu().long()
        rows = c["kp"].cpu()[s // bs, :, s % bs]
        vals = rows.double() if cache == "bf16" else R.e4m3_values(rows)
        assert bool((vals[4, 1] == 0).all()) and bool(vals[6, 0].isnan().any())
        keep = torch.ones(12, 2, dtype=torch.bool)
        keep[6, 0] = False
        assert bool(vals[keep].isfinite().all())


def test_captured_and_replayed():
    c = make(33, 8, 4, 128, 16, "fp8_token", seed=9)
    q_out = torch.empty(33, 8, 128, dtype=torch.bfloat16, device="cuda")
    want = call(c).clone()
    pools = copies(c)
    replay = K.graphed(lambda: call(c, q_out=q_out))
    for t in ("kp", "vp"):
        c[t].fill_(W.CANARY_FP8)
    q_out.zero_()
    replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, want)
    s = c["slots"].cpu().long()
    for t, p in zip(("kp", "vp"), pools):
        assert torch.equal(c[t].cpu()[s // 16, :, s % 16], p.cpu()[s // 16, :, s % 16])


def test_on_another_stream():
    c = make(64, 16, 8, 128, 16, "bf16", seed=10)
    want = call(c).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("N", [1, 64, 4001])
def test_in_place_while_other_rows_are_loaded(N, style):
    """q_out is q, in the fused projection: a token divided among warps, and more tokens than resident warps,
    whose next loads are in flight while rows are written. The result is the one of a separate q_out, bit for bit."""
    c = make(N, 32, 8, 128, 16, "bf16", seed=12)
    want = call(c, style)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    got = call(c, style, q_out=c["q"])
    assert got is c["q"]
    assert torch.equal(got.contiguous().view(torch.int16), want.view(torch.int16))
    assert torch.equal(c["kp"].view(torch.int16), kp.view(torch.int16))
    assert torch.equal(c["vp"].view(torch.int16), vp.view(torch.int16))
