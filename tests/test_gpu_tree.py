"""Tree attention over the paged cache on the GPU against the 64-bit formula."""

import math

import pytest
import torch

import spec_reference as R
from paged_kv_cache_482_b200 import pagedkv as K
from paged_kv_cache_482_b200 import workloads as W

pytestmark = pytest.mark.gpu


def make(ql, cl, nq, nkv, d, bs, cache, seed, extra_rows=0, words=None, spare=2):
    """Pools hold canaries (NaN) wherever no token lives."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in cl]
    blocks = sum(need) + spare
    perm = torch.randperm(blocks, generator=g)
    width = max(1, max(need))
    tab = torch.full((len(cl), width), -1, dtype=torch.int32)
    slots, at = [], 0
    for i, n in enumerate(cl):
        tab[i, :need[i]] = perm[at:at + need[i]].int()
        at += need[i]
        t = torch.arange(n)
        slots.append(tab[i].long()[t // bs] * bs + t % bs)
    slots = torch.cat(slots).int().cuda()
    N = int(slots.numel())
    k, v = (torch.randn(N, nkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    shape = (blocks, nkv, bs, d)
    ks = vs = None
    if cache == "bf16":
        kp = torch.full(shape, W.CANARY_BF16, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        vp = kp.clone()
    else:
        kp = torch.full(shape, W.CANARY_FP8, dtype=torch.uint8, device="cuda")
        vp = kp.clone()
        if cache == "fp8":
            ks, vs = ((torch.rand(2, nkv, generator=g) + 0.5) / 100).cuda()
        else:
            ks, vs = (torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2))
            v = v * torch.exp(torch.randn(N, 1, 1, generator=g)).bfloat16().cuda()  # scales that differ by token
    K.store_kvcache(k, v, kp, vp, slots, ks, vs)
    T = sum(ql)
    most = max(1, max(ql))
    words = words or -(-most // 32)
    masks = []
    for c in ql:
        parents = [int(torch.randint(max(-1, j - 6), j, (1,), generator=g)) for j in range(c)]
        masks.append(K.tree_mask(parents, words=words)[0])
    masks.append(torch.full((extra_rows, words), -1, dtype=torch.int32))
    q = (torch.randn(T + extra_rows, nq, d, generator=g) * 2).bfloat16().cuda()
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32).cuda()
    return dict(q=q, kp=kp, vp=vp, ks=ks, vs=vs, tab=tab.cuda(), cu=cu, ctx=torch.tensor(cl, dtype=torch.int32).cuda(),
                mask=torch.cat(masks).cuda(), most=most, scale=1 / math.sqrt(d), cache=cache)


def call(c, **kw):
    a = dict(k_scale=c["ks"], v_scale=c["vs"])
    a.update(kw)
    return K.paged_attention_tree(c["q"], c["kp"], c["vp"], c["tab"], c["cu"], c["ctx"], c["mask"], c["scale"],
                                  a.pop("max_q_len", c["most"]), **a)


def reference(c):
    return R.tree_attention(c["q"], R.cache_values(c["kp"], c["ks"]), R.cache_values(c["vp"], c["vs"]), c["tab"],
                            c["cu"], c["ctx"], c["mask"], c["scale"])


def close(c, out, ref, mag, what=""):
    g = out.double().cpu()
    live = ~ref.isnan()
    tol = R.tree_tolerance(ref, mag, c["cache"] != "bf16", c["cache"] == "fp8_token")
    bad = ((g - ref).abs() > tol) | g.isnan()
    assert not bool(bad[live].any()), f"{what}: off by {float(((g - ref).abs() / tol)[live].max()):.3g} tolerances"


def check(c, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, dev_err=err, **kw)
    assert K.read_device_error(err) == K.PKV_OK
    ref, mag = reference(c)
    close(c, out, ref, mag)
    return out


SHAPES = [(8, 2, 128, 16), (4, 4, 64, 8), (8, 4, 64, 256), (8, 1, 128, 64), (16, 2, 64, 1024)]


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("nq,nkv,d,bs", SHAPES)
def test_against_the_formula(nq, nkv, d, bs, cache):
    check(make([1, 8, 17, 3, 33], [1, 90, 300, 515, 129], nq, nkv, d, bs, cache, seed=nq * d + bs))


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
def test_lengths_around_tiles(cache):
    """Contexts and drafts on, before and behind the borders of 64 and 128."""
    cl = [63, 64, 65, 127, 128, 129, 191, 192, 193, 256, 257]
    check(make([1, 2, 31, 32, 33, 63, 64, 64, 5, 64, 7], cl, 8, 2, 128, 16, cache, seed=1))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("cache", ["bf16", "fp8_token"])
def test_wide_trees(G, cache):
    """Rows that fill several query tiles, masks of several words."""
    check(make([100, 257, 128], [400, 700, 128], 8, 8 // G, 128, 64, cache, seed=G))


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("shares", [0, 1, 2, 3, 10, 37, 300])
def test_any_cut_of_the_work(cache, shares):
    """One block for everything, a few, and more blocks than tiles: units whole,
    cut once, cut many times, and joined from a workspace of NaN."""
    c = make([4, 9, 1, 20, 50], [2500, 70, 1, 1111, 180], 8, 2, 128, 16, cache, seed=11)
    p = K.plan_tree(5, 8, 2, 128, 16, 50, 2512, cache_dtype=K.cache_dtype(c["kp"], c["ks"]), shares=shares)
    ws = torch.full((max(256, p["workspace_bytes"]),), 0xFF, dtype=torch.uint8, device="cuda")
    check(c, shares=shares, workspace=ws)


def test_rows_without_keys_are_zeros_and_others_are_not():
    """No cached token before the drafts and an empty mask row; a row whose own
    bit is not set; bits at and above the chunk's length."""
    for cache in ("bf16", "fp8", "fp8_token"):
        c = make([5, 6, 1], [5, 70, 1], 8, 2, 128, 16, cache, seed=13)
        c["mask"][0] = 0
        c["mask"][3] = 1 << 1
        c["mask"][5] = 0          # of the second sequence: the prefix alone
        c["mask"][6] |= -64       # bits at 6 and above
        c["mask"][11] = 0         # a one-token sequence that sees nothing
        out = check(c)
        assert bool((out[0] == 0).all()) and bool((out[11] == 0).all()) and bool((out[3] != 0).any())


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_masked_does_not_reach_a_row(cache, d):
    """Infinities and NaN in K and V of a draft reach exactly the rows that see it."""
    c = make([12, 40], [50, 200], 8, 2, d, 16, cache, seed=17)
    clean = call(c).clone()
    tab = c["tab"].cpu().long()
    for seq, u in ((0, 3), (1, 7), (1, 36)):
        t = int(c["ctx"][seq]) - int(c["cu"][seq + 1] - c["cu"][seq]) + u
        blk, off = int(tab[seq, t // 16]), t % 16
        if cache == "bf16":
            c["kp"][blk, :, off, 1] = float("nan")
            c["vp"][blk, 0, off] = float("inf")
            c["vp"][blk, 1, off, 5] = float("nan")
        else:
            c["kp"][blk, :, off, 1] = 0x7F
            c["vp"][blk, 0, off] = 0x7F
            c["vp"][blk, 1, off, 5] = 0x7F
            if cache == "fp8_token":
                c["vs"][blk, 1, off] = float("inf")
    out = call(c)
    saw = torch.zeros(52, dtype=torch.bool)
    bits = R.sees(c["mask"], 64)
    saw[:12] = bits[:12, 3]
    saw[12:] = bits[12:, 7] | bits[12:, 36]
    assert bool(saw.any()) and not bool(saw.all())
    assert torch.equal(out.cpu()[~saw], clean.cpu()[~saw])
    assert bool(out.cpu()[saw].isnan().any(-1).all())


def test_non_finite_v_reaches_the_elements_it_is_in():
    c = make([6], [80], 4, 2, 64, 16, "bf16", seed=18)
    c["mask"].copy_(torch.tensor([[1], [3], [5], [9], [17], [35]], dtype=torch.int32))
    t = 74 + 1
    blk, off = int(c["tab"][0, t // 16]), t % 16
    clean = call(c).clone()
    c["vp"][blk, :, off, 9] = float("inf")
    out = call(c)
    for r in range(6):
        hit = r in (1, 5)
        want = clean[r].clone()
        if hit:
            want[:, 9] = float("inf")
        assert torch.equal(out[r], want), r


def test_bad_input_gives_zeros_and_is_reported():
    c = make([3, 4, 5, 6, 2], [40, 50, 60, 70, 33], 8, 2, 128, 16, "bf16", seed=19)
    good = call(c).clone()
    c["tab"][1, 2] = c["kp"].shape[0]
    c["tab"][3, 0] = -1
    c["ctx"][2] = 4  # shorter than its drafts
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(good, 5.0)
    call(c, out=out, dev_err=err)
    assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS
    assert torch.equal(out[:3], good[:3]) and torch.equal(out[18:], good[18:])
    assert bool((out[3:18] == 0).all())
    # a chunk above max_q_len, a context above max_context_len
    c = make([3, 4], [40, 50], 8, 2, 128, 16, "bf16", seed=20)
    good = call(c).clone()
    for kw in (dict(max_q_len=3), dict(max_context_len=49)):
        err.zero_()
        out.fill_(5.0)
        call(c, out=out[:7], dev_err=err, **kw)
        assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS
        assert bool((out[3:7] == 0).all()) and torch.equal(out[:3], good[:3])
    # cu_q_lens that descends or leaves the rows: those rows stay
    for cu in ([0, 5, 3], [-2, 3, 7], [0, 3, 9]):
        c["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        err.zero_()
        out.fill_(5.0)
        call(c, out=out[:7], dev_err=err, max_q_len=9)
        assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS, cu
        assert bool((out[7:] == 5.0).all())


def test_rows_behind_the_last_sequence_stay():
    c = make([3, 0, 4], [40, 20, 50], 8, 2, 128, 16, "bf16", seed=21, extra_rows=6)
    out = torch.full((13, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    check(c, out=out)
    assert bool((out[7:] == 5.0).all())


def test_scores_far_apart_and_rising():
    """Scores that rise along the context by far more than the exponent range,
    and a single key far above all others."""
    for cache in ("bf16", "fp8_token"):
        c = make([4, 3], [700, 300], 8, 2, 128, 16, cache, seed=22)
        tab = c["tab"].cpu().long()
        if cache == "bf16":
            for t in range(0, 690, 10):
                c["kp"][int(tab[0, t // 16]), :, t % 16] *= (1 + t / 40)
        else:
            for t in range(0, 690, 10):
                c["ks"][int(tab[0, t // 16]), :, t % 16] *= (1 + t / 40)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(c, dev_err=err)
        ref, mag = reference(c)
        g = out.double().cpu()
        # scores reach some 2^9: their binary32 error (2^-24 of sums of that size, 2^3 in all) moves weights by up to 2^-10
        tol = R.tree_tolerance(ref, mag, cache != "bf16", cache == "fp8_token") + 2.0 ** -9 * mag
        assert bool(((g - ref).abs() <= tol).all())


def test_same_call_gives_the_same_bits_and_graphs_replay():
    for cache in ("bf16", "fp8"):
        c = make([8, 30], [3000, 900], 8, 2, 128, 16, cache, seed=23)
        want = call(c).clone()
        for _ in range(3):
            assert torch.equal(call(c), want)
        need = K.plan_tree(2, 8, 2, 128, 16, 30, c["tab"].shape[1] * 16,
                           cache_dtype=K.cache_dtype(c["kp"], c["ks"]))["workspace_bytes"]
        ws = torch.full((max(256, need),), 0xFF, dtype=torch.uint8, device="cuda")
        outs = [torch.zeros_like(want) for _ in range(2)]
        # two captured calls on one workspace, replayed in turn
        replays = [K.graphed(lambda o=o: call(c, out=o, workspace=ws)) for o in outs]
        for o in outs:
            o.zero_()
        for _ in range(2):
            for r in replays:
                r()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want)
        # replay after the lengths and the mask changed in place
        c["ctx"].copy_(torch.tensor([2900, 890], dtype=torch.int32))
        c["mask"].copy_(c["mask"] & 0x55555555)
        replays[0]()
        torch.cuda.synchronize()
        ref, mag = reference(c)
        close(c, outs[0], ref, mag)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
def test_many_ragged_trees_again_and_again(cache):
    """More CTAs than fit at once, rows that leave warps without work, calls
    back to back: every wait ends and every call gives the same bits."""
    ql = [1 + (7 * i) % 40 for i in range(48)]
    c = make(ql, [q + (131 * i) % 900 for i, q in enumerate(ql)], 32, 8, 128, 16, cache, seed=31)
    want = check(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [call(c, dev_err=err) for _ in range(40)]
    assert K.read_device_error(err) == K.PKV_OK
    for o in outs:
        assert torch.equal(o, want)


def test_on_another_stream_with_its_own_workspace():
    c = make([8, 30], [3000, 900], 8, 2, 128, 16, "bf16", seed=24)
    want = call(c).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [call(c, stream=side), call(c)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("shares", [0, 50])
def test_more_sequences_than_threads(shares):
    """Lengths are summed in chunks of the block's threads."""
    n = 700
    ql = [(i * 5) % 4 for i in range(n)]  # some without drafts
    c = make(ql, [q + (i * 11) % 150 + (q == 0) for i, q in enumerate(ql)], 4, 2, 64, 16, "bf16", seed=33)
    check(c, shares=shares)


def test_key_scales_of_either_sign_and_zero():
    c = make([5, 40], [90, 300], 12, 3, 128, 16, "fp8", seed=34)
    c["ks"][0] *= -1
    c["ks"][1] = 0
    check(c)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
def test_queries_of_any_size(cache):
    """Rows of zeros, of tiny and of large values; an infinite one is its own rows' matter."""
    c = make([6, 9], [90, 200], 8, 2, 128, 16, cache, seed=35)
    c["q"][0] = 0
    c["q"][1] *= 2.0 ** -100
    c["q"][2, :, ::7] *= 2.0 ** -30
    c["q"][3] *= 2.0 ** 3
    c["q"][7, 2, 5] = float("inf")
    c["q"][8, 1, 3] = float("nan")
    out = call(c)
    ref, mag = reference(c)
    hit = torch.zeros(15, 8, dtype=torch.bool)
    hit[7, 2] = hit[8, 1] = True
    g = out.double().cpu()
    # scores up to 2^8 here: 2^-24 of that, summed over 2^7 products, moves a weight by less than 2^-10;
    # E4M3 queries are off by 2^-17 of the row's largest, 2^-9 of a score unit in all
    tol = R.tree_tolerance(ref, mag, cache != "bf16", cache == "fp8_token") + 2.0 ** -8 * mag
    assert bool(((g - ref).abs() <= tol)[~hit].all())
    assert bool(g[hit].isnan().all())


def test_a_causal_chain_equals_prefill():
    """A tree that is a chain is a causal chunk: the prefill's result, to the roundings of both."""
    c = make([20, 50], [333, 1000], 8, 2, 128, 16, "bf16", seed=25)
    c["mask"] = torch.cat([K.tree_mask(list(range(-1, n - 1)), words=2)[0] for n in (20, 50)]).cuda()
    out = check(c)
    pre = K.paged_attention_prefill(c["q"], c["kp"], c["vp"], c["tab"], c["cu"], c["ctx"], c["scale"], c["most"])
    ref, mag = reference(c)
    close(c, pre, ref, mag)
    assert out.shape == pre.shape


def test_far_blocks_pass_32_bits():
    """Rows whose byte offsets in the pool pass 2^31 and 2^32."""
    nkv, bs, d = 8, 256, 128
    blocks = 9000  # 9000 * 8 * 256 * 128 * 2 bytes = 4.7e9
    kp = torch.zeros((blocks, nkv, bs, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    tab = torch.tensor([[8999, 0, 4200], [8500, 8998, -1]], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(3)
    cl, ql = [600, 300], [5, 3]
    slots = torch.cat([tab[i].cpu().long()[torch.arange(n) // bs] * bs + torch.arange(n) % bs
                       for i, n in enumerate(cl)]).int().cuda()
    k, v = (torch.randn(900, nkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    K.store_kvcache(k, v, kp, vp, slots)
    small = make(ql, cl, 32, nkv, d, bs, "bf16", seed=26)
    t2 = small["tab"].cpu().long()
    s2 = torch.cat([t2[i][torch.arange(n) // bs] * bs + torch.arange(n) % bs for i, n in enumerate(cl)]).int().cuda()
    K.store_kvcache(k, v, small["kp"], small["vp"], s2)
    want = check(small)
    out = K.paged_attention_tree(small["q"], kp, vp, tab, small["cu"], small["ctx"], small["mask"], small["scale"],
                                 small["most"])
    assert torch.equal(out, want)


def test_followed_by_a_copy_when_nothing_is_cut():
    """Every share is exactly one unit, so there is nothing to join: a copy queued behind the call still
    finds the finished rows, eagerly and replayed."""
    S, nkv = 6, 2
    c = make([16] * S, [16384] * S, 8, nkv, 128, 64, "bf16", 71)
    ref, mag = reference(c)
    plan = K.plan_tree(S, 8, nkv, 128, 64, c["most"], 16384, shares=S * nkv)
    ws = torch.empty(plan["workspace_bytes"], dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["q"])
    copy = torch.empty_like(out)

    def step():
        out.fill_(float("nan"))
        call(c, out=out, workspace=ws, shares=S * nkv, max_context_len=16384)
        copy.copy_(out)

    for run in (step, K.graphed(step)):
        for _ in range(5):
            copy.zero_()
            run()
            close(c, copy, ref, mag)


def put(c, seq, first, k, v):
    """Store rows k, v [n, nkv, d] as the tokens first .. first + n - 1 of a sequence."""
    bs = c["kp"].shape[2]
    t = torch.arange(first, first + k.shape[0])
    slots = (c["tab"][seq].cpu().long()[t // bs] * bs + t % bs).int().cuda()
    K.store_kvcache(k.bfloat16().cuda(), v.bfloat16().cuda(), c["kp"], c["vp"], slots, c["ks"], c["vs"])


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("drafts", [8, 24, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_maxima_that_grow_in_every_half_of_a_tile(d, drafts, cache):
    """Half of the heads meet scores that rise by more than 2^8 every 32 keys, the others scores that fall as
    fast, so what a tile has stored of its weights and results is scaled twice within each tile. V grows
    backwards by 2^8, so that the scaled parts weigh as much as the rest. Units of two copies (E4M3), of one
    row tile, and of two."""
    steps = 29
    base = 32 * steps
    c = make([drafts], [base + drafts], 8, 2, d, 16, cache, seed=41, words=2)
    g = torch.Generator().manual_seed(42)
    if cache == "fp8":
        c["ks"].fill_(1.0)
        c["vs"].fill_(1.0)
    n = base + drafts
    step = (torch.arange(n) // 32).clamp(max=steps - 1)
    k = torch.randn(n, 2, d, generator=g)
    k[:, :, 0] = (32.0 * (step - 14))[:, None]  # every one of them an E4M3 value
    back = steps - 1 - step
    size = torch.where(back == 0, 2.0 ** -8, torch.where(back == 1, 1.0, 256.0))
    v = torch.where(torch.rand(n, 2, d, generator=g) < 0.5, -1.0, 1.0) * size[:, None, None]
    put(c, 0, 0, k, v)
    # a step is 32 * 2.25 / sqrt(d) * log2(e) = 9.2 (d 128) or 13 (d 64) powers of two, the others' share below 1
    q = 0.25 * torch.randn(drafts, 8, d, generator=g)
    q[:, :, 0] = torch.where(torch.arange(8) % 2 == 0, 2.25, -2.25)
    c["q"].copy_(q.bfloat16())
    for shares in (0, 1):
        check(c, shares=shares)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("gap", [20, 24])
@pytest.mark.parametrize("n,drafts", [(32768, 4), (65536, 2), (2048, 36)])
def test_one_key_far_above_a_long_flat_rest(n, drafts, gap, cache):
    """One key's weight is 2^gap times every other's and its V is zero, so the small weights are the answer.
    All of V is positive: errors of one sign add up. In one share (every weight next to the large one) and
    in many."""
    c = make([drafts], [n], 4, 1, 128, 256, cache, seed=51, words=2)
    g = torch.Generator().manual_seed(52)
    if cache == "fp8":
        c["ks"].fill_(2.0 ** -6)
        c["vs"].fill_(2.0 ** -8)
    # queries of +-1 are exact in every operand type, so are the binary32 scores, nearly
    q = torch.where(torch.rand(drafts, 4, 128, generator=g) < 0.5, -1.0, 1.0)
    q[:, :, :64] = 1.0
    c["q"].copy_(q.bfloat16())
    k = 0.25 * torch.randn(n, 1, 128, generator=g)
    k[5, :, :64] = gap * math.log(2) * math.sqrt(128) / 64
    k[5, :, 64:] = 0
    v = 0.5 + torch.rand(n, 1, 128, generator=g)
    v[5] = 0
    put(c, 0, 0, k, v)
    ref, mag = reference(c)
    assert float(mag.min()) > 0
    for shares in (1, 0):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(c, shares=shares, dev_err=err)
        assert K.read_device_error(err) == K.PKV_OK
        # f16 weights below 2^-21 of the largest: each off by at most 2^-32 of it (a sum of at least 1), V at most 1.5 (1 + 2^-4)
        small = 1.6 * n * 2.0 ** -32 if cache == "fp8" else 0.0
        g64 = out.double().cpu()
        tol = R.tree_tolerance(ref, mag, cache != "bf16", cache == "fp8_token") + small * (1 + R.U_BF16)
        off = ((g64 - ref).abs() / tol)
        assert bool((off <= 1).all()), f"{shares} shares: off by {float(off.max()):.3g} tolerances"


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("drafts", [6, 24, 40])
def test_rows_that_see_nothing_are_zeros_whatever_their_query_holds(drafts, bad, cache):
    """No token before the drafts and an empty mask row: zeros, even for a query that is not finite. The same
    query where something is seen gives NaN, in its own row and head alone."""
    c = make([drafts, drafts], [drafts, drafts], 8, 2, 128, 16, cache, seed=61, words=2)
    c["mask"][2] = 0
    clean = check(c)
    for row in (2, drafts - 1, drafts + 3):
        c["q"][row, 1, ::2] = bad
        c["q"][row, 6] = bad
    out = call(c)
    hit = torch.zeros(2 * drafts, 8, dtype=torch.bool)
    for row in (drafts - 1, drafts + 3):
        hit[row, 1] = hit[row, 6] = True
    assert bool((out[2] == 0).all())
    assert bool(out.cpu()[hit].isnan().all())
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])


def test_rows_of_lost_sequences_stay_and_the_others_are_right():
    """cu_q_lens that descends or leaves the rows: the sequence's own rows are not written, the other
    sequence's are as ever."""
    for cu, ok, rows in (([0, 5, 3], 0, (0, 5)), ([-2, 3, 7], 1, (3, 7)), ([0, 3, 9], 0, (0, 3))):
        c = make([3, 4], [40, 50], 8, 2, 128, 16, "bf16", seed=20)
        c["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(c["q"], 5.0)
        call(c, out=out, dev_err=err, max_q_len=9)
        assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS, cu
        a, b = rows
        assert bool((out[:a] == 5.0).all()) and bool((out[b:] == 5.0).all()), cu
        one = dict(c, q=c["q"][a:b], mask=c["mask"][a:b], tab=c["tab"][ok:ok + 1], ctx=c["ctx"][ok:ok + 1],
                   cu=torch.tensor([0, b - a], dtype=torch.int32))
        ref, mag = reference(one)
        close(c, out[a:b], ref, mag, str(cu))


def test_a_causal_chain_equals_prefill_row_by_row():
    """Both calls are within the tolerance of the formula, so within twice that of each other."""
    c = make([20, 50], [333, 1000], 8, 2, 128, 16, "bf16", seed=25)
    c["mask"] = torch.cat([K.tree_mask(list(range(-1, n - 1)), words=2)[0] for n in (20, 50)]).cuda()
    out = call(c)
    pre = K.paged_attention_prefill(c["q"], c["kp"], c["vp"], c["tab"], c["cu"], c["ctx"], c["scale"], c["most"])
    ref, mag = reference(c)
    tol = R.tree_tolerance(ref, mag, False, False)
    assert bool(((out.double() - pre.double()).abs().cpu() <= 2 * tol).all())


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("ql", [[4, 9, 1, 16, 12], [20, 32, 17, 5, 25]])
@pytest.mark.parametrize("shares", [1, 2, 3, 10, 37, 300])
def test_any_cut_of_units_of_one_row_tile(shares, ql, cache):
    """As test_any_cut_of_the_work, with at most 128 rows: units of one copy of their rows and of two."""
    c = make(ql, [2500, 70, 1, 1111, 180], 8, 2, 128, 16, cache, seed=11) if ql[2] == 1 else \
        make(ql, [2500, 70, 40, 1111, 180], 8, 2, 128, 16, cache, seed=11)
    p = K.plan_tree(5, 8, 2, 128, 16, c["most"], 2512, cache_dtype=K.cache_dtype(c["kp"], c["ks"]), shares=shares)
    ws = torch.full((max(256, p["workspace_bytes"]),), 0xFF, dtype=torch.uint8, device="cuda")
    check(c, shares=shares, workspace=ws)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("ql", [[12, 16], [12, 30]])
@pytest.mark.parametrize("shares", [0, 1, 7])
def test_what_is_masked_does_not_reach_a_row_of_one_row_tile(shares, ql, cache):
    """As test_what_is_masked_does_not_reach_a_row, with units of one row tile and of two copies."""
    c = make(ql, [50, 200], 8, 2, 128, 16, cache, seed=17)
    clean = call(c, shares=shares).clone()
    tab = c["tab"].cpu().long()
    for seq, u in ((0, 3), (1, 7), (1, 11)):
        t = int(c["ctx"][seq]) - ql[seq] + u
        blk, off = int(tab[seq, t // 16]), t % 16
        if cache == "bf16":
            c["kp"][blk, :, off, 1] = float("nan")
            c["vp"][blk, 0, off] = float("inf")
            c["vp"][blk, 1, off, 5] = float("nan")
        else:
            c["kp"][blk, :, off, 1] = 0x7F
            c["vp"][blk, 0, off] = 0x7F
            c["vp"][blk, 1, off, 5] = 0x7F
            if cache == "fp8_token":
                c["vs"][blk, 1, off] = float("inf")
    out = call(c, shares=shares)
    saw = torch.zeros(sum(ql), dtype=torch.bool)
    bits = R.sees(c["mask"], 32)
    saw[:12] = bits[:12, 3]
    saw[12:] = bits[12:, 7] | bits[12:, 11]
    assert bool(saw.any()) and not bool(saw.all())
    assert torch.equal(out.cpu()[~saw], clean.cpu()[~saw])
    assert bool(out.cpu()[saw].isnan().any(-1).all())


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("d", [64, 128])
def test_trees_that_are_small_against_the_bound(d, cache):
    """max_q_len allows units of two row tiles, of which these trees fill a part of the first."""
    check(make([8, 1, 5, 30, 3], [500, 60, 300, 1000, 3], 8, 2, d, 16, cache, seed=81, words=4), max_q_len=128)
