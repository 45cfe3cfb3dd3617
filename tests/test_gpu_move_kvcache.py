"""compact_kvcache and load_kvcache on the GPU: rows moved or read back bit for bit."""

import pytest
import torch

from paged_kv_cache_482_b200 import pagedkv as K

pytestmark = pytest.mark.gpu


def pools(blocks, nkv, bs, d, cache, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (blocks, nkv, bs, d)
    if cache == "bf16":
        return [torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2)] + [None, None]
    codes = [torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    n = (nkv,) if cache == "fp8" else shape[:3]
    return codes + [(torch.rand(n, generator=g) + 0.1).cuda() for _ in range(2)]


def tables(lens, bs, blocks, seed):
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(blocks, generator=g)
    width = max(1, max(-(-n // bs) for n in lens))
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(lens):
        m = -(-n // bs)
        t[i, :m] = perm[at:at + m].int()
        at += m
    return t.cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32([0] + torch.tensor(lens).cumsum(0).tolist())


def blocks_for(lens, bs):
    return sum(-(-n // bs) for n in lens) + 2


def compact_want(p, tab, ql, cl, lists, bs, skip=()):
    out = [None if x is None else x.cpu().clone() for x in p]
    src = [None if x is None else x.cpu() for x in p]
    t = tab.cpu().long()
    move = [0, 1] + ([2, 3] if p[2] is not None and p[2].dim() == 3 else [])
    for i, keep in enumerate(lists):
        if i in skip:
            continue
        base = cl[i] - ql[i]
        for j, a in enumerate(keep):
            for k in move:
                out[k][t[i, (base + j) // bs], :, (base + j) % bs] = src[k][t[i, (base + a) // bs], :, (base + a) % bs]
    return out


def run_compact(p, tab, ql, cl, lists, most=None, err=None, stream=None):
    most = most or max(1, max(len(x) for x in lists))
    acc = i32([list(x) + [-7] * (most - len(x)) for x in lists])
    K.compact_kvcache(p[0], p[1], tab, cu_of(ql), i32(cl), acc, i32([len(x) for x in lists]), k_scale=p[2],
                      v_scale=p[3], dev_err=err, stream=stream)


def same(got, want):
    for a, b in zip(got, want):
        if a is not None:
            assert torch.equal(a.cpu().view(torch.uint8 if a.element_size() == 1 else torch.int16 if a.element_size() == 2
                                            else torch.int32), b.view(torch.uint8 if b.element_size() == 1 else
                                                                      torch.int16 if b.element_size() == 2 else torch.int32))


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("nkv,d,bs", [(8, 128, 16), (2, 64, 256), (3, 24, 5), (1, 8, 8)])
def test_compact_moves_rows_exactly(cache, nkv, d, bs):
    g = torch.Generator().manual_seed(nkv * d)
    ql = [8, 64, 1, 33, 5, 300, 2]
    cl = [n + int(torch.randint(0, 90, (1,), generator=g)) for n in ql]
    cl[4] = 5  # nothing but drafts
    lists = [[0, 2, 3, 7], list(range(1, 64)), [0], [], [4], list(range(0, 300, 2)), [0, 1]]
    p = pools(blocks_for(cl, bs), nkv, bs, d, cache, 3)
    tab = tables(cl, bs, p[0].shape[0], 4)
    want = compact_want(p, tab, ql, cl, lists, bs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_compact(p, tab, ql, cl, lists, err=err)
    assert K.read_device_error(err) == K.PKV_OK
    same(p, want)


def test_compact_leaves_bad_sequences_alone():
    bs, ql = 16, [4] * 9
    cl = [20] * 9
    lists = [[0, 2], [2, 1], [1, 1], [3, 4], [-1, 2], [1, 3], [1, 3], [0, 1], [1, 2]]
    p = pools(blocks_for(cl, bs), 2, bs, 64, "fp8_token", 5)
    tab = tables(cl, bs, p[0].shape[0], 6)
    tab[5, 1] = p[0].shape[0]  # a block outside the pool
    tab[6, 1] = -1
    want = compact_want(p, tab, ql, cl, lists, bs, skip=(1, 2, 3, 4, 5, 6))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_compact(p, tab, ql, cl, lists, err=err)
    assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS
    same(p, want)
    # lengths out of range, each sequence on its own
    for cu, ctx, n in (([0, 4], 3, 2), ([0, 4], 33, 2), ([0, 4], 20, 5), ([0, 4], 20, -1), ([4, 0], 20, 2),
                       ([-1, 3], 20, 2), ([0, 1], 20, 2), ([0, 4], 20, 3)):
        before = [x.clone() for x in p]
        err.zero_()
        K.compact_kvcache(p[0], p[1], tab[:1].contiguous(), i32(cu), i32([ctx]), i32([[1, 3]]), i32([n]),
                          k_scale=p[2], v_scale=p[3], dev_err=err)
        assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS, (cu, ctx, n)
        same(p, [x.cpu() for x in before])


def test_compact_captured_replays_on_new_lists():
    bs, ql, cl = 16, [8, 8], [30, 41]
    p = pools(blocks_for(cl, bs), 4, bs, 128, "bf16", 7)
    tab = tables(cl, bs, p[0].shape[0], 8)
    acc, n, cu, ctx = i32([[0, 1, 2]] * 2), i32([0, 0]), cu_of(ql), i32(cl)
    replay = K.graphed(lambda: K.compact_kvcache(p[0], p[1], tab, cu, ctx, acc, n))
    for lists in ([[0, 3, 5], [1]], [[2], [0, 6, 7]]):
        want = compact_want(p, tab, ql, cl, lists, bs)
        acc.copy_(i32([x + [0] * (3 - len(x)) for x in lists]))
        n.copy_(i32([len(x) for x in lists]))
        replay()
        torch.cuda.synchronize()
        same(p, want)


def load_want(p, tab, lens, starts, bs):
    out = []
    for x, s in ((p[0], p[2]), (p[1], p[3])):
        if x.dtype == torch.bfloat16:
            y = x.cpu()
        else:
            y = x.cpu().view(torch.float8_e4m3fn).float()
            y = (y * (s.cpu()[..., None] if s.dim() == 3 else s.cpu()[None, :, None, None])).bfloat16()
        rows = []
        for i, n in enumerate(lens):
            t = starts[i] + torch.arange(n)
            rows.append(y[tab.cpu().long()[i][t // bs], :, t % bs])
        out.append(torch.cat(rows))
    return out


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("nkv,d,bs", [(8, 128, 16), (2, 64, 256), (3, 24, 5), (1, 8, 8)])
@pytest.mark.parametrize("with_starts", [False, True])
def test_load_reads_rows_exactly(cache, nkv, d, bs, with_starts):
    lens = [1, 0, 37, 130, 0, 0, 255, 16, 3]
    starts = [5, 2, 0, 17, 0, 1, 3, 16, 250] if with_starts else [0] * 9
    held = [a + b for a, b in zip(lens, starts)]
    p = pools(blocks_for(held, bs), nkv, bs, d, cache, 9)
    tab = tables(held, bs, p[0].shape[0], 10)
    total = sum(lens)
    k, v = (torch.full((total + 5, nkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = K.load_kvcache(p[0], p[1], tab, cu_of(lens), k_out=k, v_out=v, starts=i32(starts) if with_starts else None,
                         k_scale=p[2], v_scale=p[3], dev_err=err)
    assert K.read_device_error(err) == K.PKV_OK and got[0] is k and got[1] is v
    for g, w in zip(got, load_want(p, tab, lens, starts, bs)):
        assert torch.equal(g[:total].cpu().view(torch.int16), w.view(torch.int16))
        assert bool((g[total:] == 3.0).all()), "rows of no sequence"


def test_load_allocates_and_bad_input_is_reported():
    lens, bs = [20, 30], 16
    p = pools(blocks_for(lens, bs), 2, bs, 64, "bf16", 11)
    tab = tables(lens, bs, p[0].shape[0], 12)
    want = load_want(p, tab, lens, [0, 0], bs)
    k, v = K.load_kvcache(p[0], p[1], tab, cu_of(lens), total_rows=50)
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    assert K.load_kvcache(p[0], p[1], tab, i32([0, 0, 0]), total_rows=0)[0].shape == (0, 2, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = tab.clone()
    bad[0, 1], bad[1, 0] = p[0].shape[0], -1
    k, v = K.load_kvcache(p[0], p[1], bad, cu_of(lens), total_rows=50, dev_err=err)
    assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS
    zero = torch.zeros(50, dtype=torch.bool)
    zero[16:20] = zero[20:36] = True
    assert bool((k.cpu()[zero] == 0).all()) and torch.equal(k.cpu()[~zero], want[0][~zero])
    for starts in ([-1, 0], [0, 5]):  # tokens outside the table
        err.zero_()
        K.load_kvcache(p[0], p[1], tab, cu_of(lens), total_rows=50, starts=i32(starts), dev_err=err)
        assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS
    for cu in ([0, 40, 30], [-3, 20, 50], [0, 20, 60]):
        err.zero_()
        K.load_kvcache(p[0], p[1], tab, i32(cu), total_rows=50, dev_err=err)
        assert K.read_device_error(err) == K.PKV_ERR_DEVICE_BOUNDS, cu
