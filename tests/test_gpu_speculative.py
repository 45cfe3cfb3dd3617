"""A speculative decoding step, its operators run together as a server runs them.

Prompts and drafts are normed, rotated and stored; the drafts' tree attends;
the accepted path's rows are moved together; the next token is decoded. The
cache must then be, bit for bit, the one that holds the accepted tokens alone.
"""

import math

import pytest
import torch

import spec_reference as R
from paged_kv_cache_482_b200 import pagedkv as K
from paged_kv_cache_482_b200 import workloads as W

pytestmark = pytest.mark.gpu

NQ, NKV, D, BS, EPS = 8, 2, 128, 16, 1e-6
PROMPTS = [37, 5, 130]
PARENTS = [[-1, 0, 0, 1, 2, 3, 5, 5], [-1, -1, 1], [-1] + [max(0, j - 3) for j in range(1, 40)]]
PATHS = [[0, 1, 3, 5, 7], [], None]  # None: the third tree's longest chain


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def chain(parents):
    """The path to the last draft."""
    path = [len(parents) - 1]
    while parents[path[-1]] >= 0:
        path.append(parents[path[-1]])
    return path[::-1]


class Cache:
    """Pools and tables with room for every token of the step."""

    def __init__(self, cache, seed):
        g = torch.Generator().manual_seed(seed)
        most = [p + len(t) + 1 for p, t in zip(PROMPTS, PARENTS)]
        need = [-(-n // BS) for n in most]
        blocks = sum(need) + 2
        perm = torch.randperm(blocks, generator=g)
        self.tab = torch.full((3, max(need)), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.tab[i, :n] = perm[at:at + n].int()
            at += n
        shape = (blocks, NKV, BS, D)
        self.ks = self.vs = None
        if cache == "bf16":
            self.k = torch.full(shape, W.CANARY_BF16, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        else:
            self.k = torch.full(shape, W.CANARY_FP8, dtype=torch.uint8, device="cuda")
            if cache == "fp8":
                self.ks, self.vs = torch.tensor([[0.01, 0.02], [0.02, 0.01]], device="cuda")
            else:
                self.ks, self.vs = (torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2))
        self.v = self.k.clone()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dtab = self.tab.cuda()

    def slots(self, places):
        """places[i]: token positions of sequence i."""
        return i32([int(self.tab[i, t // BS]) * BS + t % BS for i, p in enumerate(places) for t in p])

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs, dev_err=self.err)


class Model:
    """What a layer gives: the QKV rows of tokens, weights, the rotary table."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        n = sum(PROMPTS) + sum(map(len, PARENTS)) + 3
        self.qkv = torch.randn(n, (NQ + 2 * NKV) * D, generator=g).bfloat16().cuda()
        self.qw, self.kw = (1 + 0.2 * torch.randn(2, D, generator=g)).bfloat16().cuda()
        self.cs = W.rope_cache(400, D).cuda()

    def store(self, c, rows, positions, places):
        q, k, v = (x.unflatten(1, (-1, D)) for x in self.qkv[rows].split([NQ * D, NKV * D, NKV * D], 1))
        return K.store_kvcache_norm_rope(k, v, c.k, c.v, c.slots(places), i32(positions), self.cs, self.kw, EPS, q=q,
                                         q_weight=self.qw, **c.scales())


def rows_of(c, lens):
    cu = i32([0] + torch.tensor(lens).cumsum(0).tolist())
    return K.load_kvcache(c.k, c.v, c.dtab, cu, total_rows=sum(lens), **c.scales())


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp8_token"])
def test_step(cache):
    m, scale = Model(1), 1 / math.sqrt(D)
    paths = [p if p is not None else chain(t) for p, t in zip(PATHS, PARENTS)]
    drafts = [len(t) for t in PARENTS]
    first = [sum(PROMPTS) + sum(drafts[:i]) for i in range(3)]  # rows of the drafts in m.qkv
    bonus = sum(PROMPTS) + sum(drafts)

    def prompt(c):
        m.store(c, torch.arange(sum(PROMPTS)), [t for n in PROMPTS for t in range(n)], [range(n) for n in PROMPTS])

    # the speculative step
    a = Cache(cache, 2)
    prompt(a)
    made = [K.tree_mask(t, words=2) for t in PARENTS]
    mask = torch.cat([x for x, _ in made]).cuda()
    positions = [p + int(x) for p, (_, depth) in zip(PROMPTS, made) for x in depth]
    q = m.store(a, torch.arange(first[0], bonus), positions, [range(p, p + n) for p, n in zip(PROMPTS, drafts)])
    ctx = [p + n for p, n in zip(PROMPTS, drafts)]
    cu = i32([0] + torch.tensor(drafts).cumsum(0).tolist())
    out = K.paged_attention_tree(q, a.k, a.v, a.dtab, cu, i32(ctx), mask, scale, max(drafts), **a.scales())
    ref, mag = R.tree_attention(q, R.cache_values(a.k, a.ks), R.cache_values(a.v, a.vs), a.tab, cu, i32(ctx), mask,
                                scale)
    tol = R.tree_tolerance(ref, mag, cache != "bf16", cache == "fp8_token")
    assert bool(((out.double().cpu() - ref).abs() <= tol).all())
    most = max(map(len, paths))
    K.compact_kvcache(a.k, a.v, a.dtab, cu, i32(ctx), i32([p + [0] * (most - len(p)) for p in paths]),
                      i32([len(p) for p in paths]), **a.scales())

    # the accepted tokens alone
    b = Cache(cache, 3)
    prompt(b)
    m.store(b, torch.tensor([f + j for f, p in zip(first, paths) for j in p]),
            [n + j for n, p in zip(PROMPTS, paths) for j in range(len(p))],
            [range(n, n + len(p)) for n, p in zip(PROMPTS, paths)])
    lens = [n + len(p) for n, p in zip(PROMPTS, paths)]
    for x, y in zip(rows_of(a, lens), rows_of(b, lens)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))

    # the next token, on both
    outs = []
    for c in (a, b):
        q1 = m.store(c, torch.arange(bonus, bonus + 3), lens, [[n] for n in lens])
        outs.append(K.paged_attention_decode(q1, c.k, c.v, c.dtab, i32([n + 1 for n in lens]), scale, **c.scales()))
    assert torch.equal(*outs)
    # a single token is a tree too
    one = K.paged_attention_tree(q1, b.k, b.v, b.dtab, i32([0, 1, 2, 3]), i32([n + 1 for n in lens]), i32([[1]] * 3),
                                 scale, 1, **b.scales())
    ref, mag = R.tree_attention(q1, R.cache_values(b.k, b.ks), R.cache_values(b.v, b.vs), b.tab, i32([0, 1, 2, 3]),
                                i32([n + 1 for n in lens]), i32([[1]] * 3), scale)
    tol = R.tree_tolerance(ref, mag, cache != "bf16", cache == "fp8_token")
    assert bool(((one.double().cpu() - ref).abs() <= tol).all())
    for c in (a, b):
        assert K.read_device_error(c.err) == K.PKV_OK


def test_step_as_one_graph():
    """Store, tree and compaction captured together and replayed from a fresh cache."""
    m, scale = Model(4), 1 / math.sqrt(D)
    drafts = [len(t) for t in PARENTS]
    paths = [p if p is not None else chain(t) for p, t in zip(PATHS, PARENTS)]
    c = Cache("fp8_token", 5)
    m.store(c, torch.arange(sum(PROMPTS)), [t for n in PROMPTS for t in range(n)], [range(n) for n in PROMPTS])
    made = [K.tree_mask(t, words=2) for t in PARENTS]
    mask = torch.cat([x for x, _ in made]).cuda()
    rows = torch.arange(sum(PROMPTS), sum(PROMPTS) + sum(drafts))
    q, k, v = (x.unflatten(1, (-1, D)) for x in m.qkv[rows].split([NQ * D, NKV * D, NKV * D], 1))
    slots = c.slots([range(p, p + n) for p, n in zip(PROMPTS, drafts)])
    pos = i32([p + int(x) for p, (_, depth) in zip(PROMPTS, made) for x in depth])
    ctx, cu = i32([p + n for p, n in zip(PROMPTS, drafts)]), i32([0] + torch.tensor(drafts).cumsum(0).tolist())
    most = max(map(len, paths))
    acc, num = i32([p + [0] * (most - len(p)) for p in paths]), i32([len(p) for p in paths])
    need = K.plan_tree(3, NQ, NKV, D, BS, max(drafts), c.tab.shape[1] * BS, cache_dtype=K.cache_dtype(c.k, c.ks))
    ws = torch.empty(max(256, need["workspace_bytes"]), dtype=torch.uint8, device="cuda")
    q_out, out = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape, dtype=q.dtype, device="cuda")

    def step():
        K.store_kvcache_norm_rope(k, v, c.k, c.v, slots, pos, m.cs, m.kw, EPS, q=q, q_weight=m.qw, q_out=q_out,
                                  **c.scales())
        K.paged_attention_tree(q_out, c.k, c.v, c.dtab, cu, ctx, mask, scale, max(drafts), out=out, workspace=ws,
                               **c.scales())
        K.compact_kvcache(c.k, c.v, c.dtab, cu, ctx, acc, num, **c.scales())

    step()
    want = [x.clone() for x in (q_out, out, c.k, c.v, c.ks, c.vs)]
    replay = K.graphed(step)
    for x in (q_out, out):
        x.zero_()
    replay()
    replay()
    torch.cuda.synchronize()
    assert K.read_device_error(c.err) == K.PKV_OK
    for x, y in zip((q_out, out, c.k, c.v), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for x, y in zip((c.ks, c.vs), want[4:]):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
