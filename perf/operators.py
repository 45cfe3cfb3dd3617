"""Cases of four operators around a paged KV cache: a speculative decoding step.

A step of speculative decoding over the paged cache normalises and rotates the
drafted tokens' queries and keys and stores them (``norm_rope``), attends a
tree of drafted tokens over the cached context (``tree``), and moves the rows
of the accepted drafts together (``compact``); a request's cached rows are read
back as bf16, for instance to hand the request to another worker (``load``).

``run`` computes an operator in plain torch operations, or, where ``own`` is
true, through ``paged_kv_cache_482_b200.pagedkv``. Lengths follow from the
case alone, values, block tables and trees from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one request's next token: the smallest call an engine makes per layer
        dict(name="norm_rope_one", op="norm_rope", n=1, nq=32, nkv=8, d=128, bs=256, cache="bf16", style=0, skip=0),
        # a prefill step's 8192 tokens, read in place from the fused projection's output
        dict(name="norm_rope_prefill", op="norm_rope", n=8192, nq=32, nkv=8, d=128, bs=256, cache="bf16", style=0,
             skip=0),
        # an odd number of tokens into an E4M3 cache with a scale per token, adjacent pairs, cached prefix tokens skipped
        dict(name="norm_rope_fp8_token", op="norm_rope", n=2777, nq=16, nkv=8, d=128, bs=16, cache="fp8_token",
             style=1, skip=5),
        # one request with eight drafts on a short context: latency
        dict(name="tree_one", op="tree", seqs=1, dlo=8, dhi=8, clo=500, chi=500, nq=32, nkv=8, d=128, bs=256,
             cache="bf16"),
        # a serving batch: ragged trees and contexts
        dict(name="tree_batch", op="tree", seqs=64, dlo=1, dhi=32, clo=100, chi=2048, nq=32, nkv=8, d=128, bs=256,
             cache="bf16"),
        # long contexts, E4M3 cache, small pages
        dict(name="tree_long_fp8", op="tree", seqs=16, dlo=16, dhi=16, clo=16384, chi=32768, nq=32, nkv=8, d=128,
             bs=16, cache="fp8"),
        # wide trees: the rows of one KV head fill several tensor-core tiles
        dict(name="tree_wide", op="tree", seqs=32, dlo=40, dhi=64, clo=1000, chi=4096, nq=32, nkv=8, d=128, bs=256,
             cache="bf16"),
        # small heads, eight queries to a KV head, a scale per token, odd lengths
        dict(name="tree_fp8_token_d64", op="tree", seqs=37, dlo=5, dhi=21, clo=63, chi=3001, nq=16, nkv=2, d=64,
             bs=16, cache="fp8_token"),
        # after one request's verification
        dict(name="compact_one", op="compact", seqs=1, dlo=8, dhi=8, nq=32, nkv=8, d=128, bs=256, cache="bf16"),
        # after a batch's verification, wide trees, small pages
        dict(name="compact_batch", op="compact", seqs=256, dlo=33, dhi=64, nq=32, nkv=8, d=128, bs=16,
             cache="fp8_token"),
        # a short request's rows
        dict(name="load_one", op="load", seqs=1, clo=133, chi=133, nkv=8, d=128, bs=256, cache="bf16"),
        # the rows of a batch's requests, E4M3 cache, small pages
        dict(name="load_batch_fp8", op="load", seqs=16, clo=2048, chi=8192, nkv=8, d=128, bs=16, cache="fp8"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo .. hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "tree", "tree", "tree", "compact", "load"])
    nq, nkv = rng.choice([(32, 8), (16, 8), (16, 2), (8, 1), (4, 4)])
    c = dict(op=op, nq=nq, nkv=nkv, d=rng.choice([64, 128, 128]), bs=rng.choice([8, 16, 64, 256]),
             cache=rng.choice(["bf16", "bf16", "fp8", "fp8_token"]))
    if op == "norm_rope":
        return dict(c, n=_log(rng, 1, 8192), style=rng.choice([0, 1]), skip=rng.choice([0, 0, 3]))
    if op == "tree":
        dhi = _log(rng, 1, 64)
        chi = _log(rng, dhi + 1, 32768)
        clo = rng.randint(max(dhi, chi // 3), chi)
        # at most the cached rows and the scores of the largest listed cases
        seqs = _log(rng, 1, max(1, min(64, 400000 // chi, 6000000 // (chi * dhi))))
        return dict(c, seqs=seqs, dlo=rng.randint(1, dhi), dhi=dhi, clo=clo, chi=chi)
    if op == "compact":
        dhi = _log(rng, 2, 64)
        return dict(c, seqs=_log(rng, 1, 256), dlo=rng.randint(1, dhi), dhi=dhi)
    chi = _log(rng, 2, 8192)
    return dict({k: v for k, v in c.items() if k != "nq"}, seqs=_log(rng, 1, max(1, min(64, 80000 // chi))),
                clo=rng.randint(1, chi), chi=chi)


def _lens(case):
    """(drafted tokens, context lengths counting them) of every sequence: the case's alone."""
    r = random.Random("lens")
    if case["op"] == "compact":
        q = [r.randint(case["dlo"], case["dhi"]) for _ in range(case["seqs"])]
        return q, [n + r.randint(0, 160) for n in q]
    if case["op"] == "load":
        return None, [r.randint(case["clo"], case["chi"]) for _ in range(case["seqs"])]
    q = [r.randint(case["dlo"], case["dhi"]) for _ in range(case["seqs"])]
    return q, [max(n, r.randint(case["clo"], case["chi"])) for n in q]


def _accepted_lens(case):
    """How many of its drafts each sequence keeps: none, in a batch, of some."""
    r = random.Random("accepted")
    return [r.randint(1 if i == 0 else 0, min(n, 9)) for i, n in enumerate(_lens(case)[0])]


def _row_bytes(case):
    """Bytes of one cached (token, KV head) row of K or V."""
    return {"bf16": 2 * case["d"], "fp8": case["d"], "fp8_token": case["d"] + 4}[case["cache"]]


def work(case):
    op, d = case["op"], case["d"]
    if op == "norm_rope":
        n, nq, nkv = case["n"], case["nq"], case["nkv"]
        return {"bytes": n * (4 * nq * d + 2 * nkv * 2 * d + 2 * nkv * _row_bytes(case) + 4 * d + 8),
                "flops": n * (nq + nkv) * d * 7}
    if op == "tree":
        ql, cl = _lens(case)
        nq, nkv = case["nq"], case["nkv"]
        return {"bytes": sum(cl) * 2 * nkv * _row_bytes(case) + sum(ql) * 4 * nq * d,
                "flops": sum(4 * nq * d * a * b for a, b in zip(ql, cl))}
    if op == "compact":
        return {"bytes": sum(_accepted_lens(case)) * case["nkv"] * 4 * _row_bytes(case), "flops": 0}
    cl = _lens(case)[1]
    return {"bytes": sum(cl) * case["nkv"] * 2 * (_row_bytes(case) + 2 * d), "flops": sum(cl) * case["nkv"] * 2 * d}


class _State:
    pass


def _pools(case, blocks, gen):
    """K and V pools full of other tokens' rows, and their scales."""
    s = _State()
    shape = (blocks, case["nkv"], case["bs"], case["d"])
    s.k_scale = s.v_scale = None
    s.k_cache = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    s.v_cache = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    if case["cache"] != "bf16":
        s.k_cache = (s.k_cache * 64).to(torch.float8_e4m3fn)
        s.v_cache = (s.v_cache * 64).to(torch.float8_e4m3fn)
        n = (case["nkv"],) if case["cache"] == "fp8" else shape[:3]
        s.k_scale = (torch.rand(n, generator=gen, device=DEV) + 0.5) / 64
        s.v_scale = (torch.rand(n, generator=gen, device=DEV) + 0.5) / 64
    s.dev_err = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _tables(case, lens, gen):
    """Scattered blocks for every sequence; -1 behind a sequence's last one."""
    bs = case["bs"]
    need = torch.tensor([-(-n // bs) for n in lens])
    blocks = int(need.sum()) + 3
    perm = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    first = (torch.cumsum(need, 0) - need).to(DEV)
    j = torch.arange(int(need.max()), device=DEV)
    tab = perm[(first[:, None] + j).clamp(max=blocks - 1)]
    return torch.where(j < need.to(DEV)[:, None], tab, -1).to(torch.int32).contiguous(), blocks


def _cu(lens):
    return torch.tensor([0] + torch.cumsum(torch.tensor(lens), 0).tolist(), dtype=torch.int32, device=DEV)


def _trees(seqs, most, gen):
    """[seqs, most, most] bool: draft t sees draft u (itself and its ancestors); a node's parent is one of the eight before it."""
    r = torch.rand((seqs, most), generator=gen, device=DEV).cpu()
    sees = torch.zeros((seqs, most, most), dtype=torch.bool)
    at = torch.arange(seqs)
    for t in range(most):
        parent = t - 1 - (r[:, t] * min(t + 1, 8)).long()
        if t:
            sees[:, t] = sees[at, parent.clamp(min=0)] & (parent >= 0)[:, None]
        sees[:, t, t] = True
    return sees.to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, bs, d = case["op"], case["bs"], case["d"]
    if op == "norm_rope":
        n, nq, nkv = case["n"], case["nq"], case["nkv"]
        s = _pools(case, -(-n // bs) + 3, gen)
        qkv = torch.randn((n, (nq + 2 * nkv) * d), generator=gen, device=DEV, dtype=torch.bfloat16) * 1.5
        s.q, s.k, s.v = (x.view(n, -1, d) for x in qkv.split([nq * d, nkv * d, nkv * d], 1))
        s.q_out = torch.empty((n, nq, d), dtype=torch.bfloat16, device=DEV)
        s.q_weight, s.k_weight = (1 + 0.2 * torch.randn((2, d), generator=gen, device=DEV)).bfloat16()
        s.slots = torch.randperm(s.k_cache.shape[0] * bs, generator=gen, device=DEV)[:n].to(torch.int32)
        if case["skip"]:  # tokens whose block already holds them
            s.slots[:: case["skip"]] = -1
        top = 32768
        s.positions = torch.randint(0, top, (n,), generator=gen, device=DEV, dtype=torch.int32)
        angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * \
            (1e6 ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d))
        s.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s.style = case["style"]
        s.op = op
        return s
    ql, cl = _lens(case)
    tables, blocks = _tables(case, cl, gen)
    s = _pools(case, blocks, gen)
    s.op, s.tables = op, tables
    s.ctx = torch.tensor(cl, dtype=torch.int32, device=DEV)
    if op == "load":
        s.cu = _cu(cl)
        s.k_out = torch.empty((sum(cl), case["nkv"], d), dtype=torch.bfloat16, device=DEV)
        s.v_out = torch.empty_like(s.k_out)
        return s
    s.cu, s.most_q = _cu(ql), max(ql)
    sees = _trees(len(ql), s.most_q, gen)
    if op == "compact":
        # a path of the tree, as a verification keeps it
        n = torch.tensor(_accepted_lens(case), device=DEV)
        a = torch.rand((len(ql), s.most_q), generator=gen, device=DEV)
        a = a.masked_fill(torch.arange(s.most_q, device=DEV) >= torch.tensor(ql, device=DEV)[:, None], 2.0)
        keep = a.argsort(1)[:, : max(1, int(n.max()))]
        live = torch.arange(keep.shape[1], device=DEV) < n[:, None]
        keep = keep.masked_fill(~live, 1 << 20).sort(1).values
        s.accepted = torch.where(live, keep, -1).to(torch.int32).contiguous()
        s.num_accepted = n.to(torch.int32)
        return s
    s.scale, s.most_ctx = 1 / math.sqrt(d), max(cl)
    s.q = torch.randn((sum(ql), case["nq"], d), generator=gen, device=DEV, dtype=torch.bfloat16) * 2
    words = -(-s.most_q // 32)
    bits = torch.zeros((len(ql), s.most_q, words * 32), dtype=torch.int64, device=DEV)
    bits[:, :, : s.most_q] = sees
    packed = (bits.view(len(ql), s.most_q, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
    live = torch.arange(s.most_q, device=DEV) < torch.tensor(ql, device=DEV)[:, None]
    s.mask = packed[live].contiguous()
    s.out = torch.empty_like(s.q)
    if own:
        from paged_kv_cache_482_b200 import pagedkv as K

        n = K.plan_tree(len(ql), case["nq"], case["nkv"], d, bs, s.most_q, s.most_ctx,
                        cache_dtype=K.cache_dtype(s.k_cache, s.k_scale))["workspace_bytes"]
        s.workspace = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    return s


def run(state):
    return {"norm_rope": _norm_rope, "tree": _tree, "compact": _compact, "load": _load}[state.op](state)


def _pool_outputs(s):
    """The pools (E4M3 codes as the values they stand for) and, with a scale per token, the scales."""
    if s.k_scale is not None and s.k_scale.dim() == 3:
        return [s.k_cache, s.v_cache, s.k_scale, s.v_scale]
    return [s.k_cache, s.v_cache]


def _bytes(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def _norm_rope(s):
    if own:
        from paged_kv_cache_482_b200 import pagedkv as K

        K.store_kvcache_norm_rope(s.k, s.v, s.k_cache, s.v_cache, s.slots, s.positions, s.cos_sin, s.k_weight, EPS,
                                  q=s.q, q_weight=s.q_weight, q_out=s.q_out, style=s.style, k_scale=s.k_scale,
                                  v_scale=s.v_scale, dev_err=s.dev_err)
        return [s.q_out] + _pool_outputs(s)
    half = s.q.shape[2] // 2
    cs = s.cos_sin[s.positions.long()][:, None, :]
    cos, sin = cs[..., :half], cs[..., half:]

    def rotated(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        if s.style == 0:
            a, b = x[..., :half], x[..., half:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)

    bs = s.k_cache.shape[2]
    live = s.slots >= 0
    slot = s.slots[live].long()
    blk, off = slot // bs, slot % bs
    for x, pool, scale in ((rotated(s.k, s.k_weight), s.k_cache, s.k_scale), (s.v.float(), s.v_cache, s.v_scale)):
        x = x[live]
        if scale is None:
            pool[blk, :, off] = x.to(torch.bfloat16)
            continue
        if scale.dim() == 3:
            by = x.abs().amax(-1) / 448
            scale[blk, :, off] = by
        else:
            by = scale.expand(x.shape[:2])
        _bytes(pool)[blk, :, off] = (x / by[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return [rotated(s.q, s.q_weight).to(torch.bfloat16)] + _pool_outputs(s)


def _rows(s, pool, scale, blk, off):
    """Cached rows [..., nkv, d] in 32 bits."""
    x = _bytes(pool)[blk, :, off]
    x = x.view(torch.float8_e4m3fn).float() if pool.dtype == torch.float8_e4m3fn else x.float()
    if scale is not None:
        x = x * (scale[blk, :, off] if scale.dim() == 3 else scale)[..., None]
    return x


def _tree(s):
    if own:
        from paged_kv_cache_482_b200 import pagedkv as K

        return K.paged_attention_tree(s.q, s.k_cache, s.v_cache, s.tables, s.cu, s.ctx, s.mask, s.scale, s.most_q,
                                      out=s.out, k_scale=s.k_scale, v_scale=s.v_scale, max_context_len=s.most_ctx,
                                      workspace=s.workspace, dev_err=s.dev_err)
    n, nq, d = s.q.shape
    nkv, bs, seqs, width = s.k_cache.shape[1], s.k_cache.shape[2], s.tables.shape[0], s.most_q
    t = torch.arange(s.most_ctx, device=DEV)
    blk = s.tables[:, t // bs].clamp(min=0).long()
    off = (t % bs).expand(seqs, -1)
    k = _rows(s, s.k_cache, s.k_scale, blk, off).permute(0, 2, 3, 1)  # [seqs, nkv, d, tokens]
    v = _rows(s, s.v_cache, s.v_scale, blk, off).permute(0, 2, 1, 3)
    cu, ctx = s.cu.long(), s.ctx.long()
    row = torch.arange(n, device=DEV)
    seq = torch.bucketize(row, cu[1:], right=True)
    loc = row - cu[seq]
    q = torch.zeros((seqs, width, nq, d), device=DEV)
    q[seq, loc] = s.q.float()
    q = q.view(seqs, width, nkv, nq // nkv, d).permute(0, 2, 3, 1, 4).reshape(seqs, nkv, -1, d)
    sees = torch.zeros((seqs, width, s.mask.shape[1] * 32), dtype=torch.bool, device=DEV)
    sees[seq, loc] = ((s.mask[..., None] >> torch.arange(32, device=DEV)) & 1).bool().flatten(1)
    drafts = cu[1:] - cu[:-1]
    u = t - (ctx - drafts)[:, None]  # [seqs, tokens]: the draft that sits there
    seen = sees.gather(2, u.clamp(0, sees.shape[2] - 1)[:, None, :].expand(-1, width, -1))
    seen = ((u < 0)[:, None] | (seen & (u < drafts[:, None])[:, None]))[:, None, None]
    x = (q @ k).mul_(s.scale).view(seqs, nkv, nq // nkv, width, -1)
    x.masked_fill_(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(seqs, nkv, -1, x.shape[-1]) @ v).view(seqs, nkv, nq // nkv, width, d)
    o = o / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, width, nq, d)[seq, loc].to(torch.bfloat16)


def _compact(s):
    if own:
        from paged_kv_cache_482_b200 import pagedkv as K

        K.compact_kvcache(s.k_cache, s.v_cache, s.tables, s.cu, s.ctx, s.accepted, s.num_accepted,
                          k_scale=s.k_scale, v_scale=s.v_scale, dev_err=s.dev_err)
        return _pool_outputs(s)
    bs = s.k_cache.shape[2]
    j = torch.arange(s.accepted.shape[1], device=DEV).expand_as(s.accepted)
    live = j < s.num_accepted[:, None]
    base = (s.ctx - (s.cu[1:] - s.cu[:-1])).long()[:, None]
    seq = torch.arange(s.tables.shape[0], device=DEV)[:, None].expand_as(s.accepted)[live]
    source, target = (base + s.accepted)[live], (base + j)[live]
    a, b = s.tables[seq, source // bs].long(), s.tables[seq, target // bs].long()
    pools = [_bytes(s.k_cache), _bytes(s.v_cache)] + (_pool_outputs(s)[2:])
    for pool in pools:
        pool[b, :, target % bs] = pool[a, :, source % bs]
    return _pool_outputs(s)


def _load(s):
    if own:
        from paged_kv_cache_482_b200 import pagedkv as K

        return list(K.load_kvcache(s.k_cache, s.v_cache, s.tables, s.cu, k_out=s.k_out, v_out=s.v_out,
                                   k_scale=s.k_scale, v_scale=s.v_scale, dev_err=s.dev_err))
    bs = s.k_cache.shape[2]
    row = torch.arange(s.k_out.shape[0], device=DEV)
    seq = torch.bucketize(row, s.cu[1:].long(), right=True)
    t = row - s.cu.long()[seq]
    blk = s.tables[seq, t // bs].long()
    return [_rows(s, p, c, blk, t % bs).to(torch.bfloat16) for p, c in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale))]


# ------------------------------------------------------------------ in 64 bits


def _values(pool, scale, block, offset):
    """Cached rows of one block-and-offset list, [tokens, nkv, d], in 64 bits."""
    if scale is None:
        return pool[block, :, offset].double()
    x = pool.view(torch.uint8)[block, :, offset].view(torch.float8_e4m3fn).double()
    by = scale.double()[block, :, offset] if scale.dim() == 3 else scale.double()[None, :]
    return x * by.unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    d, bs = case["d"], case["bs"]
    if case["op"] == "norm_rope":
        theta = s.cos_sin.double()[s.positions.long()]
        turn = torch.complex(theta[:, : d // 2], theta[:, d // 2:]).unsqueeze(1)

        def norm_turned(x, w):
            x = x.double()
            x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            pair = x.unflatten(-1, (2, d // 2)).transpose(-1, -2) if case["style"] == 0 else x.unflatten(-1, (d // 2, 2))
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            return (y.transpose(-1, -2) if case["style"] == 0 else y).flatten(-2)

        keep = torch.nonzero(s.slots >= 0).flatten()
        to = s.slots.long()[keep]
        pools, scales = [], []
        for x, pool, scale in ((norm_turned(s.k, s.k_weight), s.k_cache, s.k_scale), (s.v.double(), s.v_cache, s.v_scale)):
            rows, p = x[keep], pool.double()
            if scale is not None:
                by = rows.abs().amax(-1) / 448 if scale.dim() == 3 else scale.double().repeat(len(keep), 1)
                rows = (rows / by.unsqueeze(-1)).clamp(-448, 448)
                if scale.dim() == 3:
                    c = scale.double()
                    c[to // bs, :, to % bs] = by
                    scales.append(c)
            p[to // bs, :, to % bs] = rows
            pools.append(p)
        return [norm_turned(s.q, s.q_weight)] + pools + scales
    ql, cl = _lens(case)
    if case["op"] == "tree":
        outs, words = [], s.mask.cpu().long() & 0xFFFFFFFF
        group, row = case["nq"] // case["nkv"], 0
        for i, (c, n) in enumerate(zip(ql, cl)):
            at = torch.arange(n, device=DEV)
            block, offset = s.tables[i].long()[at // bs], at % bs
            kk, vv = (_values(p, f, block, offset) for p, f in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)))
            w = words[row:row + c]
            tree = torch.stack([(w[:, u // 32] >> (u % 32)) & 1 for u in range(c)], 1).bool().to(DEV)
            allowed = torch.cat([torch.ones((c, n - c), dtype=torch.bool, device=DEV), tree], 1)
            qq = s.q[row:row + c].double()
            heads = []
            for h in range(case["nq"]):
                z = qq[:, h] @ kk[:, h // group].T / math.sqrt(d)
                z = z.masked_fill(~allowed, -math.inf)
                heads.append(torch.softmax(z, -1) @ vv[:, h // group])
            outs.append(torch.stack(heads, 1))
            row += c
        return torch.cat(outs)
    if case["op"] == "compact":
        answer = [p.double() for p in _pool_outputs(s)]
        before = [p.clone() for p in answer]
        tables, accepted = s.tables.cpu(), s.accepted.cpu()
        for i, n in enumerate(_accepted_lens(case)):
            start = cl[i] - ql[i]
            for j in range(n):
                a, b = start + int(accepted[i, j]), start + j
                for x, y in zip(before, answer):
                    y[int(tables[i, b // bs]), :, b % bs] = x[int(tables[i, a // bs]), :, a % bs]
        return answer
    at = [torch.arange(n, device=DEV) for n in cl]
    block = torch.cat([s.tables[i].long()[a // bs] for i, a in enumerate(at)])
    offset = torch.cat([a % bs for a in at])
    return [_values(p, f, block, offset) for p, f in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale))]
