"""Plain 64-bit forms of the speculative-step operators, on the CPU.

Written from the formulas with torch and python loops; the GPU tests hold the
kernels to them with tolerances that count roundings: a value rounded to
nearest is off by at most u times itself (u = finfo.eps / 2), so a sum of
products with several rounded factors is off by at most the sum of their u
times the sum of the magnitudes.
"""

from __future__ import annotations

import torch

U_BF16 = torch.finfo(torch.bfloat16).eps / 2
U_F16 = torch.finfo(torch.float16).eps / 2
U_F32 = torch.finfo(torch.float32).eps / 2
U_E4M3 = 2.0 ** -4
E4M3_STEP = 2.0 ** -9  # spacing of the subnormal codes


def e4m3_values(pool: torch.Tensor) -> torch.Tensor:
    return pool.cpu().view(torch.uint8).view(torch.float8_e4m3fn).double()


def cache_values(pool, scale=None) -> torch.Tensor:
    """The pool's values [blocks, heads, block_size, d] in 64 bits."""
    if pool.dtype == torch.bfloat16:
        return pool.cpu().double()
    x = e4m3_values(pool)
    s = scale.cpu().double()
    return x * (s[..., None] if s.dim() == 3 else s[None, :, None, None])


def tree_rows(values, table, n):
    """[n, heads, d]: the first n tokens of a block-table row."""
    bs = values.shape[2]
    t = torch.arange(n)
    return values[table.cpu().long()[t // bs], :, t % bs]


def sees(mask, c):
    """[rows, c] bool of int32 mask words."""
    m = mask.cpu().long() & 0xFFFFFFFF
    u = torch.arange(c)
    return ((m[:, u // 32] >> (u % 32)) & 1).bool()


def tree_attention(q, k_values, v_values, tables, cu, ctx, mask, scale):
    """(out, sum of weight * |v|) in 64 bits; rows of no sequence are NaN.
    Only the visible keys are touched, so what others hold cannot matter."""
    q = q.cpu().double()
    out = torch.full_like(q, float("nan"))
    mag = torch.zeros_like(q)
    cu, ctx = cu.tolist(), ctx.tolist()
    G = q.shape[1] // k_values.shape[1]
    for i, n in enumerate(ctx):
        a, b = cu[i], cu[i + 1]
        c = b - a
        K, V = tree_rows(k_values, tables[i], n), tree_rows(v_values, tables[i], n)
        vis = torch.cat([torch.ones(c, n - c, dtype=torch.bool), sees(mask[a:b], c)], 1)
        for r in range(c):
            keys = torch.nonzero(vis[r]).flatten()
            if len(keys) == 0:
                out[a + r] = 0
                continue
            kk, vv = K[keys].repeat_interleave(G, 1), V[keys].repeat_interleave(G, 1)
            s = torch.einsum("hd,thd->ht", q[a + r], kk) * scale
            p = torch.softmax(s, 1)
            out[a + r] = torch.einsum("ht,thd->hd", p, vv)
            mag[a + r] = torch.einsum("ht,thd->hd", p, vv.abs())
    return out, mag


def tree_tolerance(out, mag, fp8, token):
    """Elementwise bound of the kernel's distance from tree_attention.

    The weights are rounded once before P V (bf16; f16 for E4M3 with a scale
    per KV head), so the numerator is off by u_p of its magnitude, and the
    normaliser, were it to sum the rounded ones, by u_p of its own; per-token V
    may be rounded to bf16 when it is dequantised; the output is, too. The binary32 sums and
    the exponential add less than 2^-10 of the magnitude for the scores of
    these tests (below 2^6, with sums of at most 2^7 products).
    """
    u_p = U_F16 if fp8 and not token else U_BF16
    u_v = U_BF16 if token else 0.0
    return U_BF16 * out.abs() + (2 * u_p + u_v + 2.0 ** -10) * mag * (1 + U_BF16) + 1e-30


def norm_rope(x, weight, eps, positions, cos_sin, style):
    """(result, sum of the two products' magnitudes) in 64 bits, [N, heads, d]."""
    x = x.cpu().double()
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.cpu().double()
    d = x.shape[-1]
    cs = cos_sin.cpu().double()[positions.cpu().long().clamp(0, cos_sin.shape[0] - 1)][:, None]
    cos, sin = cs[..., : d // 2], cs[..., d // 2:]
    if style == 0:
        a, b = n[..., : d // 2], n[..., d // 2:]
        join = lambda u, v: torch.cat([u, v], -1)  # noqa: E731
    else:
        a, b = n[..., 0::2], n[..., 1::2]
        join = lambda u, v: torch.stack([u, v], -1).flatten(-2)  # noqa: E731
    return (join(a * cos - b * sin, b * cos + a * sin),
            join((a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()))
