// tree.cu -- attention of a tree of drafted tokens over the paged cache (sm_100a).
//
// Sequence s brings c = cu_q_lens[s + 1] - cu_q_lens[s] drafted tokens whose
// K/V are already the last c of its context_lens[s] cached positions. With
// base = context - c, draft j attends to the positions t < base and to the
// drafts u with bit u of its mask set:
//   out[j][h] = sum_t softmax_t(scale * q[j][h] . K_t) V_t
// over those t; a row that sees nothing is zeros.
//
// One warp per (draft, query head), the row's d elements spread over the
// lanes, one pass over the visible tokens with the running maximum and sum.
#include "pkv_common.cuh"
#include "pkv_launch.h"

namespace pkv {

namespace {

template <int D, int MODE>
__global__ void __launch_bounds__(128) tree_simple_kernel(TreeArgs a, int rows_per_seq) {
    constexpr int E = D / 32;  // elements per lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks_per_seq = (rows_per_seq + 3) / 4;
    const int s = blockIdx.x / blocks_per_seq;
    const int item = (blockIdx.x % blocks_per_seq) * 4 + warp;  // draft * num_q_heads + head
    const int nq = a.num_q_heads;
    const int j = item / nq, h = item % nq;
    const int q0 = a.cu_q_lens[s], q1 = a.cu_q_lens[s + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.total_q) {
        if (threadIdx.x == 0) set_error(a.dev_err, PKV_DEVERR_BOUNDS);
        return;
    }
    const int c = q1 - q0;
    if (item >= rows_per_seq || j >= c) return;
    const int ctx = a.context_lens[s];
    const int kh = h / (nq / a.num_kv_heads);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + ((long long)(q0 + j) * nq + h) * D + lane * E;
    const int32_t *table = a.block_tables + (long long)s * a.max_blocks_per_seq;
    bool bad = c > a.max_q_len || ctx < c || ctx > a.max_context_len;
    const int nblk = bad ? 0 : (ctx + a.block_size - 1) / a.block_size;
    for (int i = lane; i < nblk; i += 32) {
        const int b = table[i];
        bad |= b < 0 || b >= a.num_blocks;
    }
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float m = -INFINITY, l = 0.f;
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) set_error(a.dev_err, PKV_DEVERR_BOUNDS);
        for (long long r = j + a.max_q_len; r < c; r += a.max_q_len)  // a chunk longer than the grid expects
            for (int e = 0; e < E; ++e) out[(r - j) * nq * D + e] = __float2bfloat16_rn(0.f);
    } else {
        const int base = ctx - c;
        const uint32_t *mask = a.mask + (long long)(q0 + j) * a.mask_words;
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + ((long long)(q0 + j) * nq + h) * D + lane * E;
        float qv[E];
#pragma unroll
        for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(q[e]) * a.scale * 1.4426950408889634f;
        for (int t = 0; t < ctx; ++t) {
            if (t >= base) {
                const int u = t - base;
                if (!((mask[u >> 5] >> (u & 31)) & 1u)) continue;
            }
            const long long row = ((long long)table[t / a.block_size] * a.num_kv_heads + kh) * a.block_size +
                                  t % a.block_size;
            float kx[E], vx[E];
            if constexpr (MODE == 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    kx[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.k_cache)[row * D + lane * E + e]);
                    vx[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v_cache)[row * D + lane * E + e]);
                }
            } else {
                const float ks = a.k_scale[MODE == 2 ? row : kh], vs = a.v_scale[MODE == 2 ? row : kh];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 k2 = e4m3x2_to_float2(
                        *reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(a.k_cache) + row * D + lane * E + e));
                    const float2 v2 = e4m3x2_to_float2(
                        *reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(a.v_cache) + row * D + lane * E + e));
                    kx[e] = k2.x * ks;
                    kx[e + 1] = k2.y * ks;
                    vx[e] = v2.x * vs;
                    vx[e + 1] = v2.y * vs;
                }
            }
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(qv[e], kx[e], x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            const float mn = fmaxf(m, x);
            const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
            const float p = mn == -INFINITY ? 0.f : exp2f(x - mn);
            l = l * alpha + p;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(p, vx[e], acc[e] * alpha);
            m = mn;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = __float2bfloat16_rn(acc[e] * inv);
}

template <int D>
cudaError_t launch_simple(const TreeArgs &a, cudaStream_t stream) {
    const int rows = a.max_q_len * a.num_q_heads;
    const long long blocks = (long long)a.num_seqs * ((rows + 3) / 4);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (a.mode == 2)
        tree_simple_kernel<D, 2><<<(unsigned)blocks, 128, 0, stream>>>(a, rows);
    else if (a.mode == 1)
        tree_simple_kernel<D, 1><<<(unsigned)blocks, 128, 0, stream>>>(a, rows);
    else
        tree_simple_kernel<D, 0><<<(unsigned)blocks, 128, 0, stream>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeArgs &a, cudaStream_t stream) {
    return a.head_dim == 128 ? launch_simple<128>(a, stream) : launch_simple<64>(a, stream);
}

}  // namespace pkv
