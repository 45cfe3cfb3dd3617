// norm_rope.cu -- RMSNorm of every query and key head, the rotary position
// embedding and the store of the step's K/V rows, in one pass (sm_100a).
//
// For a row x of head_dim elements (a query or key head of one token at
// position m) with its weight w, all in binary32:
//   n_i = x_i / sqrt(mean(x^2) + eps) * w_i
//   x'_i = n_i cos(m, p) - n_j sin(m, p),  x'_j = n_j cos(m, p) + n_i sin(m, p)
// for the pairs p = (i, j) of store_kvcache_rope (the rotation of the RoFormer
// paper, Su et al. 2021), with cos and sin from the caller's table. The result
// is rounded once: to bf16 for q_out and a bf16 cache, to E4M3 for an E4M3
// cache (no bf16 in between, unlike store_kvcache_rope, whose rotated k is a
// bf16 tensor of the caller's: here the normed k exists only in registers, and
// a second rounding would only lose bits). v is stored as store_kvcache does.
//
// q, k and v are read where the projection left them: a token's heads are
// contiguous, tokens lie a caller-given stride apart (for instance one row of
// the fused QKV projection).
//
// One thread handles 8 pairs of one (token, row); a row takes head_dim / 16
// adjacent lanes, which add up the row's sum of squares with shuffles.
#include "pkv_common.cuh"
#include "pkv_launch.h"
#include "store_common.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16lo(w[j]);
        f[2 * j + 1] = bf16hi(w[j]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// E4M3 of x / scale (one IEEE division each, round to nearest even, saturating).
__device__ __forceinline__ uint2 quantise8f(const float (&x)[8], float scale) {
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = __nv_cvt_float_to_fp8(__fdiv_rn(x[j], scale), __NV_SATFINITE, __NV_E4M3);
        out[j >> 2] |= c << ((j & 3) * 8);
    }
    return make_uint2(out[0], out[1]);
}

// MODE 0: bf16 cache; 1: E4M3, a scale per KV head; 2: E4M3, a scale per row.
template <int MODE, int STYLE>
__global__ void __launch_bounds__(256) store_norm_rope_kernel(NormRopeArgs p) {
    const int L = p.head_dim / 16;  // lanes per row
    const int rows = p.num_q_heads + p.num_kv_heads;
    const long long units = (long long)p.num_tokens * rows * L;
    const long long stride = (long long)gridDim.x * blockDim.x;
    for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < units; u += stride) {
        const int c = (int)(u % L);
        const long long rowi = u / L;
        const int r = (int)(rowi % rows);
        const long long token = rowi / rows;
        // 16-byte chunks of the two halves this lane handles
        const int ca = STYLE == 1 ? 2 * c : c;
        const int cb = STYLE == 1 ? 2 * c + 1 : c + L;
        const bool is_q = r < p.num_q_heads;
        const int head = is_q ? r : r - p.num_q_heads;
        const int m = __ldg(p.positions + token);
        if (m < 0 || m >= p.max_position) {
            if (c == 0 && r == 0) set_error(p.dev_err, PKV_DEVERR_BOUNDS);
            continue;
        }
        long long slot = 0;
        if (!is_q) {
            slot = __ldg(p.slots + token);
            if (slot < 0) continue;
            if (slot >= p.pool_slots) {
                set_error(p.dev_err, PKV_DEVERR_BOUNDS);
                continue;
            }
        }
        const __nv_bfloat16 *src = is_q ? p.q + token * p.q_stride : p.k + token * p.k_stride;
        const uint4 *x = reinterpret_cast<const uint4 *>(src + (long long)head * p.head_dim);
        uint4 a = x[ca], b = x[cb];
        const uint4 *w = reinterpret_cast<const uint4 *>(is_q ? p.q_weight : p.k_weight);
        uint4 wa = __ldg(w + ca), wb = __ldg(w + cb);
        if constexpr (STYLE == 1) {
            uint4 t0, t1;
            deinterleave(a, b, t0, t1);
            a = t0;
            b = t1;
            deinterleave(wa, wb, t0, t1);
            wa = t0;
            wb = t1;
        }
        float xa[8], xb[8], va[8], vb[8];
        unpack8(a, xa);
        unpack8(b, xb);
        unpack8(wa, va);
        unpack8(wb, vb);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], ss));
        const int lane = threadIdx.x & 31;
        const unsigned group = (L == 32 ? 0xffffffffu : ((1u << L) - 1u)) << (lane & ~(L - 1));
        for (int o = L >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o, L);
        const float inv = rsqrtf(ss / (float)p.head_dim + p.eps);
        const float *cs = p.cos_sin + (long long)m * p.head_dim + 8 * c;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float cc = __ldg(cs + j), sn = __ldg(cs + p.head_dim / 2 + j);
            const float na = xa[j] * inv * va[j], nb = xb[j] * inv * vb[j];
            xa[j] = fmaf(-nb, sn, na * cc);
            xb[j] = fmaf(na, sn, nb * cc);
        }
        if (is_q || MODE == 0) {
            uint4 oa = pack8(xa), ob = pack8(xb);
            if constexpr (STYLE == 1) {
                uint4 t0, t1;
                interleave(oa, ob, t0, t1);
                oa = t0;
                ob = t1;
            }
            if (is_q) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + token * p.q_out_stride + (long long)head * p.head_dim);
                dst[ca] = oa;
                dst[cb] = ob;
                continue;
            }
            a = oa;
            b = ob;
        }
        const uint4 *vsrc = reinterpret_cast<const uint4 *>(p.v + token * p.v_stride + (long long)head * p.head_dim);
        const uint4 v0 = vsrc[ca], v1 = vsrc[cb];
        const long long blk = slot / p.block_size;
        const long long off = slot - blk * p.block_size;
        const long long row = (blk * p.num_kv_heads + head) * p.block_size + off;  // pool row
        const long long ea = row * p.head_dim + ca * 8LL, eb = row * p.head_dim + cb * 8LL;
        if constexpr (MODE == 0) {
            __nv_bfloat16 *kc = static_cast<__nv_bfloat16 *>(p.k_cache), *vc = static_cast<__nv_bfloat16 *>(p.v_cache);
            *reinterpret_cast<uint4 *>(kc + ea) = a;
            *reinterpret_cast<uint4 *>(kc + eb) = b;
            *reinterpret_cast<uint4 *>(vc + ea) = v0;
            *reinterpret_cast<uint4 *>(vc + eb) = v1;
        } else {
            float ks, vs;
            if constexpr (MODE == 2) {
                float km = 0.f, vm = fmaxf(amax8(v0), amax8(v1));
#pragma unroll
                for (int j = 0; j < 8; ++j) km = fmaxf(km, fmaxf(fabsf(xa[j]), fabsf(xb[j])));
                for (int o = L >> 1; o > 0; o >>= 1) {
                    km = fmaxf(km, __shfl_xor_sync(group, km, o, L));
                    vm = fmaxf(vm, __shfl_xor_sync(group, vm, o, L));
                }
                ks = token_scale(km);
                vs = token_scale(vm);
                if (c == 0) {
                    p.k_scale[row] = ks;
                    p.v_scale[row] = vs;
                }
            } else {
                ks = __ldg(p.k_scale + head);
                vs = __ldg(p.v_scale + head);
            }
            uint2 qa = quantise8f(xa, ks), qb = quantise8f(xb, ks);
            if constexpr (STYLE == 1) {  // the codes back to interleaved order
                const uint2 t0 = qa, t1 = qb;
                qa = make_uint2(__byte_perm(t0.x, t1.x, 0x5140), __byte_perm(t0.x, t1.x, 0x7362));
                qb = make_uint2(__byte_perm(t0.y, t1.y, 0x5140), __byte_perm(t0.y, t1.y, 0x7362));
            }
            uint8_t *kc = static_cast<uint8_t *>(p.k_cache), *vc = static_cast<uint8_t *>(p.v_cache);
            *reinterpret_cast<uint2 *>(kc + ea) = qa;
            *reinterpret_cast<uint2 *>(kc + eb) = qb;
            *reinterpret_cast<uint2 *>(vc + ea) = quantise8(v0, vs);
            *reinterpret_cast<uint2 *>(vc + eb) = quantise8(v1, vs);
        }
    }
}

template <int MODE>
void launch_mode(const NormRopeArgs &p, int style, unsigned blocks, cudaStream_t stream) {
    if (style == 1)
        store_norm_rope_kernel<MODE, 1><<<blocks, 256, 0, stream>>>(p);
    else
        store_norm_rope_kernel<MODE, 0><<<blocks, 256, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_store_norm_rope(const NormRopeArgs &a, int style, int mode, int num_sms, cudaStream_t stream) {
    const long long units = (long long)a.num_tokens * (a.num_q_heads + a.num_kv_heads) * (a.head_dim / 16);
    long long blocks = (units + 255) / 256;
    const long long cap = (long long)num_sms * 16;
    if (blocks > cap) blocks = cap;
    if (blocks < 1) blocks = 1;
    if (mode == 2)
        launch_mode<2>(a, style, (unsigned)blocks, stream);
    else if (mode == 1)
        launch_mode<1>(a, style, (unsigned)blocks, stream);
    else
        launch_mode<0>(a, style, (unsigned)blocks, stream);
    return cudaGetLastError();
}

}  // namespace pkv
