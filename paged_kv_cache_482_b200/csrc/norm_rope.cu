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
// Bandwidth bounds it (4 bytes of q per element, 2 of k and v and what the cache
// holds), if the table's row, twice the size of a q row, is not read again for
// every head. So a warp takes a token: its lanes hold the token's cosines and
// sines and the weight in registers, and walk the token's heads, 32 / L at a
// time (a row of head_dim elements is L = head_dim / 16 lanes of 8 pairs, which
// add up its sum of squares with shuffles), kBatch steps' loads in flight.
// Few tokens are spread over more warps, each with a part of the heads.
//
// Measured (B200): 8192 tokens, 32 query and 8 KV heads of 128, bf16: 43.1 us, 4.8
// TB/s (a group of lanes per row, which reads the table for every head: 53 us);
// into E4M3 with a scale per head 51.4 us; 2777 tokens, 16 and 8 heads, per-token E4M3:
// 15.9 us; one token: 2.8 us.
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

// E4M3 of x / scale, as with one IEEE division each, round to nearest even,
// saturating. The quotient is formed with one reciprocal: y = x * (1 / scale) is
// within 3 units of its last place of the division's result, so both round to
// the same code unless a point between two codes is that near. Those points, and
// the codes, have 19 zeros at the end of their binary32 significand: where y's
// last 19 bits are within 3 of zero the divisions are done (not below 2^-11 or
// above 440, where both round to 0 or 448).
__device__ __forceinline__ uint2 quantise8f(const float (&x)[8], float scale) {
    const bool plain = scale > 1e-36f && scale < 1e36f;  // the reciprocal is a normal number
    const float r = plain ? __frcp_rn(scale) : 0.0f;
    float y[8];
    bool near = !plain;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = x[j] * r;
        near |= ((__float_as_uint(y[j]) + 3u) & 0x7FFFFu) <= 6u && fabsf(y[j]) > 4e-4f && fabsf(y[j]) < 440.0f;
    }
    if (near) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(x[j], scale);
    }
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        out[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j], y[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
}

constexpr int kThreads = 128;
constexpr int kBatch = 2;
// Resident blocks per SM (102 registers a thread): with 4 and 6, 8192 tokens took
// 47.5 and 48.1 us instead of 43.1, 2777 into an E4M3 cache 18.3 and 22.5 instead of 16.
constexpr int kMinBlocks = 5;

// 16 bytes that the call does not read again. Not a read-only load: q_out may be q,
// whose elements the thread that loaded them writes back.
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Sum or maximum over the L adjacent lanes of a row (every lane of the warp calls).
__device__ __forceinline__ float row_sum(float x, int L) {
    for (int o = L >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float row_max(float x, int L) {
    for (int o = L >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// 8 pairs of a row: x (first elements) and y (second ones) normed and rotated.
template <int STYLE>
__device__ __forceinline__ void norm_rotate(uint4 a, uint4 b, const uint4 &wa, const uint4 &wb, const float (&cs)[8],
                                            const float (&sn)[8], int L, float inv_d, float eps, float (&x)[8],
                                            float (&y)[8]) {
    if constexpr (STYLE == 1) {
        uint4 t0, t1;
        deinterleave(a, b, t0, t1);
        a = t0;
        b = t1;
    }
    unpack8(a, x);
    unpack8(b, y);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
    const float inv = rsqrtf(fmaf(row_sum(ss, L), inv_d, eps));
    float u[8], v[8];
    unpack8(wa, u);
    unpack8(wb, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float na = x[j] * inv * u[j], nb = y[j] * inv * v[j];
        x[j] = fmaf(-nb, sn[j], na * cs[j]);
        y[j] = fmaf(na, sn[j], nb * cs[j]);
    }
}

// The two 16-byte chunks of a bf16 row.
template <int STYLE>
__device__ __forceinline__ void pack_row(const float (&x)[8], const float (&y)[8], uint4 &a, uint4 &b) {
    a = pack8(x);
    b = pack8(y);
    if constexpr (STYLE == 1) {
        uint4 t0, t1;
        interleave(a, b, t0, t1);
        a = t0;
        b = t1;
    }
}

// MODE 0: bf16 cache; 1: E4M3, a scale per KV head; 2: E4M3, a scale per row.
// A token's rows are `steps` steps of 32 / L rows: the q heads', the k heads',
// the v heads'. A warp takes up to `part` of them at a time; the loads of the
// next kBatch steps are issued before the current ones are worked on, and the
// first ones before the token's position and slot are known.
template <int MODE, int STYLE>
__global__ void __launch_bounds__(kThreads, kMinBlocks) store_norm_rope_kernel(NormRopeArgs p, int log2_l, int part,
                                                                               int parts) {
    const int L = 1 << log2_l, lane = threadIdx.x & 31;
    const int c = lane & (L - 1), sub = lane >> log2_l, rows = 32 >> log2_l;
    const int q_steps = (p.num_q_heads + rows - 1) / rows, kv_steps = (p.num_kv_heads + rows - 1) / rows;
    const int k_end = q_steps + kv_steps, steps = k_end + kv_steps;
    // element offsets of the two halves this lane handles, in a row
    const int ea = 8 * (STYLE == 1 ? 2 * c : c), eb = 8 * (STYLE == 1 ? 2 * c + 1 : c + L);
    const float inv_d = 1.0f / (float)p.head_dim;  // exact: a power of two
    auto load_weight = [&](const __nv_bfloat16 *w, uint4 &wa, uint4 &wb) {
        wa = __ldg(reinterpret_cast<const uint4 *>(w + ea));
        wb = __ldg(reinterpret_cast<const uint4 *>(w + eb));
        if constexpr (STYLE == 1) {
            uint4 t0, t1;
            deinterleave(wa, wb, t0, t1);
            wa = t0;
            wb = t1;
        }
    };
    const long long units = (long long)p.num_tokens * parts;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const long long token = u / parts;
        const int s0 = (int)(u % parts) * part, s1 = min(s0 + part, steps);
        const int m = __ldg(p.positions + token);
        const long long slot = __ldg(p.slots + token);
        const __nv_bfloat16 *qt = p.q + token * p.q_stride, *kt = p.k + token * p.k_stride, *vt = p.v + token * p.v_stride;
        uint4 na[kBatch], nb[kBatch];  // the next steps' chunks
        auto load = [&](int s) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int si = s + i;
                const int head = (si < q_steps ? si : si < k_end ? si - q_steps : si - k_end) * rows + sub;
                const __nv_bfloat16 *src = (si < q_steps ? qt : si < k_end ? kt : vt) + (long long)head * p.head_dim;
                na[i] = nb[i] = make_uint4(0, 0, 0, 0);
                if (si < s1 && head < (si < q_steps ? p.num_q_heads : p.num_kv_heads)) {
                    na[i] = load_row(src + ea);
                    nb[i] = load_row(src + eb);
                }
            }
        };
        load(s0);
        if (m < 0 || m >= p.max_position) {  // the same for the whole warp
            if (lane == 0 && s0 == 0) set_error(p.dev_err, PKV_DEVERR_BOUNDS);
            continue;
        }
        int last = s1;  // steps to be done
        if (slot < 0 || slot >= p.pool_slots) {
            last = min(s1, q_steps);
            if (slot >= 0 && s1 > q_steps && lane == 0) set_error(p.dev_err, PKV_DEVERR_BOUNDS);
        }
        const long long blk = slot / p.block_size, off = slot - blk * p.block_size;
        float cs[8], sn[8];
        const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (long long)m * p.head_dim + 8 * c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 x = __ldg(row + h), y = __ldg(row + p.head_dim / 8 + h);
            cs[4 * h] = x.x;
            cs[4 * h + 1] = x.y;
            cs[4 * h + 2] = x.z;
            cs[4 * h + 3] = x.w;
            sn[4 * h] = y.x;
            sn[4 * h + 1] = y.y;
            sn[4 * h + 2] = y.z;
            sn[4 * h + 3] = y.w;
        }
        uint4 wa, wb;  // the q weight, then the k weight
        load_weight(s0 < q_steps ? p.q_weight : p.k_weight, wa, wb);
        for (int s = s0; s < last; s += kBatch) {
            uint4 a[kBatch], b[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                a[i] = na[i];
                b[i] = nb[i];
            }
            if (s + kBatch < last) load(s + kBatch);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int si = s + i;  // the same in every lane, so is the kind of row
                if (si >= last) break;
                if (si == q_steps && si > s0) load_weight(p.k_weight, wa, wb);
                float x[8], y[8];
                if (si < q_steps) {
                    const int head = si * rows + sub;
                    norm_rotate<STYLE>(a[i], b[i], wa, wb, cs, sn, L, inv_d, p.eps, x, y);
                    if (head < p.num_q_heads) {
                        uint4 oa, ob;
                        pack_row<STYLE>(x, y, oa, ob);
                        __nv_bfloat16 *dst = p.q_out + token * p.q_out_stride + (long long)head * p.head_dim;
                        *reinterpret_cast<uint4 *>(dst + ea) = oa;
                        *reinterpret_cast<uint4 *>(dst + eb) = ob;
                    }
                    continue;
                }
                const bool is_k = si < k_end;
                const int head = (si - (is_k ? q_steps : k_end)) * rows + sub;
                const bool live = head < p.num_kv_heads;
                const long long prow = (blk * p.num_kv_heads + (live ? head : 0)) * p.block_size + off;  // pool row
                uint4 oa = a[i], ob = b[i];
                if (is_k) norm_rotate<STYLE>(a[i], b[i], wa, wb, cs, sn, L, inv_d, p.eps, x, y);
                if constexpr (MODE == 0) {
                    if (is_k) pack_row<STYLE>(x, y, oa, ob);
                    if (live) {
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_k ? p.k_cache : p.v_cache) + prow * p.head_dim;
                        *reinterpret_cast<uint4 *>(dst + ea) = oa;
                        *reinterpret_cast<uint4 *>(dst + eb) = ob;
                    }
                } else {
                    if (!is_k) {
                        unpack8(oa, x);
                        unpack8(ob, y);
                    }
                    float *scales = is_k ? p.k_scale : p.v_scale;
                    float scale;
                    if constexpr (MODE == 2) {
                        float top = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(fabsf(x[j]), fabsf(y[j])));
                        scale = token_scale(row_max(top, L));
                        if (live && c == 0) scales[prow] = scale;
                    } else {
                        scale = __ldg(scales + (live ? head : 0));
                    }
                    uint2 ca = quantise8f(x, scale), cb = quantise8f(y, scale);
                    if (STYLE == 1 && is_k) {  // the codes back to interleaved order
                        const uint2 t0 = ca, t1 = cb;
                        ca = make_uint2(__byte_perm(t0.x, t1.x, 0x5140), __byte_perm(t0.x, t1.x, 0x7362));
                        cb = make_uint2(__byte_perm(t0.y, t1.y, 0x5140), __byte_perm(t0.y, t1.y, 0x7362));
                    }
                    if (live) {
                        uint8_t *dst = static_cast<uint8_t *>(is_k ? p.k_cache : p.v_cache) + prow * p.head_dim;
                        *reinterpret_cast<uint2 *>(dst + ea) = ca;
                        *reinterpret_cast<uint2 *>(dst + eb) = cb;
                    }
                }
            }
        }
    }
}

template <int MODE, int STYLE>
cudaError_t launch_style(const NormRopeArgs &p, int num_sms, cudaStream_t stream) {
    auto kern = store_norm_rope_kernel<MODE, STYLE>;
    int log2_l = 0;
    while ((16 << log2_l) < p.head_dim) ++log2_l;
    const int rows = 32 >> log2_l;
    const int steps = (p.num_q_heads + rows - 1) / rows + 2 * ((p.num_kv_heads + rows - 1) / rows);
    // a token is divided among warps while that leaves resident ones without work
    // (one token, 32 query and 8 KV heads: 2.9 us, undivided 6.8)
    const long long resident = (long long)num_sms * kMinBlocks * (kThreads / 32);
    long long part = ((long long)p.num_tokens * steps + resident - 1) / resident;
    if (part > steps) part = steps;
    const int parts = (int)((steps + part - 1) / part);
    const long long units = (long long)p.num_tokens * parts;
    long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > (long long)num_sms * kMinBlocks) blocks = (long long)num_sms * kMinBlocks;
    kern<<<(unsigned)blocks, kThreads, 0, stream>>>(p, log2_l, (int)part, parts);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_store_norm_rope(const NormRopeArgs &a, int style, int mode, int num_sms, cudaStream_t stream) {
    if (mode == 2) return style == 1 ? launch_style<2, 1>(a, num_sms, stream) : launch_style<2, 0>(a, num_sms, stream);
    if (mode == 1) return style == 1 ? launch_style<1, 1>(a, num_sms, stream) : launch_style<1, 0>(a, num_sms, stream);
    return style == 1 ? launch_style<0, 1>(a, num_sms, stream) : launch_style<0, 0>(a, num_sms, stream);
}

}  // namespace pkv
