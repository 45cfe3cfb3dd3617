// move_kvcache.cu -- cached rows moved or read back (sm_100a): the rows of
// accepted drafts closed up after a tree's verification (compact_kvcache), and
// a batch's rows read back as bf16 (load_kvcache).
#include "pkv_common.cuh"
#include "pkv_launch.h"
#include "tc_common.cuh"

namespace pkv {

namespace {

using tc::e4m3x8_scaled_bf16x8;

// ------------------------------------------------------------------ compact
//
// Sequence i keeps the drafts accepted[i][0] < accepted[i][1] < ...; draft
// accepted[i][j] moves to place j of the draft region (position base + j). No
// arithmetic: codes and scales move as they are.
//
// One block per (sequence, KV head). Places and drafts overlap (place j may be
// the source of an earlier place), so a pass reads its rows, waits for the
// block, and writes them. accepted[i][j] >= j because the list ascends, so a
// pass over places [a, b) writes only below b and every later pass reads only
// at or above b: passes need nothing more between them.
//
// Latency bounds it: the chain lengths -> list -> table -> row -> store. Measured
// (B200): one sequence of 8 drafts 2.7 us, 256 sequences of 33-64 drafts 7.2 us.
constexpr int kMoveThreads = 256;

// U: the copy unit (uint4, or uint2 where rows are not a multiple of 16 bytes).
template <typename U>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(CompactArgs p) {
    const int s = blockIdx.x / p.num_kv_heads;
    const int kh = blockIdx.x % p.num_kv_heads;
    const int tid = threadIdx.x;
    const int q0 = p.cu_q_lens[s], q1 = p.cu_q_lens[s + 1];
    const int ctx = p.context_lens[s], n = p.num_accepted[s];
    const long long c = (long long)q1 - q0;
    const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
    // a sequence with anything out of range is left as it is
    bool bad = q0 < 0 || c < 0 || ctx < c || ctx > cap || n < 0 || n > c || n > p.max_accepted;
    const int32_t *list = p.accepted + (long long)s * p.max_accepted;
    const int32_t *table = p.block_tables + (long long)s * p.max_blocks_per_seq;
    const int base = bad ? 0 : (int)(ctx - c);
    for (int j = tid; j < n && !bad; j += kMoveThreads) {
        const int a = list[j];
        if (a < 0 || a >= c || (j > 0 && list[j - 1] >= a)) {
            bad = true;
            break;
        }
        const int b0 = table[(base + a) / p.block_size], b1 = table[(base + j) / p.block_size];
        if (b0 < 0 || b0 >= p.num_blocks || b1 < 0 || b1 >= p.num_blocks) bad = true;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) set_error(p.dev_err, PKV_DEVERR_BOUNDS);
        return;
    }
    auto pool_row = [&](int t) {
        return ((long long)table[t / p.block_size] * p.num_kv_heads + kh) * p.block_size + t % p.block_size;
    };
    const int per_row = p.row_bytes / (int)sizeof(U);  // copy units of a K (or V) row
    const long long total = (long long)n * per_row * 2;
    for (long long i0 = 0; i0 < total; i0 += kMoveThreads) {
        // units in row order, so that a pass is a range of places
        const long long i = i0 + tid;
        const int j = (int)(i / (2 * per_row));
        const int u = (int)(i % (2 * per_row));
        const bool live = i < total && list[j] != j;
        U *pool = static_cast<U *>(u < per_row ? p.k_cache : p.v_cache);
        const int col = u < per_row ? u : u - per_row;
        U x;
        long long dst = 0;
        if (live) {
            x = pool[pool_row(base + list[j]) * per_row + col];
            dst = pool_row(base + j);
        }
        __syncthreads();
        if (live) pool[dst * per_row + col] = x;
    }
    if (p.k_scale) {
        for (int j0 = 0; j0 < n; j0 += kMoveThreads) {
            const int j = j0 + tid;
            const bool live = j < n && list[j] != j;
            float ks = 0.f, vs = 0.f;
            long long dst = 0;
            if (live) {
                const long long src = pool_row(base + list[j]);
                ks = p.k_scale[src];
                vs = p.v_scale[src];
                dst = pool_row(base + j);
            }
            __syncthreads();
            if (live) {
                p.k_scale[dst] = ks;
                p.v_scale[dst] = vs;
            }
        }
    }
}

// --------------------------------------------------------------------- load
//
// Output row cu_rows[i] + r is token starts[i] + r of sequence i: bf16 rows
// copied, E4M3 codes times their scale in binary32 and rounded to bf16.
// Bandwidth bounds it. A warp takes up to kLoadRows consecutive rows: its lanes find
// each row's sequence (by bisection over cu_rows) and pool block together, one
// row per lane, and then move the rows' 16-byte output chunks, kLoadBatch of a
// lane in flight.
// Measured (B200): 16 sequences of 2048-8192 E4M3 tokens in blocks of 16, 8 heads of
// 128: 88 us, 5.1 TB/s (a thread per chunk that finds its own sequence: 114 us), with a
// scale per token the same, bf16 103 us, 5.8 TB/s; 133 bf16 tokens: 3.9 us.
constexpr int kLoadThreads = 256;
constexpr int kLoadRows = 8;  // at most; fewer while that leaves SMs without warps
constexpr int kLoadBatch = 4;

// Output chunk of 8 elements from a pool row's chunk.
template <int MODE>
__device__ __forceinline__ uint4 load_chunk(const void *pool, long long at) {
    if constexpr (MODE == 0) return __ldg(static_cast<const uint4 *>(pool) + at);
    const uint2 w = __ldg(static_cast<const uint2 *>(pool) + at);
    return make_uint4(w.x, w.y, 0, 0);
}

template <int MODE>
__global__ void __launch_bounds__(kLoadThreads) load_kernel(LoadArgs p, int rows) {
    const int cpr = p.head_dim / 8, per_row = p.num_kv_heads * cpr;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0) {  // the bisection below trusts an ascending list
        for (int i = threadIdx.x; i < p.num_seqs; i += kLoadThreads)
            if (p.cu_rows[i] < 0 || p.cu_rows[i + 1] < p.cu_rows[i] || p.cu_rows[i + 1] > p.total_rows)
                set_error(p.dev_err, PKV_DEVERR_BOUNDS);
    }
    const long long tiles = ((long long)p.total_rows + rows - 1) / rows;
    const long long warps = (long long)gridDim.x * (kLoadThreads / 32);
    for (long long tile = (long long)blockIdx.x * (kLoadThreads / 32) + (threadIdx.x >> 5); tile < tiles; tile += warps) {
        const long long row0 = tile * rows;
        // lane r: row row0 + r; base: pool row of its KV head 0, -1: zeros, -2: no sequence's row
        long long base = -2;
        if (lane < rows && row0 + lane < p.total_rows) {
            const int row = (int)(row0 + lane);
            int lo = 0, hi = p.num_seqs;  // the last sequence that starts at or before the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (__ldg(p.cu_rows + mid) <= row) lo = mid;
                else hi = mid;
            }
            const int first = __ldg(p.cu_rows + lo);
            if (row >= first && row < __ldg(p.cu_rows + lo + 1)) {
                const long long t = (p.starts ? (long long)__ldg(p.starts + lo) : 0) + (row - first);
                int blk = -1;
                if (t >= 0 && t < (long long)p.max_blocks_per_seq * p.block_size)
                    blk = __ldg(p.block_tables + (long long)lo * p.max_blocks_per_seq + t / p.block_size);
                if (blk < 0 || blk >= p.num_blocks) {
                    set_error(p.dev_err, PKV_DEVERR_BOUNDS);
                    base = -1;
                } else {
                    base = (long long)blk * p.num_kv_heads * p.block_size + t % p.block_size;
                }
            }
        }
        const int units = rows * per_row;
        for (int i0 = 0; i0 < units; i0 += 32 * kLoadBatch) {
            uint4 k[kLoadBatch], v[kLoadBatch];
            float ks[kLoadBatch], vs[kLoadBatch];
            long long from[kLoadBatch];
#pragma unroll
            for (int j = 0; j < kLoadBatch; ++j) {
                const int i = i0 + 32 * j + lane;
                const int r = i / per_row, x = i - r * per_row;
                const int kh = x / cpr, c = x - kh * cpr;
                const long long b = __shfl_sync(0xffffffffu, base, r & 31);
                from[j] = i < units ? b : -2;
                k[j] = v[j] = make_uint4(0, 0, 0, 0);
                ks[j] = vs[j] = 0.0f;
                if (from[j] >= 0) {
                    const long long prow = b + (long long)kh * p.block_size;
                    k[j] = load_chunk<MODE>(p.k_cache, prow * cpr + c);
                    v[j] = load_chunk<MODE>(p.v_cache, prow * cpr + c);
                    if constexpr (MODE != 0) {
                        ks[j] = __ldg(p.k_scale + (MODE == 2 ? prow : kh));
                        vs[j] = __ldg(p.v_scale + (MODE == 2 ? prow : kh));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kLoadBatch; ++j) {
                if (from[j] == -2) continue;
                if constexpr (MODE != 0) {
                    k[j] = e4m3x8_scaled_bf16x8(make_uint2(k[j].x, k[j].y), ks[j]);
                    v[j] = e4m3x8_scaled_bf16x8(make_uint2(v[j].x, v[j].y), vs[j]);
                }
                const long long to = row0 * per_row + i0 + 32 * j + lane;
                __stcs(p.k_out + to, k[j]);  // not read again here
                __stcs(p.v_out + to, v[j]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream) {
    const long long blocks = (long long)a.num_seqs * a.num_kv_heads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (a.row_bytes % 16 == 0)
        compact_kernel<uint4><<<(unsigned)blocks, kMoveThreads, 0, stream>>>(a);
    else
        compact_kernel<uint2><<<(unsigned)blocks, kMoveThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_load(const LoadArgs &a, int mode, int num_sms, cudaStream_t stream) {
    // rows per warp: 8, and fewer while 32 warps per SM would not all have some (133
    // rows: 3.9 us, with 8 each 11.7; 73 thousand rows take 8 either way)
    long long rows = a.total_rows / (32LL * num_sms);
    rows = rows < 1 ? 1 : rows > kLoadRows ? kLoadRows : rows;
    const long long warps = (a.total_rows + rows - 1) / rows;
    long long blocks = (warps + kLoadThreads / 32 - 1) / (kLoadThreads / 32);
    const long long cap = (long long)num_sms * 8;
    if (blocks > cap) blocks = cap;
    if (mode == 2)
        load_kernel<2><<<(unsigned)blocks, kLoadThreads, 0, stream>>>(a, (int)rows);
    else if (mode == 1)
        load_kernel<1><<<(unsigned)blocks, kLoadThreads, 0, stream>>>(a, (int)rows);
    else
        load_kernel<0><<<(unsigned)blocks, kLoadThreads, 0, stream>>>(a, (int)rows);
    return cudaGetLastError();
}

}  // namespace pkv
