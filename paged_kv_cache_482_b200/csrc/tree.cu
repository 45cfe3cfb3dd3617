// tree.cu -- attention of a tree of drafted tokens over the paged cache, on the
// 5th-generation tensor cores (sm_100a).
//
// Sequence s brings c = cu_q_lens[s + 1] - cu_q_lens[s] drafted tokens whose
// K/V are already the last c of its context_lens[s] cached positions. With
// base = context - c, draft j attends to the positions t < base and to the
// drafts u with bit u of its mask set:
//   out[j][h] = sum_t softmax_t(scale * q[j][h] . K_t) V_t
// over those t; a row that sees nothing is zeros.
//
// What bounds it: a cached (token, KV head) pair is 4 d bytes (bf16) and costs
// 4 c G d multiply-adds for the c drafts and G heads that share it, c G per
// byte, and the machine's ratio is some 230: below about that many rows the
// cache's bytes bound the call, above it the tensor cores do.
//
// Work: a unit is (sequence, KV head, 128 NT rows), a row a (draft, head of the
// group) pair. NT = 1 for trees of at most 128 rows: two CTAs per SM, so that
// one's unit changes overlap the other's stream. NT = 2 for wider ones: one CTA
// per SM, every key tile multiplied with two row tiles, which halves the reads.
// The units' key tiles, laid end to end, are cut into equal shares, one per CTA:
// lengths need not be alike, no CTA idles, and a unit is cut only where a share
// ends. A CTA computes its share from the lengths; the partial results of cut
// units (at most two per CTA) go to the workspace and a second kernel joins
// them. Warp roles:
//   4 NT warps  softmax, one row per thread;
//   1 warp      producer: copies 64-token K and V tiles into two rings, its lanes
//               issuing one copy each (blocks smaller than the tile);
//   1 warp      tensor-memory allocation and the MMA issue, S(0), then
//               S(j + 1), P V(j), so that the tensor core forms the next scores
//               while the softmax of tile j runs;
//   2 NT warps  E4M3 only: widen the V codes of a tile into the ring P V reads.
// Tensor memory (256 columns per row tile): two S buffers of 64 columns and O. P
// (16-bit pairs) is written over the S it came from and is the A operand of P V.
// Between units the next queries are loaded (and their first scores formed)
// before the results are written.
//
// Few rows: an E4M3 unit with at most half of its one row tile in use holds two copies
// of its rows, and the warps of copy k handle the k-th half of a tile's keys, with weights
// of zero for the other: a copy is a split of the keys inside the CTA, joined at the end
// of the unit. 64 trees of 16 drafts on 1024-4096 tokens with per-token scales: 196 us,
// without copies 245; 16 of 16 on 16384-32768 with a scale per head: 263 and 282. A bf16
// unit never does (16 of 8 drafts on 16384-32768: with copies 290 us, without 276; 64 ragged
// trees 79 and 74), nor one of two row tiles (head_dim 64: 41.8 and 40.1); four copies of a
// quarter were slower than two.
//
// Operands: a bf16 cache feeds bf16 MMAs. E4M3 keys are the operand as they
// are: Q, scaled per row by a power of two so that its largest element lies in
// [2^7, 2^8), is the sum of two E4M3 values hi + lo (a bf16 value has 8
// significant bits, an E4M3 value 4, so the pair is exact down to 2^-9 of the
// row's largest element and off by at most 2^-17 of it below), and S = hi K^T +
// lo K^T in binary32 -- the tensor time of one 16-bit product, and no key is
// converted. V's codes are widened exactly, to f16 with a scale per KV head, where
// P is rounded to f16 (kF16Lift), and to bf16 with a scale per token, where a weight times its
// token's V scale is rounded to bf16 (whose range any scale fits). One product takes P and V
// in one 16-bit type, so bf16 V needs bf16 P: the outputs are off by 2.3e-3 of their size in
// the mean square (f16 P: 1.7e-3, as with exact weights and the result rounded to bf16). The softmax
// runs in base 2 with a reference maximum that moves only when a key exceeds it by 8; the
// normaliser sums the weights in binary32 as they are before rounding, which is unbiased.
//
// Masked keys: a score that the row does not see becomes -inf whatever it
// was, so its weight is zero; and V elements of drafts that are not finite are
// set to zero in the staged tile (0 * inf would be NaN for the rows that do
// not see the draft) and added to exactly the rows that see them at the end, as
// they are: a seen draft's weight is not zero, though binary32 may hold it as zero.
//
// Measured (B200, GPU time with the join, 32 query and 8 KV heads of 128):
//   64 ragged trees of 1-32 drafts on 100-2048 bf16 tokens    74 us, 3.9 TB/s: in the
//     loop the reads run near the copy rate; unit changes and uneven ends take the rest
//   32 trees of 40-64 drafts on 1000-4096 bf16 tokens        128 us, 2.6 TB/s: two row
//     tiles' exponentials and operand reads from shared memory, per key tile
//   16 trees of 16 drafts on 16384-32768 E4M3 tokens         270 us, 3.0 TB/s: shared
//     memory (hi and lo Q are read again for every 64 keys) and one copy per 16-token block
//   one tree of 8 drafts on 500 bf16 tokens                   13 us: starts of two kernels
//
// Every wait is bounded (PKV_DEVERR_TIMEOUT); every block id and length is
// checked before anything is copied (PKV_DEVERR_BOUNDS).
#include <atomic>

#include "tc_common.cuh"

namespace pkv {

namespace {

using namespace tc;

constexpr int kRows = 128;  // MMA M
constexpr int kBN = 64;     // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
// f16 weights are formed 2^7 larger: the reference maximum may lag by 2^8, so they stay
// below 2^15, and those down to 2^-21 of the reference instead of 2^-14 are normal numbers.
// Behind one key far above all others, the usual state of long contexts, the rest of the
// row is such small weights; unlifted, a row of weights 2^-24 of its largest came out a
// quarter off. The sums carry the same factor, and so it cancels. Below 2^-21 a weight's
// error is at most 2^-32 of the reference's weight.
constexpr float kF16Lift = 7.0f;

template <int D, int MODE, int NT>
struct Tree {
    static constexpr bool kFp8 = MODE != 0;
    static constexpr bool kF16 = MODE == 1;  // type of P and V
    static constexpr bool kTwoCopies = kFp8 && NT == 1;  // units of few rows may hold two copies
    static constexpr int kUnitRows = NT * kRows;
    static constexpr int kSoftmaxWarps = 4 * NT;
    static constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
    static constexpr int kProducerWarp = kSoftmaxWarps;
    static constexpr int kMmaWarp = kSoftmaxWarps + 1;
    static constexpr int kConvWarps = 2 * NT;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 2 + (kFp8 ? kConvWarps : 0));
    static constexpr int kCtasPerSm = NT == 1 ? 2 : 1;
    static constexpr uint32_t kTmemCols = 256 * NT;  // per row tile: S0 | S1 | O
    // ring depths (tiles): keys, V as P V reads it, E4M3 V codes
    static constexpr uint32_t kNK = NT == 1 ? 2 : 4;
    static constexpr uint32_t kNV = NT == 1 ? 2 : (kFp8 ? 3 : 4);
    static constexpr uint32_t kNR = NT == 1 ? 2 : 4;
    static constexpr uint32_t kQTile = kRows * D * 2;  // bf16 [D / 64][rows][128 B]; E4M3 hi, lo [rows][D B]
    static constexpr uint32_t kKSlot = kBN * D * (kFp8 ? 1 : 2);
    static constexpr uint32_t kVSlot = kBN * D * 2;
    static constexpr uint32_t kRSlot = kFp8 ? kBN * D : 0;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + NT * kQTile;
    static constexpr uint32_t kV = kK + kNK * kKSlot;
    static constexpr uint32_t kR = kV + kNV * kVSlot;
    static constexpr uint32_t kKs = kR + kNR * kRSlot;  // per-token scales [slot][kBN] fp32
    static constexpr uint32_t kVs = kKs + (MODE == 2 ? kNK * kBN * 4 : 0);  // both with the tile's K
    static constexpr uint32_t kBar = kVs + (MODE == 2 ? kNK * kBN * 4 : 0);
    static constexpr uint32_t kMl = kBar + 512;  // [2][kUnitRows] fp32: maxima and sums of the copies
    static constexpr uint32_t kOut = kMl + 2 * kUnitRows * 4;  // two copies: [kRows][kOutStride] fp32, 8 columns
    static constexpr int kOutStride = 12;
    static constexpr uint32_t kBytes = kOut + (kTwoCopies ? kRows * kOutStride * 4 : 0);
    static constexpr uint32_t kMin = (NT == 1 ? 80u : 120u) * 1024u;  // no more CTAs per SM than tensor memory has room for
    static constexpr uint32_t kAlloc = kBytes + 1024 > kMin ? kBytes + 1024 : kMin;  // + base alignment
    static_assert(kCtasPerSm * (kAlloc + 1024) <= 228u * 1024u, "shared memory");
};

template <int NT>
struct TreeBars {
    uint64_t q_full;
    uint64_t k_full[4], k_empty[4];
    uint64_t v_full[4], v_empty[4];  // the tile P V reads
    uint64_t r_full[4], r_empty[4];  // E4M3 V codes
    uint64_t s_full[NT][2];
    uint64_t p_full[NT][2];
    uint64_t pv_done[NT];  // per tile; S(j) done and P of tile j missing leave it in phase j - 1 or j
    uint64_t o_done[NT];   // per unit, after its last tile
    uint64_t drained;
    uint32_t tmem;
    int nonfinite[2];  // by unit parity: a draft's V held an infinity or NaN
    int bad[2];        // by unit parity: a block id outside the pool
    int failed;        // a softmax wait gave up
    int unserved;      // some sequence cannot be served
    long long scan[16];  // share computation
};
static_assert(sizeof(TreeBars<2>) <= 512, "barrier space");

// 16-byte chunk c of row r in an operand of `D`-byte rows (E4M3): the 128-byte
// swizzle (D 128) or the 64-byte one (D 64: chunk c of row r at c ^ (r / 2 % 4)).
template <int D>
__device__ __forceinline__ uint32_t swz8(int r, int c) {
    if constexpr (D == 128) return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
    else return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Descriptor of a K-major E4M3 operand with D-byte rows.
template <int D>
__device__ __forceinline__ uint64_t desc8(uint32_t saddr) {
    if constexpr (D == 128) return sw128_desc(saddr, 16, 1024);
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(512 >> 4) << 32) |
           (1ull << 46) | (4ull << 61);
}

__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// 16 consecutive columns of this thread's tensor-memory lane. The load is
// asynchronous: the registers hold the columns after tmem_wait16.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// 8 columns, waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}

// 8 columns into this thread's lane, not waited for: tmem_wait_st() before the
// columns are loaded again.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&w)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Cost of a unit besides its tiles (query loads, first scores, results), in tiles
// (64 ragged trees: 2: 91.7 us, 4: 87.4, 6: 86.0, 8: 86.7).
constexpr int kUnitCost = 6;
// Shares are at least this long where the number of shares is chosen here: a
// shorter one spends most of its time starting and joining (8 drafts on 500
// tokens: 1: 14.2 us, 2: 13.2, 3: 13.7, 4: 15).
constexpr int kMinShare = 2;

// A sequence's work. invalid: lengths that cannot be served.
struct Seq {
    int q0, c, ctx, tiles, row_tiles;
    bool lost, invalid;
    __device__ __forceinline__ long long cost(int nkv) const {
        return static_cast<long long>(row_tiles) * nkv * (tiles + kUnitCost);
    }
};

__device__ __forceinline__ Seq load_seq(const TreeArgs &a, int s, int log2_g) {
    Seq q;
    q.q0 = __ldg(a.cu_q_lens + s);
    const int q1 = __ldg(a.cu_q_lens + s + 1);
    q.ctx = __ldg(a.context_lens + s);
    q.lost = q.q0 < 0 || q1 < q.q0 || q1 > a.total_q;  // its rows cannot be located
    q.c = q.lost ? 0 : q1 - q.q0;
    q.invalid = !q.lost && q.c > 0 && (q.c > a.max_q_len || q.ctx < q.c || q.ctx > a.max_context_len);
    const bool work = !q.lost && !q.invalid && q.c > 0;
    q.tiles = work ? (q.ctx + kBN - 1) / kBN : 0;
    q.row_tiles = work ? ((q.c << log2_g) + a.unit_rows - 1) / a.unit_rows : 0;
    return q;
}

// What a CTA works on at a time; the same in every thread.
struct Unit {
    int s, kh, q0, c, ctx, base;
    int row0;    // first row (draft * G + head)
    int rows;    // live rows
    int per_copy, copies;
    int t0, t1;  // its keys here
    int tiles;   // and their tiles
    int slot;    // workspace slot of a cut unit, -1 of a whole one
};

// All shares: the laid out cost is cut into equal ranges (the first total %
// shares of them one longer); the tiles of a unit at cost p lie at p +
// kUnitCost and behind.
struct Shares {
    long long total, each;
    int shares, longer;
    __device__ __forceinline__ long long begin(int b) const { return each * b + min(b, longer); }
};

// x / y for x >= 0, y > 0: in 32 bits where that does (64-bit divisions are long code).
__device__ __forceinline__ long long divide(long long x, int y) {
    return (x >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}

// The total cost, and the sequence that holds the border `index` of the shares
// (its begin) with the cost before it; for every thread of the block. `scratch`
// is shared memory for 16 values; *unserved (shared memory) is set where a
// sequence cannot be served.
template <int THREADS>
__device__ __forceinline__ Shares find_share(const TreeArgs &a, int log2_g, int index, long long *scratch, int &seq,
                                             long long &before, int *unserved = nullptr) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Shares sh;
    sh.total = sh.each = 0;
    sh.shares = 1;
    sh.longer = 0;
    long long at = 0, cost = 0, done = 0, x = -1;
    const int chunks = (a.num_seqs + THREADS - 1) / THREADS;
    seq = 0;
    before = 0;
    // first round: the total (with one chunk of sequences the border is then
    // looked for at once); second round: the border's chunk
    for (int i = 0; i < 2 * chunks; ++i) {
        const int s = (i < chunks ? i : i - chunks) * THREADS + threadIdx.x;
        if (chunks > 1 || i == 0) {
            if (i == chunks) done = 0;
            cost = 0;
            if (s < a.num_seqs) {
                const Seq q = load_seq(a, s, log2_g);
                cost = q.cost(a.num_kv_heads);
                if (unserved && (q.lost || q.invalid)) *unserved = 1;
            }
            long long inc = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) scratch[warp] = inc;
            __syncthreads();
            at = done + inc;  // cost up to and with this sequence
            for (int w = 0; w < THREADS / 32; ++w) {
                const long long v = scratch[w];
                if (w < warp) at += v;
                done += v;
            }
            __syncthreads();
        }
        if (i == chunks - 1) {
            sh.total = done;
            const long long most = divide(done, a.min_share);
            sh.shares = static_cast<int>(most < 1 ? 1 : most < a.max_shares ? most : a.max_shares);
            sh.each = divide(done, sh.shares);
            sh.longer = static_cast<int>(done - sh.each * sh.shares);
            if (done == 0 || index >= sh.shares) return sh;
            x = sh.begin(index);
        }
        if (i >= chunks && x < done) {  // uniform: the border lies in this chunk
            if (x >= at - cost && x < at) {
                scratch[0] = s;
                scratch[1] = at - cost;
            }
            __syncthreads();
            seq = static_cast<int>(scratch[0]);
            before = scratch[1];
            __syncthreads();
            return sh;
        }
    }
    return sh;
}

// Tiles of a unit of n tiles at cost p before cost x.
__device__ __forceinline__ int tiles_before(long long x, long long p, int n) {
    const long long t = x - p - kUnitCost;
    return t <= 0 ? 0 : t >= n ? n : static_cast<int>(t);
}

// Goes through the units of a share.
struct Walk {
    long long x0, x1, p;  // the share, and the cost of the next unit
    int s, k, share, rows;
    Seq q;
    __device__ __forceinline__ void start(const TreeArgs &a, const Shares &sh, int b, int seq, long long before,
                                          int log2_g, int unit_rows) {
        share = b;
        x0 = sh.begin(b);
        x1 = sh.begin(b + 1);
        s = seq;
        q = load_seq(a, s, log2_g);
        rows = unit_rows;
        k = static_cast<int>(divide(x0 - before, q.tiles + kUnitCost));
        p = before + static_cast<long long>(k) * (q.tiles + kUnitCost);
    }
    __device__ __forceinline__ bool next(const TreeArgs &a, int log2_g, Unit &u) {
        while (p < x1) {
            while (k >= q.row_tiles * a.num_kv_heads) {
                if (++s >= a.num_seqs) return false;
                k = 0;
                q = load_seq(a, s, log2_g);
            }
            const int tb = tiles_before(x0, p, q.tiles), te = tiles_before(x1, p, q.tiles);
            const int kk = k;
            p += q.tiles + kUnitCost;
            ++k;
            if (tb >= te) continue;
            u.s = s;
            u.kh = kk / q.row_tiles;
            u.q0 = q.q0;
            u.c = q.c;
            u.ctx = q.ctx;
            u.base = q.ctx - q.c;
            u.row0 = (kk % q.row_tiles) * rows;
            u.rows = min(rows, (q.c << log2_g) - u.row0);
            u.copies = a.mode != 0 && rows == kRows && u.rows * 2 <= rows ? 2 : 1;
            u.per_copy = rows / u.copies;
            u.t0 = tb * kBN;
            u.t1 = min(q.ctx, te * kBN);
            u.tiles = te - tb;
            u.slot = tb > 0 ? 2 * share : te < q.tiles ? 2 * share + 1 : -1;
            return true;
        }
        return false;
    }
};

// Bits [start, start + 32) of a row's view of the context, position start being
// bit 0: everything below base, the mask's drafts, nothing at or past the end.
__device__ __forceinline__ uint32_t visible32(const uint32_t *mask, int c, int start, int base) {
    auto word = [&](int i) -> uint32_t {
        const int left = c - 32 * i;
        if (left <= 0) return 0u;
        const uint32_t w = __ldg(mask + i);
        return left >= 32 ? w : w & ((1u << left) - 1u);
    };
    const int u = start - base;
    if (u <= -32) return 0xffffffffu;
    if (u < 0) return ((1u << -u) - 1u) | (word(0) << -u);
    const int sh = u & 31;
    const uint32_t lo = word(u >> 5);
    return sh == 0 ? lo : __funnelshift_r(lo, word((u >> 5) + 1), sh);
}

// V rows of the staged tile: rows at or past the end become zeros (zero_tail)
// and elements that are not finite in the drafts' rows too; returns whether
// there were any. F16: f16 elements, else bf16.
template <int D, bool F16, int THREADS>
__device__ __forceinline__ bool mend_v(uint32_t sv, int first, int end, bool zero_tail) {
    constexpr int kChunks = D / 8;
    constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
    bool found = false;
    const int last = zero_tail ? kBN : end;
    for (int i = first * kChunks + threadIdx.x; i < last * kChunks; i += THREADS) {
        const int r = i / kChunks, c16 = i % kChunks;
        const uint32_t at = sv + swz(kBN, r, c16);
        if (r >= end) {
            st_shared16(at, make_uint4(0, 0, 0, 0));
            continue;
        }
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at));
        bool any = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if ((w[k] & kExp) == kExp) {
                w[k] &= 0xFFFF0000u;
                any = true;
            }
            if ((w[k] & (kExp << 16)) == (kExp << 16)) {
                w[k] &= 0x0000FFFFu;
                any = true;
            }
        }
        if (any) {
            st_shared16(at, make_uint4(w[0], w[1], w[2], w[3]));
            found = true;
        }
    }
    return found;
}

// A weight pair, rounded to the operand type.
template <bool F16>
__device__ __forceinline__ uint32_t pack_p(float p0, float p1) { return F16 ? pack_f16(p0, p1) : pack_bf16(p0, p1); }

// Softmax of this warp's rows over the unit's tiles: 64 / copies keys of every
// tile, W at a time in a loop (written out for 64 keys the code outgrew the
// instruction cache: a CTA's first tile took 8000 cycles). g0: tiles of the units
// before. Leaves the reference maximum and the sum of the row (copy).
template <int D, int MODE, int NT, int W>
__device__ __forceinline__ bool softmax_tiles(const TreeArgs &a, const Unit &u, TreeBars<NT> *bars, uint8_t *sm,
                                              uint32_t base, uint32_t tmem, float sl2, bool live, int draft,
                                              uint32_t g0, int unit, float &m_out, float &l_out) {
    using L = Tree<D, MODE, NT>;
    constexpr bool kF16 = L::kF16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp >> 2;  // row tile
    const bool idle = !__any_sync(0xffffffffu, live);  // no row in this warp: its weights are never read
    const int cols = L::kTwoCopies ? kBN / u.copies : kBN, col0 = L::kTwoCopies ? (warp * 32) / u.per_copy * cols : 0;
    const uint32_t *mask = a.mask + static_cast<long long>(u.q0 + draft) * a.mask_words;
    const uint32_t tw = tmem + half * 256 + (static_cast<uint32_t>((warp & 3) * 32) << 16);  // this warp's lanes
    const uint32_t to = tw + 128;
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int j = 0; j < u.tiles; ++j) {
        const uint32_t g = g0 + j;
        const int kv0 = u.t0 + j * kBN;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[half][g & 1], (g >> 1) & 1))) return false;
        tc_fence_after();
        const bool special = kv0 + kBN > u.base;  // holds drafts, or keys past the end
        if (!idle) {
            const uint32_t ts = tw + (g & 1) * kBN;
            uint32_t next[W / 16][16];
#pragma unroll
            for (int i = 0; i < W / 16; ++i) tmem_ld16(ts + col0 + 16 * i, next[i]);
            if (MODE == 2 && !__all_sync(0xffffffffu, mbar_wait(&bars->k_full[g % L::kNK], (g / L::kNK) & 1)))
                return false;
            const float *ks = reinterpret_cast<const float *>(sm + L::kKs) + (g % L::kNK) * kBN;
            const float *vs = reinterpret_cast<const float *>(sm + L::kVs) + (g % L::kNK) * kBN;
            float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
            for (int c = col0; c < col0 + cols; c += W) {
                float x[W];
#pragma unroll
                for (int i = 0; i < W / 16; ++i) tmem_wait16(next[i]);
                // scaled by the row's scale, or by the keys' own (then the row's enters below);
                // the product frees the registers for the next load
#pragma unroll
                for (int i = 0; i < W; i += 4) {
                    float4 k4 = make_float4(sl2, sl2, sl2, sl2);
                    if constexpr (MODE == 2) k4 = *reinterpret_cast<const float4 *>(ks + c + i);
                    const uint32_t *n4 = &next[i / 16][i % 16];
                    const float2 y = __fmul2_rn(make_float2(__uint_as_float(n4[0]), __uint_as_float(n4[1])),
                                                make_float2(k4.x, k4.y));
                    const float2 z = __fmul2_rn(make_float2(__uint_as_float(n4[2]), __uint_as_float(n4[3])),
                                                make_float2(k4.z, k4.w));
                    x[i] = y.x;
                    x[i + 1] = y.y;
                    x[i + 2] = z.x;
                    x[i + 3] = z.y;
                }
                if (c + W < col0 + cols) {
#pragma unroll
                    for (int i = 0; i < W / 16; ++i) tmem_ld16(ts + c + W + 16 * i, next[i]);
                }
                uint32_t vis = 0xffffffffu;
                if (special) {
                    vis = live ? visible32(mask, u.c, kv0 + c, u.base) : 0u;
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if (!((vis >> i) & 1u)) x[i] = -INFINITY;
                }
                float m4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) m4[k] = fmaxf(fmaxf(x[k], x[k + 4]), fmaxf(x[k + 8], x[k + 12]));
#pragma unroll
                for (int i = 16; i < W; ++i) m4[i & 3] = fmaxf(m4[i & 3], x[i]);
                const float mx = (MODE == 2 ? sl2 : 1.0f) * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));  // sl2 > 0
                const bool grow = mx > m + 8.0f;
                if (__any_sync(0xffffffffu, grow)) {
                    // a new reference: what was formed with the old one is scaled. This tile's
                    // earlier steps stored weights (and, if the reference grew, O) without waiting,
                    // and nothing but this wait orders those stores before the loads below.
                    tmem_wait_st();
                    const float alpha = grow ? fast_exp2(m - mx) : 1.0f;  // 0 from m = -inf
                    if (grow) {
                        m = mx;
                        l *= alpha;
                        l2[0] = __fmul2_rn(l2[0], make_float2(alpha, alpha));
                        l2[1] = __fmul2_rn(l2[1], make_float2(alpha, alpha));
                    }
#pragma unroll 1
                    for (int e = col0; e < c; e += 16) {  // this tile's weights
                        uint32_t w[8];
                        tmem_ld8(ts + e / 2, w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const __half2 f = *reinterpret_cast<const __half2 *>(&w[i]);
                            w[i] = pack_p<kF16>((kF16 ? __low2float(f) : bf16lo(w[i])) * alpha,
                                                (kF16 ? __high2float(f) : bf16hi(w[i])) * alpha);
                        }
                        tmem_st8(ts + e / 2, w);
                    }
                    if (j > 0) {  // S(j) done implies P V(j - 2) done: the next phase is P V(j - 1)
                        if (!__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[half], (g - 1) & 1))) return false;
                        tc_fence_after();
#pragma unroll 1
                        for (int ch = 0; ch < D; ch += 8) {
                            uint32_t w[8];
                            tmem_ld8(to + ch, w);
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                            tmem_st8(to + ch, w);
                        }
                    }
                }
                // nothing seen yet: weights exp2(-inf) = 0
                const float ref = m == -INFINITY ? 0.0f : (kF16 ? kF16Lift : 0.0f) - m;
#pragma unroll
                for (int h = 0; h < W / 16; ++h) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {  // 4 keys
                        float2 y[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            y[k] = make_float2(x[16 * h + i + 2 * k], x[16 * h + i + 2 * k + 1]);
                            y[k] = MODE == 2 ? __ffma2_rn(y[k], make_float2(sl2, sl2), make_float2(ref, ref))
                                             : __fadd2_rn(y[k], make_float2(ref, ref));
                            y[k] = make_float2(fast_exp2(y[k].x), fast_exp2(y[k].y));
                            l2[k] = __fadd2_rn(l2[k], y[k]);
                        }
                        if constexpr (MODE == 2) {
                            float4 v4 = *reinterpret_cast<const float4 *>(vs + c + 16 * h + i);
                            if (special) {  // not 0 times a scale that is not finite
                                const uint32_t bits = vis >> (16 * h + i);
                                if (!(bits & 1u)) v4.x = 0.0f;
                                if (!(bits & 2u)) v4.y = 0.0f;
                                if (!(bits & 4u)) v4.z = 0.0f;
                                if (!(bits & 8u)) v4.w = 0.0f;
                            }
                            y[0] = __fmul2_rn(y[0], make_float2(v4.x, v4.y));
                            y[1] = __fmul2_rn(y[1], make_float2(v4.z, v4.w));
                        }
                        w[i / 2] = pack_p<kF16>(y[0].x, y[0].y);
                        w[i / 2 + 1] = pack_p<kF16>(y[1].x, y[1].y);
                    }
                    tmem_st8(ts + c / 2 + 8 * h, w);
                }
            }
            l += (l2[0].x + l2[1].x) + (l2[0].y + l2[1].y);
            if (cols < kBN) {  // the other copies' keys
                const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                for (int c = cols / 2; c < kBN / 2; c += 8) tmem_st8(ts + ((col0 / 2 + c) & 31), zero);
            }
        }
        if constexpr (MODE == 2) {
            // here, behind instructions that used every lane's scales: released right
            // after their loads, the slot was refilled under lanes still reading it
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->k_empty[g % L::kNK]);
        }
        if (special) {
            const uint32_t slot = g % L::kNV;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->v_full[slot], (g / L::kNV) & 1))) return false;
            const int first = max(0, u.base - kv0), end = min(kBN, u.ctx - kv0);
            if (mend_v<D, kF16, L::kSoftmaxThreads>(base + L::kV + slot * L::kVSlot, first, end, MODE == 0))
                bars->nonfinite[unit & 1] = 1;
            fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[half][g & 1]);
    }
    // a barrier of its own: pv_done may be one or two phases further by now, and
    // a parity cannot tell which
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->o_done[half], unit & 1))) return false;
    tc_fence_after();
    m_out = m;
    l_out = l;
    return true;
}

// The elements of the seen drafts' V that are not finite, added to N columns
// from col of a row of the result (they were zero in the staged tiles).
template <int D, int MODE, int N>
__device__ __noinline__ void nonfinite_sum(const TreeArgs &a, const Unit &u, int draft, int col, float *v) {
    const uint32_t *mask = a.mask + static_cast<long long>(u.q0 + draft) * a.mask_words;
    const int32_t *table = a.block_tables + static_cast<long long>(u.s) * a.max_blocks_per_seq;
    for (int t = max(u.t0, u.base); t < u.t1; ++t) {
        const int d = t - u.base;
        if (!((__ldg(mask + (d >> 5)) >> (d & 31)) & 1u)) continue;
        const long long row = (static_cast<long long>(table[t / a.block_size]) * a.num_kv_heads + u.kh) * a.block_size +
                              t % a.block_size;
        for (int i = 0; i < N; ++i) {
            const long long e = row * D + col + i;
            float x;
            if constexpr (MODE == 0) {
                x = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v_cache)[e]);
            } else {
                x = e4m3x2_to_float2(static_cast<const uint8_t *>(a.v_cache)[e]).x;  // a scale enters with the weights
            }
            if (!isfinite(x)) v[i] += x;
        }
    }
}

template <int D, int MODE, int N>
__device__ __forceinline__ void add_nonfinite(const TreeArgs &a, const Unit &u, int draft, int col, float (&v)[N]) {
    float t[N];  // addressed only here, so that v stays in registers
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = v[i];
    nonfinite_sum<D, MODE, N>(a, u, draft, col, t);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = t[i];
}

// Results of a unit: normalised, the copies joined (through shared memory, 16
// columns at a time), written as bf16 or as the partial, maximum and sum of a
// cut unit.
template <int D, int MODE, int NT>
__device__ __forceinline__ void write_unit(const TreeArgs &a, const Unit &u, TreeBars<NT> *bars, uint8_t *sm,
                                           uint32_t tmem, int unit, int log2_g, bool ok, float m, float l) {
    using L = Tree<D, MODE, NT>;
    constexpr int kUnitRows = L::kUnitRows, kThreads = L::kSoftmaxThreads;
    const int tid = threadIdx.x, warp = tid >> 5, G = 1 << log2_g;
    const int r = tid & (u.per_copy - 1), copy = tid / u.per_copy;
    float *ml = reinterpret_cast<float *>(sm + L::kMl);
    float *o = reinterpret_cast<float *>(sm + L::kOut);
    ml[tid] = m;
    ml[kUnitRows + tid] = ok ? l : 0.0f;
    named_sync(1, kThreads);  // (also: the flags are complete)
    const bool bad = bars->bad[unit & 1] != 0, nonfinite = bars->nonfinite[unit & 1] != 0 && !bad;
    float top = -INFINITY, sum = 0.0f;
    for (int k = 0; k < u.copies; ++k) top = fmaxf(top, ml[k * u.per_copy + r]);
    const float ref = top == -INFINITY ? 0.0f : top;
    for (int k = 0; k < u.copies; ++k)
        sum = fmaf(fast_exp2(ml[k * u.per_copy + r] - ref), ml[kUnitRows + k * u.per_copy + r], sum);
    // a copy (or row) that saw nothing, and a bad unit, contribute zeros whatever O holds
    const bool drop = l == 0.0f || sum == 0.0f || bad || !ok;
    const float f = drop ? 0.0f : fast_exp2(m - ref) * ((MODE == 1 ? __ldg(a.v_scale + u.kh) : 1.0f) / sum);
    const bool live = r < u.rows;
    const int row = u.row0 + (live ? r : 0), draft = row >> log2_g;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) +
                         (static_cast<long long>(u.q0 + draft) * a.num_q_heads + u.kh * G + (row & (G - 1))) * D;
    const long long prow = static_cast<long long>(u.slot) * a.slot_rows + r;
    float *part = a.part_o + prow * D;
    if (u.slot >= 0 && live && copy == 0)
        *reinterpret_cast<float2 *>(a.part_ml + prow * 2) = make_float2(top, bad ? -1.0f : sum);
    const uint32_t to = tmem + (warp >> 2) * 256 + 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool two = L::kTwoCopies && u.copies == 2;
#pragma unroll 1
    for (int col = 0; col < D; col += 16) {
        uint32_t w[16];
        tmem_ld16(to + col, w);
        tmem_wait16(w);
        float v[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i / 8][i % 8] = drop ? 0.0f : __uint_as_float(w[i]) * f;
        if (two) {  // copy k keeps the columns 8 k .. 8 k + 7 and hands over the others
            float *mine = o + tid * L::kOutStride;
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<float4 *>(mine + i) =
                    copy ? make_float4(v[0][i], v[0][i + 1], v[0][i + 2], v[0][i + 3])
                         : make_float4(v[1][i], v[1][i + 1], v[1][i + 2], v[1][i + 3]);
            named_sync(1, kThreads);
        }
        if (live) {
#pragma unroll 1
            for (int h = copy; h < 2; h += u.copies) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = h ? v[1][i] : v[0][i];
                if (two) {
                    const float *other = o + (tid ^ (kRows / 2)) * L::kOutStride;
                    const float4 y = *reinterpret_cast<const float4 *>(other);
                    const float4 z = *reinterpret_cast<const float4 *>(other + 4);
                    x[0] += y.x;
                    x[1] += y.y;
                    x[2] += y.z;
                    x[3] += y.w;
                    x[4] += z.x;
                    x[5] += z.y;
                    x[6] += z.z;
                    x[7] += z.w;
                }
                const int c8 = col + 8 * h;
                if (nonfinite) add_nonfinite<D, MODE>(a, u, draft, c8, x);
                if (u.slot < 0) {
                    *reinterpret_cast<uint4 *>(out + c8) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                                      pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                } else {
                    // whole 32-byte sectors (the workspace is 256-byte aligned)
                    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(part + c8), "f"(x[0]),
                                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                                 : "memory");
                }
            }
        }
        if (two) named_sync(1, kThreads);
    }
    named_sync(1, kThreads);  // the flags are read
    if (tid == 0) {
        if (bad) set_error(a.dev_err, PKV_DEVERR_BOUNDS);
        bars->nonfinite[unit & 1] = 0;  // next used two units on
        bars->bad[unit & 1] = 0;
    }
}

// The unit's queries into shared memory (every copy of a row), the softmax
// scale of this thread's row, and the check of the unit's block ids.
template <int D, int MODE, int NT>
__device__ __forceinline__ float load_queries(const TreeArgs &a, const Unit &u, TreeBars<NT> *bars, uint32_t base,
                                              int unit, int log2_g, int log2_bs) {
    using L = Tree<D, MODE, NT>;
    constexpr int kChunks = D / 8;
    const int tid = threadIdx.x, G = 1 << log2_g;
    float sl2 = a.scale * kLog2e;
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q);
    auto row_of = [&](int row) {
        return (static_cast<long long>(u.q0 + (row >> log2_g)) * a.num_q_heads + u.kh * G + (row & (G - 1))) * D;
    };
    if constexpr (!L::kFp8) {
        for (int i = tid; i < L::kUnitRows * kChunks; i += L::kSoftmaxThreads) {
            const int p = i / kChunks, c16 = i % kChunks;
            const int r = p & (u.per_copy - 1);
            const bool ok = r < u.rows;
            cp_async16(base + L::kQ + (p / kRows) * L::kQTile + swz(kRows, p % kRows, c16),
                       qp + row_of(u.row0 + (ok ? r : 0)) + c16 * 8, ok ? 16u : 0u);
        }
        cp_async_commit();
    } else {
        const int r = tid & (u.per_copy - 1);
        const bool live = r < u.rows;
        const uint4 *qrow = reinterpret_cast<const uint4 *>(qp + row_of(u.row0 + (live ? r : 0)));
        float amax = 0.0f;
        if (live) {
#pragma unroll 8
            for (int c16 = 0; c16 < kChunks; ++c16) {
                const uint4 v4 = __ldg(qrow + c16);
                const uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16lo(w[k])), fabsf(bf16hi(w[k]))));
            }
        }
        // amax < 2^e; times 2^kq it lies in [2^7, 2^8). kq is capped at 60 so that
        // 2^-kq times the softmax scale stays normal: rows that small have scores
        // of zero to binary32 against any finite key.
        const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFF) - 126;
        const int kq = min(60, 8 - e);
        float qs = __int_as_float((kq + 127) << 23);
        sl2 *= __int_as_float((127 - kq) << 23);
        if (MODE == 1) {  // the scale's sign goes into the queries, so that sl2 stays positive
            const float ks = __ldg(a.k_scale + u.kh);
            sl2 *= fabsf(ks);
            if (ks < 0.0f) qs = -qs;
        }
        // an infinite query, which E4M3 has not, makes NaN of its row's operand: of every score then, but not of
        // the row's scale, which enters behind the mask and would reach masked keys
        if (!(amax <= 3.4e38f)) qs = __int_as_float(0x7FC00000);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {  // 16 elements: one chunk of hi and of lo
            const uint4 v0 = live ? __ldg(qrow + 2 * c) : make_uint4(0, 0, 0, 0);
            const uint4 v1 = live ? __ldg(qrow + 2 * c + 1) : make_uint4(0, 0, 0, 0);
            const uint32_t wv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float x = bf16lo(wv[k]) * qs, y = bf16hi(wv[k]) * qs;
                const uint16_t h = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
                const float2 hf = e4m3x2_to_float2(h);
                const uint16_t o = __nv_cvt_float2_to_fp8x2(make_float2(x - hf.x, y - hf.y), __NV_SATFINITE, __NV_E4M3);
                if (k & 1) {
                    hi[k >> 1] |= static_cast<uint32_t>(h) << 16;
                    lo[k >> 1] |= static_cast<uint32_t>(o) << 16;
                } else {
                    hi[k >> 1] = h;
                    lo[k >> 1] = o;
                }
            }
            const uint32_t at = base + L::kQ + (tid / kRows) * L::kQTile + swz8<D>(tid % kRows, c);
            st_shared16(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            st_shared16(at + kRows * D, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
    }
    // the producer copies block 0 in place of an id outside the pool; the results become zeros
    const int32_t *table = a.block_tables + static_cast<long long>(u.s) * a.max_blocks_per_seq;
    for (int i = (u.t0 >> log2_bs) + tid; i <= (u.t1 - 1) >> log2_bs; i += L::kSoftmaxThreads) {
        const int id = __ldg(table + i);
        if (id < 0 || id >= a.num_blocks) bars->bad[unit & 1] = 1;
    }
    if constexpr (!L::kFp8) cp_async_wait0();
    fence_proxy_async_smem();
    mbar_arrive(&bars->q_full);
    return sl2 < 1.17549435e-38f ? 1.17549435e-38f : sl2;  // not 0, which a masked score's -inf turns into NaN
}

template <int D, int MODE, int NT>
__global__ void __launch_bounds__(Tree<D, MODE, NT>::kThreads, Tree<D, MODE, NT>::kCtasPerSm)
    tree_kernel(const __grid_constant__ TreeArgs a, int log2_bs, int log2_g, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
    using L = Tree<D, MODE, NT>;
    constexpr bool kFp8 = L::kFp8;
    constexpr int kThreads = L::kThreads;
    constexpr uint32_t kNK = L::kNK, kNV = L::kNV, kNR = L::kNR;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw);
    TreeBars<NT> *bars = reinterpret_cast<TreeBars<NT> *>(sm + L::kBar);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = a.block_size;

    // the join kernel may take free slots now: it finds its borders meanwhile, and waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ------------------------------------------------ setup
    if (warp == L::kMmaWarp) tmem_alloc(smem_addr(&bars->tmem), L::kTmemCols);
    if (tid == 0) {
        mbar_init(&bars->q_full, L::kSoftmaxThreads);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], MODE == 2 ? 1 + L::kSoftmaxWarps : 1);  // the softmax reads the scales
            mbar_init(&bars->v_full[i], kFp8 ? L::kConvWarps : 1);
            mbar_init(&bars->v_empty[i], 1);
            mbar_init(&bars->r_full[i], 1);
            mbar_init(&bars->r_empty[i], L::kConvWarps);
        }
        for (int x = 0; x < NT; ++x) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars->s_full[x][i], 1);
                mbar_init(&bars->p_full[x][i], 4);
            }
            mbar_init(&bars->pv_done[x], 1);
            mbar_init(&bars->o_done[x], 1);
        }
        mbar_init(&bars->drained, 1);
        bars->nonfinite[0] = bars->nonfinite[1] = 0;
        bars->bad[0] = bars->bad[1] = 0;
        bars->failed = bars->unserved = 0;
        fence_barrier_init();
    }
    const int share = blockIdx.x;
    int seq;
    long long before;
    __syncthreads();  // barriers and flags are set
    const Shares sh = find_share<kThreads>(a, log2_g, share, bars->scan, seq, before, &bars->unserved);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (bars->unserved) {
        // sequences that cannot be served: reported, and zeros where their rows can be located
        for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
            const Seq q = load_seq(a, s, log2_g);
            if ((q.lost || q.invalid) && tid == 0) set_error(a.dev_err, PKV_DEVERR_BOUNDS);
            if (q.invalid) {
                const long long n = static_cast<long long>(q.c) * a.num_q_heads * (D / 8);
                uint4 *dst = static_cast<uint4 *>(a.out) + static_cast<long long>(q.q0) * a.num_q_heads * (D / 8);
                for (long long i = tid; i < n; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
            }
        }
    }
    const uint32_t tmem = bars->tmem;
    const bool work = sh.total > 0 && share < sh.shares;
    Walk walk;
    Unit u;
    uint32_t g = 0;  // tiles of the units before
    if (work) walk.start(a, sh, share, seq, before, log2_g, L::kUnitRows);

    if (!work) {
        // more CTAs than shares
    } else if (warp < L::kSoftmaxWarps) {
        // ================================================ softmax
        bool more = walk.next(a, log2_g, u);
        float sl2 = more ? load_queries<D, MODE, NT>(a, u, bars, base, 0, log2_g, log2_bs) : 0.0f;
        for (int unit = 0; more; ++unit) {
            // this thread's row (of copy tid / per_copy)
            const int r = tid & (u.per_copy - 1);
            const bool live = r < u.rows;
            const int draft = (u.row0 + (live ? r : 0)) >> log2_g;
            float m = -INFINITY, l = 0.0f;
            const bool ok = softmax_tiles<D, MODE, NT, 32>(a, u, bars, sm, base, tmem, sl2, live, draft, g, unit, m, l);
            if (!ok && lane == 0) {
                set_error(a.dev_err, PKV_DEVERR_TIMEOUT);
                bars->failed = 1;
            }
            g += u.tiles;
            // O is complete, so every S is: the next queries may replace these
            Unit next;
            more = walk.next(a, log2_g, next);
            if (more) sl2 = load_queries<D, MODE, NT>(a, next, bars, base, unit + 1, log2_g, log2_bs);
            write_unit<D, MODE, NT>(a, u, bars, sm, tmem, unit, log2_g, ok, m, l);
            if (bars->failed) break;  // written before a barrier of write_unit: the same for all
            u = next;
        }
        __syncwarp();
    } else if (warp == L::kProducerWarp) {
        // ================================================ producer
        constexpr int kHalves = D / 64;
        bool ok = true;
        uint32_t issued_k = 0, issued_v = 0;
        while (ok && walk.next(a, log2_g, u)) {
            const int32_t *table = a.block_tables + static_cast<long long>(u.s) * a.max_blocks_per_seq;
            // block ids, 32 at a time, the next 32 already loading
            const int last_blk = (u.t1 - 1) >> log2_bs;
            int win = u.t0 >> log2_bs;
            int id = __ldg(table + min(win + lane, last_blk)), id_next = __ldg(table + min(win + 32 + lane, last_blk));
            for (int j = 0; j < u.tiles; ++j) {
                const int kv0 = u.t0 + j * kBN;
                const int blk0 = kv0 >> log2_bs;
                if (blk0 >= win + 32) {
                    win += 32;
                    id = id_next;
                    id_next = __ldg(table + min(win + 32 + lane, last_blk));
                }
                const int run = min(bs, kBN);  // rows per copy
                const int n = bs >= kBN ? 1 : (min(kv0 + kBN, u.t1) - kv0 + bs - 1) >> log2_bs;
                // lane i handles block i of the tile (bf16: lane kHalves i + half)
                const int bi = kFp8 ? lane : lane / kHalves;
                const int half = kFp8 ? 0 : lane % kHalves;
                int blk = __shfl_sync(0xffffffffu, id, (blk0 - win + min(bi, n - 1)) & 31);
                if (blk < 0 || blk >= a.num_blocks) blk = 0;
                const long long prow = (static_cast<long long>(blk) * a.num_kv_heads + u.kh) * bs + (kv0 & (bs - 1));
                const bool mine = bi < n;
                const uint32_t t = g + j;
                auto stage = [&](bool is_k) -> bool {
                    constexpr uint32_t kN2 = kFp8 ? kNR : kNV;
                    const uint32_t slot = is_k ? t % kNK : t % kN2, use = is_k ? t / kNK : t / kN2;
                    uint64_t *empty = is_k ? &bars->k_empty[slot] : kFp8 ? &bars->r_empty[slot] : &bars->v_empty[slot];
                    uint64_t *full = is_k ? &bars->k_full[slot] : kFp8 ? &bars->r_full[slot] : &bars->v_full[slot];
                    if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(empty, (use - 1) & 1))) return false;
                    const uint32_t bytes = static_cast<uint32_t>(n * run) * (D * (kFp8 ? 1 : 2) + (MODE == 2 && is_k ? 8 : 0));
                    if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                    __syncwarp();
                    if (mine) {
                        if constexpr (!kFp8) {
                            const uint32_t dst = base + (is_k ? L::kK + slot * L::kKSlot : L::kV + slot * L::kVSlot);
                            tma_load_2d(dst + half * kBN * 128 + bi * run * 128, is_k ? &map_k : &map_v, half * 64,
                                        static_cast<int>(prow), full);
                        } else {
                            if (is_k)
                                tma_load_2d(base + L::kK + slot * L::kKSlot + bi * run * D, &map_k, 0,
                                            static_cast<int>(prow), full);
                            else
                                bulk_g2s(sm + L::kR + slot * L::kRSlot + bi * run * D,
                                         static_cast<const uint8_t *>(a.v_cache) + prow * D, run * D, full);
                            if (MODE == 2 && is_k) {
                                bulk_g2s(sm + L::kKs + slot * kBN * 4 + bi * run * 4, a.k_scale + prow, run * 4, full);
                                bulk_g2s(sm + L::kVs + slot * kBN * 4 + bi * run * 4, a.v_scale + prow, run * 4, full);
                            }
                        }
                    }
                    return true;
                };
#pragma unroll 1
                for (int which = 0; which < 2 && ok; ++which) {
                    ok = stage(which == 0);
                    if (ok) (which == 0 ? issued_k : issued_v) = t + 1;
                }
                if (!ok) break;
            }
            g += u.tiles;
        }
        __syncwarp();
        if (lane == 0) {
            if (!ok) set_error(a.dev_err, PKV_DEVERR_TIMEOUT);
            // copies still in flight (only after a timeout): wait for them before the CTA exits
            for (uint32_t j = issued_k > kNK ? issued_k - kNK : 0; j < issued_k; ++j)
                mbar_wait(&bars->k_full[j % kNK], (j / kNK) & 1);
            constexpr uint32_t kN2 = kFp8 ? kNR : kNV;
            for (uint32_t j = issued_v > kN2 ? issued_v - kN2 : 0; j < issued_v; ++j)
                mbar_wait(kFp8 ? &bars->r_full[j % kN2] : &bars->v_full[j % kN2], (j / kN2) & 1);
        }
        __syncwarp();
    } else if (warp == L::kMmaWarp) {
        // ================================================ MMA issue
        // The whole warp walks and waits, one elected lane issues: operands that
        // are the same in every lane stay in uniform registers, which the MMA
        // takes them from (from one lane alone, moving them there took longer
        // than the products).
        constexpr uint32_t kIdescS = kFp8 ? idesc_f16(kRows, kBN, false) : idesc_bf16(kRows, kBN, false);
        constexpr uint32_t kIdescPV = MODE == 1 ? idesc_f16(kRows, D, true) : idesc_bf16(kRows, D, true);
        const bool leader = elect_one();
        auto wait_all = [](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity));
        };
        const uint64_t dq = kFp8 ? desc8<D>(base + L::kQ) : sw128_desc(base + L::kQ, 16, 1024);
        const uint64_t dk = kFp8 ? desc8<D>(base + L::kK) : sw128_desc(base + L::kK, 16, 1024);
        const uint64_t dv = sw128_desc(base + L::kV, kBN * 128, 1024);
        // descriptors count 16-byte units; the shared-memory window is below their 14 bits' 256 KB
        auto issue_s = [&](uint32_t t) -> bool {
            const uint32_t slot = t % kNK;
            if (!wait_all(&bars->k_full[slot], (t / kNK) & 1)) return false;
            tc_fence_after();
            const uint64_t dks = dk + slot * (L::kKSlot >> 4);
            if (leader) {
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    const uint64_t dqx = dq + x * (L::kQTile >> 4);
                    const uint32_t ts = tmem + x * 256 + (t & 1) * kBN;
                    if constexpr (kFp8) {  // E4M3: format code 0 for A and B, 32 elements per step; hi, then lo
#pragma unroll
                        for (int kk = 0; kk < 2 * (D / 32); ++kk)
                            mma_f8(ts, dqx + (kk / (D / 32)) * (kRows * D >> 4) + (kk % (D / 32)) * 2,
                                   dks + (kk % (D / 32)) * 2, kIdescS, kk > 0 ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_bf16(ts, dqx + (kk >> 2) * (kRows * 128 >> 4) + (kk & 3) * 2,
                                     dks + (kk >> 2) * (kBN * 128 >> 4) + (kk & 3) * 2, kIdescS, kk > 0 ? 1u : 0u);
                    }
                    if (x == NT - 1) mma_commit(&bars->k_empty[slot]);
                    mma_commit(&bars->s_full[x][t & 1]);
                }
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        for (int unit = 0; ok && walk.next(a, log2_g, u); ++unit) {
            ok = wait_all(&bars->q_full, unit & 1) && issue_s(g);
            for (int j = 0; ok && j < u.tiles; ++j) {
                const uint32_t t = g + j, slot = t % kNV;
                // the next tile's S buffer was P of tile j - 1, which P V(j - 1) read before
                if (j + 1 < u.tiles) ok = issue_s(t + 1);
                ok = ok && wait_all(&bars->v_full[slot], (t / kNV) & 1);
                // every softmax warp mends a part of the V of a tile with drafts
                if (NT > 1 && ok && u.t0 + (j + 1) * kBN > u.base)
                    for (int x = 1; x < NT && ok; ++x) ok = wait_all(&bars->p_full[x][t & 1], (t >> 1) & 1);
                const uint64_t dvs = dv + slot * (L::kVSlot >> 4);
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    ok = ok && wait_all(&bars->p_full[x][t & 1], (t >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kBN / 16; ++kk)
                            mma_bf16_ts(tmem + x * 256 + 128, tmem + x * 256 + (t & 1) * kBN + kk * 8,
                                        dvs + kk * (16 * 128 >> 4), kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
                        if (x == NT - 1) mma_commit(&bars->v_empty[slot]);
                        mma_commit(&bars->pv_done[x]);
                        if (j + 1 == u.tiles) mma_commit(&bars->o_done[x]);
                    }
                    __syncwarp();
                }
            }
            g += u.tiles;
        }
        if (leader) {
            if (!ok) set_error(a.dev_err, PKV_DEVERR_TIMEOUT);
            // every MMA issued so far has finished before tensor memory is freed
            mma_commit(&bars->drained);
            mbar_wait(&bars->drained, 0);
        }
        __syncwarp();
    } else if constexpr (kFp8) {
        // ================================================ V converters
        constexpr int kCT = L::kConvWarps * 32;
        constexpr int kCPR = D / 16;  // 16-code chunks per row
        // a thread's chunks lie a multiple of 8 rows apart: one swizzle for all
        constexpr int kRowStep = kCT / kCPR, kIters = kBN / kRowStep, kTogether = kIters < 4 ? kIters : 4;
        static_assert(kRowStep % 8 == 0 && kIters % kTogether == 0, "whole steps");
        const int ct = tid - 32 * (L::kMmaWarp + 1);
        const int row = ct / kCPR;
        const uint32_t to_lo = swz(kBN, row, 2 * (ct % kCPR)), to_hi = swz(kBN, row, 2 * (ct % kCPR) + 1);
        bool ok = true;
        while (ok && walk.next(a, log2_g, u)) {
            for (int j = 0; j < u.tiles; ++j) {
                const uint32_t t = g + j, slot = t % kNV, rslot = t % kNR;
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->r_full[rslot], (t / kNR) & 1)) ||
                    (t >= kNV && !__all_sync(0xffffffffu, mbar_wait(&bars->v_empty[slot], (t / kNV - 1) & 1)))) {
                    ok = false;
                    break;
                }
                const int end = min(kBN, u.t1 - (u.t0 + j * kBN));  // rows past the end become zeros
                const uint32_t src = base + L::kR + rslot * L::kRSlot + ct * 16;
                const uint32_t dst = base + L::kV + slot * L::kVSlot;
#pragma unroll
                for (int i0 = 0; i0 < kIters; i0 += kTogether) {
                    uint4 w[kTogether];
#pragma unroll
                    for (int i = 0; i < kTogether; ++i)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                                     : "r"(src + (i0 + i) * kCT * 16));
#pragma unroll
                    for (int i = 0; i < kTogether; ++i) {
                        const int down = (i0 + i) * kRowStep;  // rows below this thread's first
                        uint4 lo, hi;
                        if constexpr (MODE == 2) {
                            lo = e4m3x8_to_bf16x8(make_uint2(w[i].x, w[i].y));
                            hi = e4m3x8_to_bf16x8(make_uint2(w[i].z, w[i].w));
                        } else {
                            const uint2 h0 = e4m3x4_to_f16x4(w[i].x), h1 = e4m3x4_to_f16x4(w[i].y);
                            const uint2 h2 = e4m3x4_to_f16x4(w[i].z), h3 = e4m3x4_to_f16x4(w[i].w);
                            lo = make_uint4(h0.x, h0.y, h1.x, h1.y);
                            hi = make_uint4(h2.x, h2.y, h3.x, h3.y);
                        }
                        if (row + down >= end) lo = hi = make_uint4(0, 0, 0, 0);
                        st_shared16(dst + to_lo + down * 128, lo);
                        st_shared16(dst + to_hi + down * 128, hi);
                    }
                }
                fence_proxy_async_smem();  // P V reads the tile through the async proxy
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->v_full[slot]);
                    mbar_arrive(&bars->r_empty[rslot]);
                }
            }
            g += u.tiles;
        }
        if (!ok && lane == 0) set_error(a.dev_err, PKV_DEVERR_TIMEOUT);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == L::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Join of the cut units: the blocks (i, *) look at the border between the shares
// i and i + 1; if it cuts a unit, they make its part of that unit's results (the
// borders inside one unit divide its results among them). It may start before
// the attention kernel has ended, and waits for that once it knows its part.
// Block 0 waits even with nothing to join: what the stream runs next is ordered
// behind this kernel's end, which must not come before the attention kernel's.
constexpr int kJoinThreads = 256;
// Blocks per border (64 ragged trees of 128 rows, both kernels: 1: 101 us, 2: 82, 4:
// 79.6, 8: 83, 16: 94; most borders' blocks find nothing to join).
constexpr int kJoinSplit = 4;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a, int log2_g) {
    __shared__ long long scratch[16];
    const int tid = threadIdx.x, G = 1 << log2_g;
    const int border = blockIdx.x / kJoinSplit + 1;
    int s;
    long long p;
    const Shares sh = find_share<kJoinThreads>(a, log2_g, border, scratch, s, p);
    if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (sh.total == 0 || border >= sh.shares) return;
    const long long x = sh.begin(border);
    const Seq q = load_seq(a, s, log2_g);
    const int k = static_cast<int>(divide(x - p, q.tiles + kUnitCost));
    p += static_cast<long long>(k) * (q.tiles + kUnitCost);
    const int cut = tiles_before(x, p, q.tiles);
    if (cut == 0 || cut == q.tiles) return;
    int first = border - 1, end = border + 1;  // the shares that hold a piece
    while (tiles_before(sh.begin(first), p, q.tiles) > 0) --first;
    while (end < sh.shares && tiles_before(sh.begin(end), p, q.tiles) < q.tiles) ++end;
    const int pieces = end - first;
    const int part = (border - 1 - first) * kJoinSplit + blockIdx.x % kJoinSplit, parts = (pieces - 1) * kJoinSplit;
    const int kh = k / q.row_tiles, row0 = (k % q.row_tiles) * a.unit_rows;
    const int rows = min(a.unit_rows, (q.c << log2_g) - row0);
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
    // a unit's first piece is in its share's second slot, the others in the first ones
    auto slot = [&](int i) { return static_cast<long long>(i == 0 ? 2 * first + 1 : 2 * (first + i)) * a.slot_rows; };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = part * kJoinThreads + tid; i < rows * (D / 4); i += parts * kJoinThreads) {
        const int r = i / (D / 4), col = (i % (D / 4)) * 4;
        float top = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0, 0, 0, 0);
        bool bad = false;
#pragma unroll 2
        for (int n = 0; n < pieces; ++n) {
            const long long at = slot(n) + r;
            const float2 y = __ldcg(ml + at);
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D + col));
            bad |= y.y < 0.0f;
            if (y.y == 0.0f) continue;  // a piece that the row saw nothing of
            const float next = fmaxf(top, y.x), ref = next == -INFINITY ? 0.0f : next;
            const float f = fast_exp2(top - ref), w = fast_exp2(y.x - ref) * y.y;  // f is 0 from top = -inf
            top = next;
            sum = fmaf(sum, f, w);
            acc.x = fmaf(w, o.x, acc.x * f);
            acc.y = fmaf(w, o.y, acc.y * f);
            acc.z = fmaf(w, o.z, acc.z * f);
            acc.w = fmaf(w, o.w, acc.w * f);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int row = row0 + r;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                             (static_cast<long long>(q.q0 + (row >> log2_g)) * a.num_q_heads + kh * G + (row & (G - 1))) * D +
                             col;
        *reinterpret_cast<uint2 *>(dst) = bad ? make_uint2(0, 0)
                                              : make_uint2(pack_bf16(acc.x * inv, acc.y * inv),
                                                           pack_bf16(acc.z * inv, acc.w * inv));
    }
}

// The pool as a 2-D tensor of rows: boxes of 64 bf16 columns (128-byte swizzle)
// or whole E4M3 rows (128- or 64-byte swizzle) of min(block_size, kBN) rows.
bool make_map(CUtensorMap *map, const void *pool, const TreeArgs &a) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool fp8 = a.mode != 0;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.head_dim),
                                static_cast<cuuint64_t>(a.num_blocks) * a.num_kv_heads * a.block_size};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.head_dim) * (fp8 ? 1 : 2)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(fp8 ? a.head_dim : 64),
                               static_cast<cuuint32_t>(a.block_size < kBN ? a.block_size : kBN)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(pool),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              fp8 && a.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int MODE, int NT>
cudaError_t launch_mode(const TreeArgs &a, cudaStream_t stream) {
    using L = Tree<D, MODE, NT>;
    const int g = a.num_q_heads / a.num_kv_heads;
    int log2_bs = 0, log2_g = 0;
    while ((1 << log2_bs) < a.block_size) ++log2_bs;
    while ((1 << log2_g) < g) ++log2_g;
    // row coordinates of the tensor maps are int32
    if (a.num_blocks * a.num_kv_heads * a.block_size > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    CUtensorMap mk, mv;
    memset(&mv, 0, sizeof(mv));
    if (!make_map(&mk, a.k_cache, a) || (MODE == 0 && !make_map(&mv, a.v_cache, a))) return cudaErrorInvalidValue;
    auto kern = tree_kernel<D, MODE, NT>;
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L::kAlloc));
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    kern<<<a.max_shares, L::kThreads, L::kAlloc, stream>>>(a, log2_bs, log2_g, mk, mv);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.max_shares == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.max_shares - 1) * kJoinSplit);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<D>, a, log2_g);
}

}  // namespace

// One or two row tiles per unit: two once a tree may have more rows than a tile
// (they share every key tile then). Trees of up to 256 rows: one 144 us, two 127; of
// up to 168 rows, head_dim 64: 41.2 either way. Of up to 128 rows: one 74.7 us, two 99.6;
// of 64 rows on long contexts 270 and 421.
int tree_unit_rows(int max_q_len, int group) {
    return static_cast<long long>(max_q_len) * group > kRows ? 2 * kRows : kRows;
}
int tree_ctas_per_sm(int max_q_len, int group) { return tree_unit_rows(max_q_len, group) == kRows ? 2 : 1; }
int tree_slot_rows(int max_q_len, int group) {
    const long long rows = static_cast<long long>(max_q_len) * group;
    const int unit = tree_unit_rows(max_q_len, group);
    return rows < unit ? static_cast<int>(rows) : unit;
}
int tree_min_share() { return kMinShare; }
// The most shares that lengths within these bounds can make.
long long tree_max_shares(int num_seqs, int num_kv_heads, int group, int max_q_len, int max_context_len) {
    const double units = static_cast<double>(num_seqs) * num_kv_heads *
                         ((static_cast<long long>(max_q_len) * group + tree_unit_rows(max_q_len, group) - 1) /
                          tree_unit_rows(max_q_len, group));
    const double shares = units * ((max_context_len + kBN - 1) / kBN + kUnitCost) / kMinShare;
    return shares < 1 ? 1 : shares > 1e9 ? 1000000000LL : static_cast<long long>(shares);
}

namespace {

template <int D, int MODE>
cudaError_t launch_rows(const TreeArgs &a, cudaStream_t stream) {
    return a.unit_rows == kRows ? launch_mode<D, MODE, 1>(a, stream) : launch_mode<D, MODE, 2>(a, stream);
}

template <int D>
cudaError_t launch_dim(const TreeArgs &a, cudaStream_t stream) {
    return a.mode == 0 ? launch_rows<D, 0>(a, stream)
                       : a.mode == 1 ? launch_rows<D, 1>(a, stream) : launch_rows<D, 2>(a, stream);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs &a, cudaStream_t stream) {
    return a.head_dim == 128 ? launch_dim<128>(a, stream) : launch_dim<64>(a, stream);
}

}  // namespace pkv
