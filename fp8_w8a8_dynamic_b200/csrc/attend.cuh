// attend.cuh — attention of a batch over a shared prefix and each sequence's
// own tokens, both in the paged FP8 cache of rope.cuh.
//
//   row (token t of sequence b, query head h), KV head h / G:
//     z_j = scale * (q . dec(K_j)) * sk_j   over the tokens the row sees: the
//           P prefix tokens, and own tokens p < kv_len[b] - n_b + (t - t_b) + 1
//           (its n_b new tokens are the last of its kv_len[b] cached ones)
//     out = sum_j e^(z_j - lse) sv_j dec(V_j),   lse = ln sum_j e^(z_j)
//   a row that sees nothing gets zeros and lse = -inf.
//
// The prefix is read once for the whole batch: the query rows of all
// sequences that share a KV head (T * G of them) form the rows of one
// matrix.  Both parts are cut along the tokens into chunks; each chunk's
// normalised output and log-sum-exp go to the workspace in fp32, and
// join_kernel weighs them together.
//
// attend_rows_kernel: row tiles of 8 or 16 on mma.sync (f16 operands, fp32 sums).
// It serves the calls that are bound by reading the cache (a decode step's
// own tokens: G rows per KV head), where a 128-row tcgen05 tile would be
// almost empty.  e4m3 codes are exact in f16.  Q goes to f16 with a power of two per
// row that puts its largest element in [2^7, 2^8): exact for elements down
// to 2^-24 of that largest, off by at most 2^-32 of it below.  A row with an
// infinity or NaN is NaN in every place: its logits are (some of its products
// are infinite or NaN, so whatever it sees, its softmax has no value).  The
// probabilities times the value scales go to f16 relative to the largest
// value scale seen (a power of two M per warp): p sv / M 2^14, 11 bits down
// to 2^-28 of M.  Sums, maxima and outputs stay in fp32.
//
// A value row with an infinity or NaN (mfp8_kv_page_store gives it a scale of
// NaN) would reach every query row of a matrix instruction, since 0 NaN = NaN:
// a later token's would spoil the queries before it.  So such rows are taken
// as zeros, and the first of them is remembered: the rows that see it (a row
// sees all tokens up to its last) get NaN at the end.  Their log-sum-exp,
// which the values have no part in, stays what it is.
//
// Each warp streams its own share of the chunk, 32 tokens at a time, through
// a ring of three cp.async stages of its own, so warps never wait for one
// another until they merge at the end.  Tokens (for z) and dimensions (for
// the output) are the 16 rows of a matrix instruction, query rows its 8
// columns, so a decode step's few rows (G <= 8) waste none of them: half the
// products, exponentials and accumulators that 16 rows need.  The dot
// products' summation order is free, so each lane's operand fragments are
// whole 16-byte pieces of code rows: the four lanes of a quad take 16 (of each
// 64) dimensions of a key row, and the eight lanes of a column group take 16
// dimensions each of four value rows, whose bytes are paired by token with
// byte permutes.  The probabilities change sides by 8 x 8 transposes.
//
// 256 sequences with 128 to 4096 own tokens (8 KV heads of 128, 1.1 GB) behind
// 8192 shared ones: 222 us in all, 5.1 TB/s, 0.78 of the copy rate.  Such own
// tokens alone, 187 us for 1.16 GB, 0.94 of it: the difference is the tall
// kernel, whose 32 CTAs hold their SMs for about 165 us, and the join's 10.
// Two blocks of four warps per SM; before (query rows as matrix rows, 16 to a
// tile) 265 us.  When that step took 220, three blocks with two stages took
// 232, with four stages of 16 tokens 240, four blocks with three stages of 16
// tokens 228; for 64 sequences of up to 1024 these took 75 us instead of 78.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace mfp8 {
namespace attend {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;    // query rows of the larger tile
constexpr int kIter = 32;    // tokens per warp and iteration
constexpr int kStages = 3;
constexpr int kMinChunk = kWarps * kIter * 2;  // tokens: below two iterations per warp a split costs more than it saves
constexpr int64_t kMaxTokens = int64_t(1) << 30;  // of one sequence
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kNotFinite = 0x7f800000u;  // a scale's bits from here on: infinity, NaN

struct Params {
    const __nv_bfloat16* Q;
    int64_t ldq;  // elements between tokens
    const int32_t* q_start;
    int B, T, Hq, Hkv, G;
    const uint8_t* K;
    const float* k_scale;
    const uint8_t* V;
    const float* v_scale;
    int64_t n_pages;
    int ps_shift;
    const int32_t* prefix_pages;
    int prefix_len;
    const int32_t* table;
    int64_t ld_table;
    int max_pages;
    const int32_t* kv_len;
    float scale_log2;  // softmax scale times log2(e)
    __nv_bfloat16* O;  // [T][Hq][D]
    float* lse;        // [T][Hq] or null
    float* part;       // [slots][T * Hq][D], normalised partial outputs
    float* part_lse;   // [slots][T * Hq], log2
    int splits_p, splits_o;  // slots of the prefix, then of the own tokens
    int tiles_p, tiles_o;    // row tiles
    int max_q;
    bool direct;  // one slot in all: write O and lse
    bool beside;  // attend_rows_kernel behind attend_wide_kernel of the same call, whose last block only waits
};

// What a block of query rows attends to.
struct Task {
    int tok0;    // first token of the sequence (or batch)
    int n;       // its tokens
    int cut;     // tokens behind those, past max_q, that the grid has no tiles for
    int len;     // cached tokens
    int offset;  // row r sees tokens below offset + r / G (own) or len (prefix)
    bool prefix;
    const int32_t* pages;
    int slot0, splits;
};

__device__ __forceinline__ Task prefix_task(const Params& p) {
    Task k;
    const int q0 = min(max(p.q_start[0], 0), p.T);
    k.tok0 = q0;
    k.n = min(max(p.q_start[p.B], q0), p.T) - q0;
    k.cut = 0;
    k.len = p.prefix_len;
    k.offset = p.prefix_len;
    k.prefix = true;
    k.pages = p.prefix_pages;
    k.slot0 = 0;
    k.splits = p.splits_p;
    return k;
}

// A sequence's place among the query tokens and its cached tokens, cut to
// what the call said and reported when they do not fit it.
struct Lengths {
    int q0, q1;  // its query tokens
    int n;       // of them, those the grid has tiles for
    int len;     // cached tokens
};
__device__ __forceinline__ Lengths lengths_of(const int32_t* q_start, const int32_t* kv_len, int b, int T, int max_q,
                                              int most) {
    Lengths x;
    const int a = q_start[b], e = q_start[b + 1], l = kv_len[b];
    x.q0 = min(max(a, 0), T);
    x.q1 = min(max(e, x.q0), T);
    x.n = min(x.q1 - x.q0, max_q);
    x.len = min(max(l, 0), most);
    if (a != x.q0 || e != x.q1 || x.n != x.q1 - x.q0 || l != x.len) record_device_status(MFP8_ERR_INDEX);
    return x;
}

__device__ __forceinline__ Task own_task(const Params& p, int b) {
    const Lengths x = lengths_of(p.q_start, p.kv_len, b, p.T, p.max_q, int(min(int64_t(p.max_pages) << p.ps_shift, kMaxTokens)));
    Task k;
    k.tok0 = x.q0;
    k.n = x.n;
    k.cut = x.q1 - x.q0 - x.n;
    k.len = x.len;
    k.offset = k.len - (x.q1 - x.q0) + 1;
    k.prefix = false;
    k.pages = p.table + int64_t(b) * p.ld_table;
    k.slot0 = p.splits_p;
    k.splits = p.splits_o;
    return k;
}

// A call without own tokens has no block that reads a sequence's lengths:
// they are checked all the same, by the first `threads` threads of each block.
// Not inlined: that spills in the tall kernel (prompts 680 -> 702 us).
__device__ __noinline__ void check_lengths(const int32_t* q_start, const int32_t* kv_len, int B, int T, int max_q,
                                           int threads) {
    if (int(threadIdx.x) >= threads) return;
    for (int64_t b = int64_t(blockIdx.x) * threads + threadIdx.x; b < B; b += int64_t(gridDim.x) * threads)
        lengths_of(q_start, kv_len, int(b), T, max_q, 0);
}

__device__ __forceinline__ int visible(const Task& k, int token) {
    return k.prefix ? k.len : min(k.len, k.offset + token);
}

// Row r of the task in Q's order of rows, KV head h.
__device__ __forceinline__ int64_t row_of(const Params& p, const Task& k, int h, int r) {
    return int64_t(k.tok0 + r / p.G) * p.Hq + h * p.G + r % p.G;
}

// Rows r0 .. r1 - 1 of KV head h see nothing of this slot's tokens.  Whole block.
template <int D>
__device__ __forceinline__ void nothing_seen(const Params& p, const Task& k, int h, int slot, int r0, int r1) {
    for (int r = r0 + int(threadIdx.x); r < r1; r += int(blockDim.x)) {
        const int64_t row = row_of(p, k, h, r);
        if (!p.direct) p.part_lse[int64_t(slot) * p.T * p.Hq + row] = -INFINITY;
        else if (p.lse) p.lse[row] = -INFINITY;
    }
    if (p.direct)
        for (int64_t i = threadIdx.x; i < int64_t(r1 - r0) * (D / 8); i += blockDim.x)
            reinterpret_cast<uint4*>(p.O)[row_of(p, k, h, r0 + int(i / (D / 8))) * (D / 8) + i % (D / 8)] =
                make_uint4(0u, 0u, 0u, 0u);
}

// Page index of token `tok` of the task, checked against the pool.  An
// ordinary load: the kernel before this one may have written the table, and no
// fence orders the read-only path.
__device__ __forceinline__ int page_of(const Params& p, const Task& k, int tok, int last) {
    const int pg = k.pages[min(tok, last) >> p.ps_shift];
    if (uint32_t(pg) >= uint64_t(p.n_pages)) {
        record_device_status(MFP8_ERR_INDEX);
        return 0;
    }
    return pg;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2_of_codes(uint16_t codes2) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(codes2));
    return h2;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// An 8 x 8 matrix of 16-bit values, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(v));
    return y;
}

// The exponent that scales row values into [2^7, 2^8) from the largest
// magnitude's bf16 bits (tiny rows are taken as 2^-119).
__device__ __forceinline__ int row_exponent(uint32_t amax_bits) { return max(int(amax_bits >> 7), 8) - 127 - 7; }

// 2^-e, which a row is multiplied by; NaN for a row that holds an infinity or NaN.
__device__ __forceinline__ float row_factor(int e, uint32_t amax_bits) {
    return amax_bits < 0x7f80u ? pow2i(-e) : quiet_nan();
}

template <int D, int ROWS>
struct RowsLayout {
    static constexpr int CHUNKS = D / 16;                 // 16-byte pieces of a code row
    static constexpr int STAGE = 2 * kIter * D + 2 * kIter * 4;  // K, V, k_scale, v_scale
    static constexpr int RING = kStages * STAGE;
    static constexpr int OPITCH = D + 4;
    static constexpr int MERGE = kWarps * ROWS * OPITCH * 4 + kWarps * ROWS * 4;
    static constexpr int SMEM = kWarps * RING > MERGE ? kWarps * RING : MERGE;
};

// Piece `ch` of row r sits at piece ch ^ swz(r): a quad's key reads (rows r,
// r + 1) and a column group's value reads (rows 2c + u, pieces g, g + 1)
// each touch every bank once per eight lanes (D = 128).
template <int D>
__device__ __forceinline__ uint32_t swz(uint32_t r) {
    return ((r & 6u) ^ ((r & 1u) << 2)) & uint32_t(D / 16 - 1);
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
attend_rows_kernel(const Params p) {
    using L = RowsLayout<D, ROWS>;
    constexpr int NB = ROWS / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    grid_launch_dependents();
    // Beside the tall kernel there is nothing to wait for: its blocks let this
    // grid start once they have waited themselves, so all that came before has
    // ended and its writes are performed, and the two write different slots.
    // What this SM's L1 held before that is kept out of sight by the fence,
    // since nothing here is read as constant (page_of).  One block more than
    // there is work waits for the tall kernel, so that this grid ends after it
    // and join_kernel, which waits for this grid, sees both.
    const bool waits = p.beside && blockIdx.x == gridDim.x - 1;
    if (!p.beside || waits) grid_dependency_wait();
    if (waits) return;
    if (p.beside) __threadfence();
    if (p.splits_o == 0) check_lengths(p.q_start, p.kv_len, p.B, p.T, p.max_q, kThreads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;

    // ---- which rows, which tokens
    uint32_t u = blockIdx.x;  // the host keeps grids below 2^31
    const uint32_t np = uint32_t(p.tiles_p * p.splits_p * p.Hkv), heads = uint32_t(p.Hkv);
    int split, h, tile;
    Task k;
    if (u < np) {
        h = int(u % heads);
        u /= heads;
        split = int(u % uint32_t(p.splits_p));
        tile = int(u / uint32_t(p.splits_p));
        k = prefix_task(p);
    } else {
        u -= np;
        h = int(u % heads);
        u /= heads;
        split = int(u % uint32_t(p.splits_o));
        u /= uint32_t(p.splits_o);
        tile = int(u % uint32_t(p.tiles_o));
        k = own_task(p, int(u / uint32_t(p.tiles_o)));
    }
    const int nrows = k.n * p.G;
    const int r0 = tile * ROWS;
    const int slot = k.slot0 + split;
    // Every slot of a row has to hold something when join_kernel reads it: query tokens past max_q see the prefix alone.
    if (tile == 0 && k.cut > 0) nothing_seen<D>(p, k, h, slot, nrows, nrows + k.cut * p.G);
    if (r0 >= nrows) return;
    const int rlast = min(r0 + ROWS, nrows) - 1;
    const int seen = max(visible(k, rlast / p.G), 0);  // of the tile's last row, which sees most
    // Chunks of whole iterations of all warps; every chunk but the last is full.
    int chunk = (k.len + k.splits - 1) / k.splits;
    chunk = max((chunk + kWarps * kIter - 1) / (kWarps * kIter) * (kWarps * kIter), kMinChunk);
    const int64_t first = int64_t(split) * chunk;
    if (first >= seen) return nothing_seen<D>(p, k, h, slot, r0, rlast + 1);
    const int k0 = int(first), k1 = min(k0 + chunk, seen);
    const int iters = (k1 - k0 + kIter - 1) / kIter;

    // ---- the ring
    const uint32_t ring = smem_u32(smem) + warp * L::RING;
    auto load = [&](int it, int page) {  // `page`: of token 8 * (lane & 3) of the iteration
        const uint32_t st = ring + uint32_t((it / kWarps) % kStages) * L::STAGE;
        const int base = k0 + it * kIter;
        constexpr int RPI = 32 / L::CHUNKS;  // rows per instruction
        const int ch = lane % L::CHUNKS;
        const int psm = (1 << p.ps_shift) - 1;
#pragma unroll
        for (int i = 0; i < kIter / RPI; ++i) {
            const int r = i * RPI + lane / L::CHUNKS;
            const int pg = __shfl_sync(0xffffffffu, page, (i * RPI) >> 3);
            const int64_t at = (((int64_t(pg) * p.Hkv + h) << p.ps_shift) + ((base + r) & psm)) * D + ch * 16;
            const uint32_t n = base + r < k1 ? 16u : 0u;  // rows past the end are filled with zeros
            const uint32_t dst = st + r * D + ((ch ^ swz<D>(r)) << 4);
            cp_async16(dst, p.K + at, n);
            cp_async16(dst + kIter * D, p.V + at, n);
        }
        const int pg = __shfl_sync(0xffffffffu, page, lane >> 3);
        const int64_t at = ((int64_t(pg) * p.Hkv + h) << p.ps_shift) + ((base + lane) & psm);
        const uint32_t n = base + lane < k1 ? 4u : 0u;
        cp_async4(st + 2 * kIter * D + lane * 4, p.k_scale + at, n);
        cp_async4(st + 2 * kIter * D + kIter * 4 + lane * 4, p.v_scale + at, n);
    };
    auto page_at = [&](int it) { return it < iters ? page_of(p, k, k0 + it * kIter + 8 * c, k1 - 1) : 0; };

    int next, page;  // next iteration to load, its page
    auto fill = [&] {
        next = warp;
        page = page_at(next);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            const int page2 = page_at(next + kWarps);
            if (next < iters) load(next, page);
            cp_async_commit();
            next += kWarps;
            page = page2;
        }
    };
    fill();

    // ---- Q fragments: word w of a lane's codes is dimensions
    // (w / 4) * 64 + c * 16 + (w % 4) * 4 .. + 3 of the row
    constexpr int W = D / 16;
    uint32_t qf[NB][W][2];
    float f[NB][2];   // of columns 2c, 2c + 1 of z
    int lim[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int r = r0 + g + 8 * nb;
        const bool live = r < nrows;
        const int t = live ? r / p.G : 0;
        const uint4* q = reinterpret_cast<const uint4*>(p.Q + int64_t(k.tok0 + t) * p.ldq +
                                                        int64_t(h * p.G + (live ? r % p.G : 0)) * D + c * 16);
        uint32_t w[W][2];
        uint32_t acc = 0;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 a = live ? q[i * 8] : make_uint4(0u, 0u, 0u, 0u);
            const uint4 b = live ? q[i * 8 + 1] : make_uint4(0u, 0u, 0u, 0u);
            acc = absmax_bits_u4(b, absmax_bits_u4(a, acc));
            w[4 * i][0] = a.x, w[4 * i][1] = a.y, w[4 * i + 1][0] = a.z, w[4 * i + 1][1] = a.w;
            w[4 * i + 2][0] = b.x, w[4 * i + 2][1] = b.y, w[4 * i + 3][0] = b.z, w[4 * i + 3][1] = b.w;
        }
        uint32_t amax = max(acc & 0xffffu, acc >> 16);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = row_exponent(amax);
        const float m = row_factor(e, amax);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            qf[nb][i][0] = pack_f16x2(bf16_lo(w[i][0]) * m, bf16_hi(w[i][0]) * m);
            qf[nb][i][1] = pack_f16x2(bf16_lo(w[i][1]) * m, bf16_hi(w[i][1]) * m);
        }
        const float fr = p.scale_log2 * pow2i(e);
        const int lr = live ? min(visible(k, t), k1) : 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f[nb][j] = __shfl_sync(0xffffffffu, fr, (2 * c + j) * 4);
            lim[nb][j] = __shfl_sync(0xffffffffu, lr, (2 * c + j) * 4);
        }
    }
    const int all_see = k.prefix ? k1 : min(visible(k, r0 / p.G), k1);  // tokens below are seen by every row

    // ---- the pass over the tokens
    constexpr int MT = kIter / 16;  // 16-token tiles of an iteration
    constexpr int NT = D / 8;       // dimensions of a lane group: g * NT ..
    float o[NB][NT / 2][4];
    float m[NB][2], l[NB][2];
    int bad_at = INT32_MAX;  // first token of this warp's whose value row is not finite, as far as looked for
    int vexp;  // biased exponent just above the largest value scale seen, at least 2^-100
    auto pass = [&](auto look) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.0f;
            m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.0f;
        }
        vexp = 27;
        for (int it = warp; it < iters; it += kWarps) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            const uint32_t st = ring + uint32_t((it / kWarps) % kStages) * L::STAGE;
            const uint32_t scales = st + 2 * kIter * D;
            const int base = k0 + it * kIter;
            // z: rows are tokens, columns query rows
            float z[MT][NB][4];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) z[t][nb][0] = z[t][nb][1] = z[t][nb][2] = z[t][nb][3] = 0.0f;
                const int ra = t * 16 + g, rb = ra + 8;
#pragma unroll
                for (int i = 0; i < W / 4; ++i) {
                    const uint4 ca = lds128(st + ra * D + (((c + 4 * i) ^ swz<D>(ra)) << 4));
                    const uint4 cb = lds128(st + rb * D + (((c + 4 * i) ^ swz<D>(rb)) << 4));
                    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a[4] = {
                            f16x2_of_codes(uint16_t(wa[e] & 0xffffu)), f16x2_of_codes(uint16_t(wb[e] & 0xffffu)),
                            f16x2_of_codes(uint16_t(wa[e] >> 16)), f16x2_of_codes(uint16_t(wb[e] >> 16))};
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_f16(z[t][nb], a, qf[nb][4 * i + e][0], qf[nb][4 * i + e][1]);
                    }
                }
            }
            float sv[MT][2];
            float mx[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mx[nb][0] = mx[nb][1] = -INFINITY;
            const bool masked = base + kIter > all_see;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint32_t at = scales + (t * 16 + g) * 4;
                const float ka = ld_shared_f32(at), kb = ld_shared_f32(at + 32);
                sv[t][0] = ld_shared_f32(at + kIter * 4), sv[t][1] = ld_shared_f32(at + kIter * 4 + 32);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float(&v)[4] = z[t][nb];
                    v[0] *= ka * f[nb][0];
                    v[1] *= ka * f[nb][1];
                    v[2] *= kb * f[nb][0];
                    v[3] *= kb * f[nb][1];
                    if (masked) {
                        const int tok = base + t * 16 + g;
                        if (tok >= lim[nb][0]) v[0] = -INFINITY;
                        if (tok >= lim[nb][1]) v[1] = -INFINITY;
                        if (tok + 8 >= lim[nb][0]) v[2] = -INFINITY;
                        if (tok + 8 >= lim[nb][1]) v[3] = -INFINITY;
                    }
                    mx[nb][0] = fmaxf(mx[nb][0], fmaxf(v[0], v[2]));
                    mx[nb][1] = fmaxf(mx[nb][1], fmaxf(v[1], v[3]));
                }
            }
            // largest value scale of the iteration's tokens, as a power of two above it
            const uint32_t svl = __float_as_uint(ld_shared_f32(scales + kIter * 4 + lane * 4));
            uint32_t svb = __reduce_max_sync(0xffffffffu, svl);
            if (decltype(look)::value && svb >= kNotFinite) {  // value rows that are not finite are taken out: zeros, with a scale of zero
                const bool bad = svl >= kNotFinite;
                if (bad) {
#pragma unroll 1
                    for (int i = 0; i < L::CHUNKS; ++i) st_shared_v4(st + kIter * D + lane * D + i * 16, 0u, 0u, 0u, 0u);
                    st_shared_u32(scales + kIter * 4 + lane * 4, 0u);
                }
                bad_at = min(bad_at, base + __ffs(int(__ballot_sync(0xffffffffu, bad))) - 1);
                svb = __reduce_max_sync(0xffffffffu, bad ? 0u : svl);
                __syncwarp();
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint32_t at = scales + kIter * 4 + (t * 16 + g) * 4;
                    sv[t][0] = ld_shared_f32(at), sv[t][1] = ld_shared_f32(at + 32);
                }
            }
            const int ve = max(vexp, min(int(svb >> 23) + 1, 254));
            const float vadj = pow2i(max(vexp - ve, -126));
            const float vnorm = pow2i(14 - (ve - 127));
            vexp = ve;
            float keep[NB][2], mm[NB][2];
            bool moved = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = mx[nb][j];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float mn = fmaxf(m[nb][j], x);
                    mm[nb][j] = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet: every term is e^-inf = 0
                    keep[nb][j] = ex2(m[nb][j] - mm[nb][j]);
                    m[nb][j] = mn;
                    l[nb][j] *= keep[nb][j];
                    keep[nb][j] *= vadj;
                    moved = moved || keep[nb][j] != 1.0f;
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < NT / 2; ++i) {
                        o[nb][i][0] *= keep[nb][0];
                        o[nb][i][1] *= keep[nb][1];
                        o[nb][i][2] *= keep[nb][0];
                        o[nb][i][3] *= keep[nb][1];
                    }
            }
            uint32_t pf[MT][NB][2];  // tokens by query rows, transposed into the layout of a second operand
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const float s0 = sv[t][0] * vnorm, s1 = sv[t][1] * vnorm;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float a0 = ex2(z[t][nb][0] - mm[nb][0]), a1 = ex2(z[t][nb][1] - mm[nb][1]);
                    const float b0 = ex2(z[t][nb][2] - mm[nb][0]), b1 = ex2(z[t][nb][3] - mm[nb][1]);
                    l[nb][0] += a0 + b0;
                    l[nb][1] += a1 + b1;
                    pf[t][nb][0] = transpose8x8(pack_f16x2(a0 * s0, a1 * s0));
                    pf[t][nb][1] = transpose8x8(pack_f16x2(b0 * s1, b1 * s1));
                }
            }
            // output: rows g and g + 8 of tile i are dimensions g * NT + 2i and + 1, columns query rows
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                uint32_t a[4][NT / 4];  // value rows 2c, 2c + 1, 2c + 8, 2c + 9 of the token tile
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int r = (2 * t + (q >> 1)) * 8 + 2 * c + (q & 1);
                    const uint32_t row = st + kIter * D + r * D;
                    if constexpr (D == 128) {
                        const uint4 v = lds128(row + ((g ^ swz<D>(r)) << 4));
                        a[q][0] = v.x, a[q][1] = v.y, a[q][2] = v.z, a[q][3] = v.w;
                    } else {
                        const uint2 v = lds64(row + (((g >> 1) ^ swz<D>(r)) << 4) + (g & 1) * 8);
                        a[q][0] = v.x, a[q][1] = v.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < NT / 4; ++q) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {  // dimensions 4q, 4q + 1, then 4q + 2, 4q + 3
                        const uint32_t sel = half ? 0x7362u : 0x5140u;
                        const uint32_t x = __byte_perm(a[0][q], a[1][q], sel), y = __byte_perm(a[2][q], a[3][q], sel);
                        const uint32_t av[4] = {f16x2_of_codes(uint16_t(x & 0xffffu)), f16x2_of_codes(uint16_t(x >> 16)),
                                                f16x2_of_codes(uint16_t(y & 0xffffu)), f16x2_of_codes(uint16_t(y >> 16))};
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][2 * q + half], av, pf[t][nb][0], pf[t][nb][1]);
                    }
                }
            }
            __syncwarp();
            const int page2 = page_at(next + kWarps);
            if (next < iters) load(next, page);
            cp_async_commit();
            next += kWarps;
            page = page2;
        }
    };
    pass(std::false_type());
    // An infinity or NaN among the value scales shows as the largest exponent that there is: the warp's tokens once
    // more, its value rows looked at (in the first pass that costs 4 us of 222 in a decode step of 256).
    if (vexp == 254) {
        cp_async_wait<0>();
        __syncwarp();
        fill();
        pass(std::true_type());
    }

    // ---- merge the warps
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring
    float* om = reinterpret_cast<float*>(smem);
    float* lm = om + kWarps * ROWS * L::OPITCH;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float sum = l[nb][j];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            float inv = sum != 0.0f ? ldexpf(1.0f / sum, vexp - 127 - 14) : 0.0f;
            if (lim[nb][j] > bad_at) inv = quiet_nan();
            const int i0 = warp * ROWS + nb * 8 + 2 * c + j;
            float4* dst = reinterpret_cast<float4*>(om + i0 * L::OPITCH + g * NT);
#pragma unroll
            for (int i = 0; i < NT / 2; i += 2)
                dst[i / 2] = make_float4(o[nb][i][j] * inv, o[nb][i][2 + j] * inv, o[nb][i + 1][j] * inv,
                                         o[nb][i + 1][2 + j] * inv);
            if (g == 0) lm[i0] = sum != 0.0f ? m[nb][j] + log2f(sum) : -INFINITY;
        }
    __syncthreads();
    constexpr int CPT = ROWS * D / kThreads;  // values per thread, all of one row
    const int i = threadIdx.x / (D / CPT), d0 = (threadIdx.x % (D / CPT)) * CPT;
    const int r = r0 + i;
    if (r >= nrows) return;
    float mx = lm[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, lm[w * ROWS + i]);
    const float mz = mx == -INFINITY ? 0.0f : mx;
    float wt[kWarps], sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += wt[w] = ex2(lm[w * ROWS + i] - mz);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    const float out_lse = sum != 0.0f ? mx + log2f(sum) : -INFINITY;
    const int64_t row = row_of(p, k, h, r);
    float y[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) y[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int j = 0; j < CPT; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(om + (w * ROWS + i) * L::OPITCH + d0 + j);
            y[j] = fmaf(wt[w], v.x, y[j]);
            y[j + 1] = fmaf(wt[w], v.y, y[j + 1]);
            y[j + 2] = fmaf(wt[w], v.z, y[j + 2]);
            y[j + 3] = fmaf(wt[w], v.w, y[j + 3]);
        }
    if (p.direct) {
        uint2* dst = reinterpret_cast<uint2*>(p.O + row * D + d0);
#pragma unroll
        for (int j = 0; j < CPT; j += 4) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(y[j] * inv, y[j + 1] * inv);
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[j + 2] * inv, y[j + 3] * inv);
            dst[j / 4] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
        if (d0 == 0 && p.lse) p.lse[row] = out_lse * kLn2;
    } else {
        const int64_t at = int64_t(slot) * p.T * p.Hq + row;
        float4* dst = reinterpret_cast<float4*>(p.part + at * D + d0);
#pragma unroll
        for (int j = 0; j < CPT / 4; ++j)
            dst[j] = make_float4(y[4 * j] * inv, y[4 * j + 1] * inv, y[4 * j + 2] * inv, y[4 * j + 3] * inv);
        if (d0 == 0) p.part_lse[at] = out_lse;
    }
}

// Joins the slots of each row: out = sum_s 2^(lse_s - lse) out_s.  One warp
// per row; slots whose lse is -inf hold no output and are not read.  Rows
// outside [q_start[0], q_start[B]) are left as they were.
template <int D>
__global__ void __launch_bounds__(256)
join_kernel(const Params p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t rows = int64_t(p.T) * p.Hq;
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int t = int(uint32_t(row) / uint32_t(p.Hq));  // T * Hq < 2^31
    if (t < p.q_start[0] || t >= p.q_start[p.B]) return;
    const int slots = p.splits_p + p.splits_o;
    constexpr int VPL = D / 32;     // values per lane
    constexpr int kAhead = 8;       // slots whose loads are in flight together
    const float* part = p.part + row * D + lane * VPL;
    const int64_t pitch = rows * D;
    auto load = [&](int s, float (&v)[VPL]) {
        if constexpr (VPL == 4) {
            const float4 x = *reinterpret_cast<const float4*>(part + s * pitch);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(part + s * pitch);
            v[0] = x.x, v[1] = x.y;
        }
    };
    // The first slots' outputs are asked for together with the log-sum-exps;
    // what a slot without weight holds is not used.
    float v[kAhead][VPL];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) v[i][j] = 0.0f;
        if (i < slots) load(i, v[i]);
    }
    float lse0 = lane < slots ? p.part_lse[int64_t(lane) * rows + row] : -INFINITY;
    float mx = lse0;
    for (int s = lane + 32; s < slots; s += 32) mx = fmaxf(mx, p.part_lse[int64_t(s) * rows + row]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float mz = mx == -INFINITY ? 0.0f : mx;
    float y[VPL], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) y[j] = 0.0f;
    for (int s0 = 0; s0 < slots; s0 += 32) {
        if (s0 > 0) lse0 = s0 + lane < slots ? p.part_lse[int64_t(s0 + lane) * rows + row] : -INFINITY;
        // -1: a slot that holds no output.  (A weight may be 0 for another reason, and its output NaN.)
        const float w = lse0 == -INFINITY ? -1.0f : ex2(lse0 - mz);
        const int n = min(32, slots - s0);
        for (int i0 = 0; i0 < n; i0 += kAhead) {
            float wi[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                wi[i] = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
                if (i0 + i >= n) wi[i] = -1.0f;
                if (s0 + i0 > 0 && !(wi[i] < 0.0f)) load(s0 + i0 + i, v[i]);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (wi[i] < 0.0f) continue;
                sum += wi[i];
#pragma unroll
                for (int j = 0; j < VPL; ++j) y[j] = fmaf(wi[i], v[i][j], y[j]);
            }
        }
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + row * D + lane * VPL);
#pragma unroll
    for (int j = 0; j < VPL; j += 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[j] * inv, y[j + 1] * inv);
        dst[j / 2] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (lane == 0 && p.lse) p.lse[row] = sum != 0.0f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

}  // namespace attend
}  // namespace mfp8
