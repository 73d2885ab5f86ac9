// attend_wide.cuh — the tall case of attend.cuh on the tcgen05 tensor cores:
// many query rows per KV head (a prefix shared by a batch, long prompts), so
// the work is bound by the products and exponentials instead of by reading
// the cache.
//
// One CTA takes up to 256 query rows of one KV head over one chunk of
// tokens, 128 tokens to a tile, in two sides of 128 rows whose softmax
// alternates with the other side's products.  With more than 128 rows the
// sides hold different rows and share every tile; with fewer they hold the
// same rows, take alternate tiles and are joined at the end.
//
//   z = Q K^T   kind::f8f6f4, M = N = 128.  The key codes go to the tensor
//               cores as they are.  Q is the sum of two e4m3 terms: bf16 has
//               8 significant bits, e4m3 has 4, so with q scaled by a power
//               of two per row, hi = e4m3(q) and lo = e4m3(q - hi) hold q
//               exactly down to 2^-9.8 of the row's largest element (which
//               lies in [224, 448]) and are off by at most 2^-17.8 of it
//               below.  Two e4m3 products cost what one f16 product costs,
//               and no key is ever converted.  A row with an infinity or
//               NaN is NaN in every place (e4m3 has no infinity: converted,
//               one would become a finite 896).
//   p           z sk_j (fp32) to e^(z - m), m lagging behind the running
//               maximum by up to kLag octaves, so O is rescaled only when
//               the maximum has grown by more; p 2^kNorm goes to f16.
//   O += P V    kind::f16, P from TMEM (it replaces z there), V converted
//               from e4m3 to f16 by a warpgroup of its own and multiplied by
//               sv_j / M (M: a power of two above every value scale read so
//               far, O is rescaled when it grows), so the softmax needs no
//               value scales; token rows of 64 dimensions, read by the MMA
//               with N contiguous.  Roundings to f16 (11 bits): p, sv_j / M
//               and their products with the codes.
//
// Warps: 0-3 and 4-7 softmax of side 0 and 1 (one row per thread), 8-11 the
// conversion of V, 12 the TMA loads, one lane per page of the tile, 13 the
// MMA issue; 14 and 15 only pad the last warpgroup.
//
// TMEM: columns 0-127 and 128-255 z (then P) of side 0 and 1, 256 and 384 O.
// The MMAs of a thread run in order, so Q K^T of a side's next tile may
// overwrite its P as soon as P V has been issued.
//
// What bounds it (B200, 1.97 GHz; a step is 128 rows x 128 tokens): the MMAs
// of a step take 1024 cycles, its exponentials 1024 on the special-function
// units, and a step takes 2300 (1.17 us): a side's tile goes through 1900 to
// 2200 cycles of softmax, 1024 of MMAs and two hand-overs (a commit, the
// waiting warp's wake-up and its arrive back take 490 to 560 cycles), and only
// two sides fit in TMEM to overlap them; P is handed over whole, so P V of a
// tile starts behind its last exponential.  Besides the steps a CTA takes about
// 10 us (Q, the ends of the pipeline, its output), and a grid that ends in part
// of a wave leaves SMs idle: 3000 query tokens of 32 heads over 10007 shared
// ones are 376 CTAs, 2.54 waves on 148 SMs, 640 us, 0.49 of the burst peak;
// their steps spread evenly would take 500.  Measured and not kept there: 16
// softmax warps 850 us; 64-token steps with two buffers of z per side 1040;
// four rows per thread in the 16 x 256-bit TMEM layout, a quarter of the
// scales' shared-memory reads, 790; an issuing lane per side in turns 670;
// waits that poll without sleeping 1.48 us a step.
//
// Every wait is bounded (wait_asleep), as in the GEMM kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.cuh"
#include "ptx.cuh"

namespace mfp8 {
namespace attend {

constexpr int kWideThreads = 512;
constexpr int kTile = 128;      // tokens per tile, rows per side
constexpr int kWideRows = 256;  // rows per CTA
constexpr float kLag = 8.0f;  // octaves; with 4, a third of the tiles of a long prefix rescaled O in some warp, 420 cycles each
constexpr int kNorm = 7;      // P holds p 2^kNorm, below 2^15 in f16
constexpr int kVNorm = 7;     // V holds dec(V) sv / M 2^kVNorm, below 448 * 2^7
constexpr int kMinVexp = 27;  // M >= 2^-100
// Registers: 512 threads are launched with 128 each; the softmax warps, which
// hold a row of 128 logits, take 192 and leave 64 to the others.
constexpr int kSoftmaxRegs = 192, kOtherRegs = 64;

template <int D>
struct WideLayout {
    static constexpr int KST = 3, VST = 2, CST = 2;
    static constexpr int Q_OFF = 0;  // [side][hi, lo][128 rows of D bytes]
    static constexpr int QB = kTile * D;
    static constexpr int K_OFF = Q_OFF + 4 * QB;
    static constexpr int V_OFF = K_OFF + KST * kTile * D;
    static constexpr int C_OFF = V_OFF + VST * kTile * D;       // f16 V: [dim / 64][token][64 dims]
    static constexpr int SST = 4;
    static constexpr int S_OFF = C_OFF + CST * kTile * D * 2;  // key scales, value scales
    static constexpr int BAR_OFF = S_OFF + SST * 1024;
    static constexpr int KFULL = 0, KEMPTY = KST, VFULL = 2 * KST, VEMPTY = VFULL + VST, CFULL = VEMPTY + VST,
                         CEMPTY = CFULL + CST, LFULL = CEMPTY + CST, LEMPTY = LFULL + SST, SFULL = LEMPTY + SST,
                         PFULL = SFULL + 2, OFULL = PFULL + 2, QFULL = OFULL + 2, DRAIN = QFULL + 1,
                         NUM_BARS = DRAIN + 1;
    static constexpr int LSE_OFF = BAR_OFF + NUM_BARS * 8;  // [128] log-sum-exps of side 1 at the end
    static constexpr int MISC_OFF = LSE_OFF + 512;
    static constexpr int USED = MISC_OFF + 16;
    static constexpr int SMEM_BYTES = USED + 1024;  // slack for 1024-byte alignment
    static_assert(BAR_OFF % 8 == 0, "barriers are 8-byte aligned");
    static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");
};

// K-major 8-bit operand rows of D bytes, D-byte swizzle (128 or 64).
template <int D>
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t addr) {
    uint64_t d = uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t((8 * D) >> 4) << 32) |
                 (uint64_t(1) << 46);
    return d | (uint64_t(D == 128 ? 2u : 4u) << 61);
}

// f16 [token][64 dims] blocks of 128-byte rows (128-byte swizzle) as an
// operand whose N (the dimensions) is contiguous: 8-token groups 1024 bytes
// apart, 64-dimension blocks kTile * 128 bytes apart.
__device__ __forceinline__ uint64_t nmajor_desc(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t((kTile * 128) >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// f16 x f16 -> fp32, A from TMEM, B with N contiguous, shape 128 x N x 16.
__device__ __forceinline__ constexpr uint32_t idesc_pv(uint32_t N) {
    return (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait with a long suspend hint (1 ms): a waiting thread sleeps in
// hardware until its phase completes.  Polling is what the pipeline does not
// stand: with a bare try_wait loop in the MMA lane alone a step took 1.48 us
// instead of 1.17.  Bounded like mbar_wait.
__device__ __forceinline__ bool wait_asleep(uint32_t bar, uint32_t parity, volatile int* abort) {
    auto attempt = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(1000000u)
            : "memory");
        return ok != 0;
    };
    if (attempt()) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (attempt()) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_device_status(MFP8_ERR_TIMEOUT);
            return false;
        }
    }
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A row's logits times the key scales (in shared memory at `sk`); their maximum.
__device__ __forceinline__ float scale_logits(uint32_t (&z)[128], uint32_t sk) {
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int q = 0; q < 128; q += 4) {
        const float4 s = ld_shared_f4(sk + q * 4);
        float z0, z1, z2, z3;
        unpack2(mul2(pack2(__uint_as_float(z[q]), __uint_as_float(z[q + 1])), pack2(s.x, s.y)), z0, z1);
        unpack2(mul2(pack2(__uint_as_float(z[q + 2]), __uint_as_float(z[q + 3])), pack2(s.z, s.w)), z2, z3);
        z[q] = __float_as_uint(z0), z[q + 1] = __float_as_uint(z1);
        z[q + 2] = __float_as_uint(z2), z[q + 3] = __float_as_uint(z3);
        float& a = mx[(q >> 1) & 3];
        float& b = mx[((q >> 1) + 1) & 3];
        a = fmaxf(a, fmaxf(z0, z1));
        b = fmaxf(b, fmaxf(z2, z3));
    }
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// The same row with tokens at and past `lim` (token `base` is column 0) out
// of it, whatever stands there; the maximum of what is left.
__device__ __forceinline__ float mask_logits(uint32_t (&z)[128], int base, int lim) {
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < 128; ++q) {
        if (base + q >= lim) z[q] = 0xff800000u;
        mx = fmaxf(mx, __uint_as_float(z[q]));
    }
    return mx;
}

// log2 of M, biased: a power of two above `before` and above the value scales
// (in shared memory at `sv`) of the tile's `valid` tokens.  Value rows that are
// not finite do not count; `bad_at` becomes the first of them (the tile starts
// at token `base`) if it is smaller.  Whole warp.
__device__ __forceinline__ int tile_vexp(int before, uint32_t sv, int valid, int lane, int base, int& bad_at) {
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < kTile / 32; ++q)
        if (lane + 32 * q < valid) top = max(top, __float_as_uint(ld_shared_f32(sv + (lane + 32 * q) * 4)));
    top = __reduce_max_sync(0xffffffffu, top);
    if (top >= kNotFinite) {
        uint32_t finite = 0, first = kTile;
#pragma unroll 1
        for (int t = lane; t < valid; t += 32) {
            const uint32_t s = __float_as_uint(ld_shared_f32(sv + t * 4));
            if (s < kNotFinite) finite = max(finite, s);
            else first = min(first, uint32_t(t));
        }
        top = __reduce_max_sync(0xffffffffu, finite);
        bad_at = min(bad_at, base + int(__reduce_min_sync(0xffffffffu, first)));
    }
    return max(before, min(int(top >> 23) + 1, 254));
}

// Which part and unit of the grid a CTA works on.
struct WideGrid {
    int pairs_p, pairs_o;  // 256-row groups of the prefix's rows, of one sequence's rows
};

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1)
attend_wide_kernel(const Params p, const WideGrid wg, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV) {
    using L = WideLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + uint32_t(L::BAR_OFF) + 8u * uint32_t(i); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
    const uint32_t warp = warp_id_sync();
    const int lane = int(lane_id());

    // What needs no input comes before the wait for the previous kernel.
    if (warp == 13) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    if (warp == 12 && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (p.splits_o == 0) check_lengths(p.q_start, p.kv_len, p.B, p.T, p.max_q, 32);

    // ---- which rows, which tokens (uniform over the CTA)
    int64_t u = blockIdx.x;
    const int64_t np = int64_t(wg.pairs_p) * p.splits_p * p.Hkv;
    int split, h, pair;
    Task k;
    h = int(u % p.Hkv);
    if (u < np) {
        u /= p.Hkv;
        split = int(u % p.splits_p);
        pair = int(u / p.splits_p);
        k = prefix_task(p);
    } else {
        u = (u - np) / p.Hkv;
        split = int(u % p.splits_o);
        u /= p.splits_o;
        pair = int(u % wg.pairs_o);
        k = own_task(p, int(u / wg.pairs_o));
    }
    const int nrows = k.n * p.G;
    const int r0 = pair * kWideRows;
    auto leave = [&] {  // before any barrier or MMA was used
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 13) tmem_dealloc(*tmem_holder, 512);
    };
    const int slot = k.slot0 + split;
    if (pair == 0 && k.cut > 0) nothing_seen<D>(p, k, h, slot, nrows, nrows + k.cut * p.G);
    if (r0 >= nrows) return leave();
    const bool both = nrows - r0 > kTile;  // the sides hold different rows
    const int rlast = min(r0 + kWideRows, nrows) - 1;
    const int seen = max(visible(k, rlast / p.G), 0);
    int chunk = (k.len + k.splits - 1) / k.splits;
    chunk = max((chunk + kTile - 1) / kTile * kTile, kTile);
    const int64_t first = int64_t(split) * chunk;
    const int64_t all_rows = int64_t(p.T) * p.Hq;
    if (first >= seen) {
        nothing_seen<D>(p, k, h, slot, r0, rlast + 1);
        return leave();
    }
    const int k0 = int(first), k1 = min(k0 + chunk, seen);
    const int nt = (k1 - k0 + kTile - 1) / kTile;
    const int steps = both ? 2 * nt : nt;  // step j: side j % 2, tile j / 2 (both) or j

    // Each softmax warp's 32 query rows, as they are, to where V's f16 tiles will go: coalesced (a thread's own
    // loads of its row would touch 32 lines an instruction, a bulk copy per row takes 70 cycles each), pieces
    // swizzled by row.  Rows past the last are zeros.
    const int side_row0 = r0 + (both && warp >= 4 ? kTile : 0) + int(warp & 3u) * 32;
    const uint32_t q_stage = sb + L::C_OFF + warp * (32 * 2 * D);
    if (warp < 8) {
        constexpr int PR = D / 8;  // pieces per row
        const int r = side_row0 + lane, t = r < nrows ? r / p.G : 0, g = r < nrows ? r - t * p.G : 0;
        const int64_t mine = int64_t(k.tok0 + t) * p.ldq + int64_t(h * p.G + g) * D;  // this lane's row
        const int piece = lane % PR;
#pragma unroll 4
        for (int i = 0; i < PR; ++i) {
            const int rr = i * (32 / PR) + lane / PR;
            const int64_t at = __shfl_sync(0xffffffffu, mine, rr);
            cp_async16(q_stage + rr * (2 * D) + ((piece ^ (rr & (PR - 1))) << 4), p.Q + at + piece * 8,
                       side_row0 + rr < nrows ? 16u : 0u);
        }
        cp_async_commit();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::NUM_BARS; ++i) {
            uint32_t n = 1;
            if (i >= L::VEMPTY && i < L::VEMPTY + L::VST) n = 4;  // converting warps
            if (i >= L::CFULL && i < L::CFULL + L::CST) n = 4;
            if (i >= L::PFULL && i < L::PFULL + 2) n = 4;  // softmax warps of the side
            if (i == L::QFULL) n = 8;
            if (i >= L::LEMPTY && i < L::LEMPTY + L::SST) n = both ? 12 : 8;  // softmax warps of the tile's sides, converters
            mbar_init(bar(i), n);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp < 8) {
        // ------------------------------------------------------ softmax
        regs_inc<kSoftmaxRegs>();
        const int side = int(warp >> 2);
        const int i = int(threadIdx.x & 127);
        const int r = side_row0 + lane;
        const bool live = r < nrows;
        const int t = live ? r / p.G : 0;
        // Q: two e4m3 terms
        float f;
        {
            cp_async_wait<0>();
            __syncwarp();
            const uint32_t src = q_stage + uint32_t(lane) * (2 * D);
            uint32_t acc = 0;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) acc = absmax_bits_u4(lds128(src + ((c ^ (lane & (D / 8 - 1))) << 4)), acc);
            const uint32_t amax = max(acc & 0xffffu, acc >> 16);
            // 2^e puts the largest element in [224, 448]: its exponent at 8, or at 7 above 1.75 * 2^n
            int e = max(int(amax >> 7), 10) - 127 - 8;
            if ((amax & 0x7fu) > 0x60u) ++e;
            const float m = row_factor(e, amax);
            f = fmaxf(p.scale_log2 * pow2i(e), kFltMin);
            const uint32_t hi = sb + L::Q_OFF + side * 2 * L::QB + i * D, lo = hi + L::QB;
            const uint32_t x = D == 128 ? uint32_t(i & 7) : uint32_t((i >> 1) & 3);
#pragma unroll 2
            for (int c = 0; c < D / 16; ++c) {
                const uint4 a = lds128(src + (((2 * c) ^ (lane & (D / 8 - 1))) << 4));
                const uint4 b = lds128(src + (((2 * c + 1) ^ (lane & (D / 8 - 1))) << 4));
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                uint32_t ch[4] = {0u, 0u, 0u, 0u}, cl[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v0 = bf16_lo(w[j]) * m, v1 = bf16_hi(w[j]) * m;
                    const uint32_t c2 = e4m3x2(v0, v1);
                    const uint32_t h2 = f16x2_of_codes(uint16_t(c2));
                    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                    ch[j >> 1] |= c2 << (16 * (j & 1));
                    cl[j >> 1] |= e4m3x2(v0 - back.x, v1 - back.y) << (16 * (j & 1));
                }
                const uint32_t at = (uint32_t(c) ^ x) << 4;
                st_shared_v4(hi + at, ch[0], ch[1], ch[2], ch[3]);
                st_shared_v4(lo + at, cl[0], cl[1], cl[2], cl[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::QFULL));
        }
        const int lim = live ? min(visible(k, t), k1) : 0;
        const int all_see = k.prefix ? k1 : min(visible(k, (r0 + (both ? side * kTile : 0)) / p.G), k1);
        const uint32_t lane_base = tmem + ((warp & 3u) << 21);
        const uint32_t tS = lane_base + uint32_t(side) * 128u, tO = lane_base + 256u + uint32_t(side) * 128u;
        float m = -INFINITY, l = 0.0f;
        int vexp = kMinVexp, n = 0, bad_at = INT32_MAX;
        const uint64_t f2 = pack2(f, f);
        for (int j = side; j < steps; j += 2, ++n) {
            const int tile = both ? j >> 1 : j;
            const int ls = tile % L::SST;
            const int base = k0 + tile * kTile;
            if (!wait_asleep(bar(L::LFULL + ls), (tile / L::SST) & 1, abort_flag)) break;
            const uint32_t sk = sb + L::S_OFF + ls * 1024;
            const int ve = tile_vexp(vexp, sk + 512, min(kTile, k1 - base), lane, base, bad_at);
            if (!wait_asleep(bar(L::SFULL + side), n & 1, abort_flag)) break;
            tc_fence_after();
            uint32_t z[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(z + c * 32));
            tmem_wait_ld();
            float mx = scale_logits(z, sk);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::LEMPTY + ls));
            if (base + kTile > all_see) mx = mask_logits(z, base, lim);
            mx *= f;
            // m = -inf (nothing seen yet) has -inf + kLag below every finite maximum
            if (__any_sync(0xffffffffu, mx > m + kLag || ve != vexp)) {
                const float mn = fmaxf(m, mx);
                float keep = mn == -INFINITY ? 1.0f : ex2(m - mn);
                m = mn;
                l *= keep;
                keep *= pow2i(max(vexp - ve, -126));
                vexp = ve;
                if (n > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(tO + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * keep);
                        tmem_st_32x32b_x32(tO + c * 32, o);
                    }
                }
            }
            // p 2^kNorm = 2^(z - m + kNorm), summed as it is
            const float off = float(kNorm) - (m == -INFINITY ? 0.0f : m);
            const uint64_t off2 = pack2(off, off);
            uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};  // pairs of +0
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int q = 0; q < 32; q += 4) {
                    float z0, z1, z2, z3;
                    const uint32_t* zz = z + c * 32 + q;
                    unpack2(fma2(pack2(__uint_as_float(zz[0]), __uint_as_float(zz[1])), f2, off2), z0, z1);
                    unpack2(fma2(pack2(__uint_as_float(zz[2]), __uint_as_float(zz[3])), f2, off2), z2, z3);
                    z0 = ex2(z0), z1 = ex2(z1), z2 = ex2(z2), z3 = ex2(z3);
                    sum2[(q >> 1) & 3] = add2(sum2[(q >> 1) & 3], pack2(z0, z1));
                    sum2[((q >> 1) + 1) & 3] = add2(sum2[((q >> 1) + 1) & 3], pack2(z2, z3));
                    w[q / 2] = pack_f16x2(z0, z1);
                    w[q / 2 + 1] = pack_f16x2(z2, z3);
                }
                tmem_st_32x32b_x16(tS + c * 16, w);
            }
            float s0, s1;
            unpack2(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])), s0, s1);
            l += s0 + s1;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::PFULL + side));
        }
        // ---- the output of this side's tiles
        const int64_t my_row = live ? row_of(p, k, h, r) : 0;
        const int mine = both ? nt : (nt + 1 - side) / 2;
        bool ok = mine > 0 && n == mine && wait_asleep(bar(L::OFULL + side), 0, abort_flag);
        if (!both && side == 1 && ok) ok = wait_asleep(bar(L::OFULL), 0, abort_flag);  // every MMA is done
        tc_fence_after();
        // l carries 2^kNorm, O that and 2^kVNorm / M
        const bool any = ok && (m > -INFINITY || l != l);  // a NaN stays one
        float inv = any ? ldexpf(1.0f / l, vexp - 127 - kVNorm) : 0.0f;
        if (lim > bad_at) inv = quiet_nan();
        float my_lse = any ? m + (log2f(l) - float(kNorm)) : -INFINITY;
        float* buf = reinterpret_cast<float*>(smem + L::Q_OFF);  // [D][128]: side 1's output when joined
        float* lbuf = reinterpret_cast<float*>(smem + L::LSE_OFF);
        float w0 = 1.0f, w1 = 0.0f;
        const bool join = !both && nt > 1;  // uniform
        if (join) {
            if (side == 1) {
                lbuf[i] = my_lse;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tO + c * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 32; ++q) buf[(c * 32 + q) * 128 + i] = __uint_as_float(o[q]) * inv;
                }
            }
            named_bar_sync(1, 256);
            const float other = lbuf[i];
            const float mxl = fmaxf(my_lse, other);
            if (my_lse == -INFINITY && other == -INFINITY) {
                w0 = 0.0f;
            } else {
                w0 = ex2(my_lse - mxl);
                w1 = ex2(other - mxl);
                const float tot = w0 + w1;
                w0 /= tot;
                w1 /= tot;
                my_lse = mxl + log2f(tot);
            }
        }
        if (both || side == 0) {  // uniform over the warp, as tcgen05.ld wants
            // O is finite wherever this side had a tile (its P is 0 for what it does not see).  A row per thread
            // would be stored 16 bytes at a time to 32 places; through shared memory (4 KB per warp that no MMA
            // reads any more, 16-byte pieces swizzled by row) four rows leave as 128 contiguous bytes each.
            const float s = inv * w0;
            const uint32_t stage = sb + (join ? L::K_OFF : L::Q_OFF + side * 2 * L::QB) + (warp & 3u) * 4096u;
            const int rbase = r0 + (both ? side * kTile : 0) + int(warp & 3u) * 32;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(tO + c * 32, o);
                tmem_wait_ld();
                __syncwarp();  // the chunk before has been read
#pragma unroll
                for (int q = 0; q < 32; q += 4) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = __uint_as_float(o[q + e]) * s;
                        if (join) y[e] = fmaf(buf[(c * 32 + q + e) * 128 + i], w1, y[e]);
                    }
                    st_shared_v4(stage + lane * 128 + (((q >> 2) ^ (lane & 7)) << 4), __float_as_uint(y[0]),
                                 __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
                }
                __syncwarp();
#pragma unroll
                for (int a = 0; a < 8; ++a) {
                    const int rr = 4 * a + (lane >> 3), piece = lane & 7;
                    const float4 y = ld_shared_f4(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
                    const int64_t row = __shfl_sync(0xffffffffu, my_row, rr);
                    if (rbase + rr < nrows) {
                        const int64_t at = row * D + c * 32 + piece * 4;
                        if (p.direct) {
                            const __nv_bfloat162 b0 = __floats2bfloat162_rn(y.x, y.y), b1 = __floats2bfloat162_rn(y.z, y.w);
                            *reinterpret_cast<uint2*>(p.O + at) =
                                make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
                        } else {
                            *reinterpret_cast<float4*>(p.part + int64_t(slot) * all_rows * D + at) = y;
                        }
                    }
                }
            }
            if (live && !p.direct) p.part_lse[int64_t(slot) * all_rows + my_row] = my_lse;
            else if (live && p.lse) p.lse[my_row] = my_lse == -INFINITY ? -INFINITY : my_lse * kLn2;
        }
    } else if (warp < 12) {
        // ------------------------------------------- V: e4m3 to f16
        regs_dec<kOtherRegs>();
        const int tid = int(threadIdx.x) - 256;
        constexpr int CH = D / 16;     // 16-code pieces per token
        constexpr int RPI = 128 / CH;  // tokens per pass
        const int ch = tid % CH;
        int vexp[2] = {kMinVexp, kMinVexp};  // of each side when they take alternate tiles
        const bool free = wait_asleep(bar(L::QFULL), 0, abort_flag);  // the f16 tiles' place holds Q until then
        for (int tile = 0; tile < nt && free; ++tile) {
            const int vs = tile % L::VST, cs = tile % L::CST;
            const int valid = min(kTile, k1 - (k0 + tile * kTile));
            if (!wait_asleep(bar(L::VFULL + vs), (tile / L::VST) & 1, abort_flag)) break;
            if (!wait_asleep(bar(L::CEMPTY + cs), ((tile / L::CST) & 1) ^ 1, abort_flag)) break;
            const uint32_t src = sb + L::V_OFF + vs * kTile * D, dst = sb + L::C_OFF + cs * kTile * D * 2;
            const int ls = tile % L::SST;
            if (!wait_asleep(bar(L::LFULL + ls), (tile / L::SST) & 1, abort_flag)) break;
            const uint32_t sc = sb + L::S_OFF + ls * 1024;
            int bad_at = INT32_MAX;
            const int ve = tile_vexp(vexp[both ? 0 : tile & 1], sc + 512, valid, lane, 0, bad_at);
            vexp[both ? 0 : tile & 1] = ve;
            const float inv = pow2i(kVNorm + 127 - ve);
#pragma unroll 4
            for (int a = 0; a < kTile / RPI; ++a) {
                const int row = a * RPI + tid / CH;
                const uint32_t x = D == 128 ? uint32_t(row & 7) : uint32_t((row >> 1) & 3);
                uint4 v = lds128(src + row * D + ((uint32_t(ch) ^ x) << 4));
                const float sv = ld_shared_f32(sc + 512 + row * 4);
                float s = sv * inv;
                // whatever the page holds past the end, NaN too; value rows that are not finite
                if (row >= valid || __float_as_uint(sv) >= kNotFinite) v = make_uint4(0u, 0u, 0u, 0u), s = 0.0f;
                const __half2 s2 = __float2half2_rn(s);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t h2 = f16x2_of_codes(uint16_t(q & 1 ? w[q >> 1] >> 16 : w[q >> 1] & 0xffffu));
                    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h2), s2);
                    o[q] = *reinterpret_cast<const uint32_t*>(&r);
                }
                // 32 bytes: pieces 2 (ch % 4) and + 1 of the row in block ch / 4; the lanes of the other block
                // write theirs in the other order, so that eight lanes touch eight pieces
                const uint32_t at = dst + (ch >> 2) * (kTile * 128) + row * 128;
                const uint32_t flip = uint32_t(ch >> 2) & 1u;
                const uint32_t p0 = ((uint32_t(ch & 3) * 2u + flip) ^ uint32_t(row & 7)) << 4;
                const uint32_t p1 = ((uint32_t(ch & 3) * 2u + (flip ^ 1u)) ^ uint32_t(row & 7)) << 4;
                if (flip) {
                    st_shared_v4(at + p0, o[4], o[5], o[6], o[7]);
                    st_shared_v4(at + p1, o[0], o[1], o[2], o[3]);
                } else {
                    st_shared_v4(at + p0, o[0], o[1], o[2], o[3]);
                    st_shared_v4(at + p1, o[4], o[5], o[6], o[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(L::CFULL + cs));
                mbar_arrive(bar(L::VEMPTY + vs));
                mbar_arrive(bar(L::LEMPTY + ls));
            }
        }
    } else {
        regs_dec<kOtherRegs>();
        if (warp == 12) {
        // -------------------------------------------------------- loads
        const int ps = 1 << p.ps_shift;
        const int box = min(ps, kTile);       // rows of one copy
        const int per = kTile / box;          // copies of a full tile, one per lane
        int issued = 0;
        auto page_for = [&](int tile) {
            const int tok = k0 + tile * kTile + lane * box;
            return tile < nt && lane < per && tok < k1 ? page_of(p, k, tok, k1 - 1) : -1;
        };
        int page = page_for(0);
        for (int tile = 0; tile < nt; ++tile) {
            const int next = page_for(tile + 1);
            const int ks = tile % L::KST, vs = tile % L::VST;
            const int base = k0 + tile * kTile;
            const int copies = min(per, (k1 - base + box - 1) / box);
            const int32_t row = int32_t(((int64_t(page) * p.Hkv + h) << p.ps_shift) + (base & (ps - 1)));
            bool ok = wait_asleep(bar(L::KEMPTY + ks), ((tile / L::KST) & 1) ^ 1, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(L::KFULL + ks), uint32_t(copies * box * D));
            __syncwarp();
            if (lane < copies) tma_load_2d(sb + L::K_OFF + ks * kTile * D + lane * box * D, &tmK, bar(L::KFULL + ks), 0, row);
            const int ls = tile % L::SST;
            ok = wait_asleep(bar(L::LEMPTY + ls), ((tile / L::SST) & 1) ^ 1, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(L::LFULL + ls), uint32_t(copies * box * 8));
            __syncwarp();
            if (lane < copies) {
                const uint32_t sc = sb + L::S_OFF + ls * 1024 + lane * box * 4;
                bulk_load(sc, p.k_scale + row, uint32_t(box * 4), bar(L::LFULL + ls));
                bulk_load(sc + 512, p.v_scale + row, uint32_t(box * 4), bar(L::LFULL + ls));
            }
            ok = wait_asleep(bar(L::VEMPTY + vs), ((tile / L::VST) & 1) ^ 1, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(L::VFULL + vs), uint32_t(copies * box * D));
            __syncwarp();
            if (lane < copies) tma_load_2d(sb + L::V_OFF + vs * kTile * D + lane * box * D, &tmV, bar(L::VFULL + vs), 0, row);
            page = next;
            ++issued;
        }
        if (*abort_flag && lane == 0) {
            // Let every copy still in flight land before the CTA exits.
            volatile int no_abort = 0;
            for (int t = max(issued - 3, 0); t <= issued && t < nt; ++t) {
                mbar_wait(bar(L::KFULL + t % L::KST), (t / L::KST) & 1, &no_abort, 10000000ull);
                mbar_wait(bar(L::LFULL + t % L::SST), (t / L::SST) & 1, &no_abort, 10000000ull);
                mbar_wait(bar(L::VFULL + t % L::VST), (t / L::VST) & 1, &no_abort, 10000000ull);
            }
        }
        } else if (warp == 13 && lane == 0) {
        // ---------------------------------------------------------- MMA
        constexpr uint32_t idesc_s = idesc_e4m3_f32(128, kTile);
        constexpr uint32_t idesc_o = idesc_pv(D);
        bool any = false;
        int done[2] = {0, 0};  // P tiles consumed by each side
        // Descriptors of a step are made once and moved by constants (an address is the low 14 bits, 16 bytes each,
        // and stays below 227 KB): made anew for every MMA they cost the lane more than the MMA's 64 cycles.
        auto pv = [&](int side, int tile) {
            if (!wait_asleep(bar(L::PFULL + side), done[side] & 1, abort_flag)) return false;
            // (a tile that both sides use was waited for with side 0; a wait costs the lane 150 cycles even when what it
            // waits for is long there)
            if ((!both || side == 0) && !wait_asleep(bar(L::CFULL + tile % L::CST), (tile / L::CST) & 1, abort_flag))
                return false;
            tc_fence_after();
            const uint64_t v = nmajor_desc(sb + L::C_OFF + (tile % L::CST) * kTile * D * 2);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
                mma_f16_tmem_a(tmem + 256u + uint32_t(side) * 128u, tmem + uint32_t(side) * 128u + kk * 8,
                               v + uint64_t(kk * 2048 >> 4), idesc_o, (done[side] | kk) != 0);
            any = true;
            ++done[side];
            if (!both || side == 1) mma_commit(bar(L::CEMPTY + tile % L::CST));
            return true;
        };
        bool ok = wait_asleep(bar(L::QFULL), 0, abort_flag);
        for (int j = 0; j < steps && ok; ++j) {
            const int side = j & 1, tile = both ? j >> 1 : j;
            if (j >= 2) ok = pv(side, both ? tile - 1 : tile - 2);
            if (!ok) break;
            const int ks = tile % L::KST;
            if (!both || side == 0) ok = wait_asleep(bar(L::KFULL + ks), (tile / L::KST) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = kmajor_desc<D>(sb + L::K_OFF + ks * kTile * D), qd = kmajor_desc<D>(sb + L::Q_OFF + side * 2 * L::QB);
#pragma unroll
            for (int kk = 0; kk < 2 * (D / 32); ++kk) {
                const uint32_t term = kk >= D / 32 ? uint32_t(L::QB) : 0u, off = uint32_t(kk % (D / 32)) * 32u;
                mma_f8(tmem + uint32_t(side) * 128u, qd + ((term + off) >> 4), kd + (off >> 4), idesc_s, kk != 0);
            }
            any = true;
            mma_commit(bar(L::SFULL + side));
            if (!both || side == 1) mma_commit(bar(L::KEMPTY + ks));
        }
        for (int j = max(steps, 2); j < steps + 2 && ok; ++j) {  // the last tile of each side
            const int side = j & 1;
            ok = pv(side, both ? (j >> 1) - 1 : j - 2);
            if (ok) mma_commit(bar(L::OFULL + side));
        }
        if (*abort_flag && any) {
            // Wait for the tensor cores to finish before TMEM is freed.
            volatile int no_abort = 0;
            mma_commit(bar(L::DRAIN));
            mbar_wait(bar(L::DRAIN), 0, &no_abort, 10000000ull);
        }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace attend
}  // namespace mfp8
