// rope.cuh — rotary positions, and the paged FP8 KV cache written behind
// them and read back.
//
// Rotary positions.  Each head row of D values is rotated in its first `rot`
// values, pair by pair; the others pass unchanged.  Pair i (0 <= i < rot/2)
// is (x[i], x[i + rot/2]) in the half layout and (x[2i], x[2i+1]) in the
// interleaved one, and
//   a = pos * inv_freq[i],  c = fl32(mscale cos a),  s = fl32(mscale sin a),
//   y1 = bf16(fl32(fl32(x1 c) - fl32(x2 s))),
//   y2 = bf16(fl32(fl32(x2 c) + fl32(x1 s))).
// A frequency may follow any of several position axes (the interleaved
// M-RoPE of the "MOSS-VL-Instruct-0708-FP8 architecture" article has three,
// and its contexts reach 256K positions, so angles are formed and reduced in
// 64 bits: at position 2^18 an fp32 angle is off by up to 2^-7).
//
// Cache.  Pages [n_pages][H][page_size][D] of e4m3 codes and scales
// [n_pages][H][page_size] fp32: within a page the rows of one head are
// contiguous, so a reader of one head takes whole lines of both.  A row is
// quantized by the rule of quant.cuh (s = max(fl32(max|x| / 448), FLT_MIN),
// q = e4m3(fl32(x / s))), keys after rotation and rounding to bf16, so the
// bytes are those of mfp8_kv_quantize on the rotated bf16 keys.  Token t goes
// to slot[t] = page * page_size + place; a negative slot is padding.
//
// Memory-bound: every value is read once (16-byte vectors) and written once,
// so what counts is how few instructions a vector costs.  A thread takes two
// vectors of a row at a time, in the half layout one of each half, which need
// the same cosines and sines; those stay in its registers for all the heads
// that it serves.  A block takes one token (or a few narrow ones): 64-bit
// sincos, about 200 instructions for a pair, once per pair and token through
// shared memory, behind the first loads.  Rotating 16384 tokens of 32 x 128
// values (268 MB) took 79 us with a vector per thread and shuffles between
// the halves (75% of the issue slots busy), 52 us with two vectors per thread
// at 80 registers, 43 us at 64 (6.2 TB/s), 62 us at 48.  At 64 every build
// spills a little: the half layout 44 bytes out and 40 in with two rows per
// pass, 100 and 216 with three.  The fused store of 16384 tokens of 32 + 8 + 8
// rows (370 MB; three rows): 117, 86, 71 us.  Lanes and rows are powers of two:
// 20 heads of 96 use 120 of 256 places in two passes, 36 heads of 64 144 of 256.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace mfp8 {
namespace rope {

constexpr int kThreads = 128;
constexpr int kBlocksPerSm = 8;  // 64 registers a thread: loads of 1024 threads in flight hide HBM's latency

// Rows of a token, in order: nq rotated rows written to Y, nk rotated rows
// quantized into the K pages, nv rows quantized into the V pages.  rot = 0
// rotates nothing.
struct Params {
    const uint4* X;      // [T] rows of ldx 8-value vectors
    int64_t ldx;         // vectors between tokens
    const int32_t* pos;  // [n_axes][T]
    const uint8_t* axis; // [rot / 2], null: axis 0
    const float* inv_freq;
    int n_axes;
    int rot;
    double mscale;
    int T, nq, nk, nv;
    int vpr;  // vectors per row, D / 8
    int tpt_shift;  // log2 of the threads per token
    uint4* Y;
    int64_t ldy;
    const int64_t* slot;
    int64_t n_slots;  // n_pages * page_size
    int ps_shift;
    uint2* K;
    float* k_scale;
    uint2* V;
    float* v_scale;
};

// Cosine and sine of pos * inv_freq, each times mscale and rounded to fp32.
// The angle is one 64-bit product; whole turns are taken off with 2 pi split
// into a 53-bit head and its remainder (Cody and Waite's reduction): the
// head's multiple is exact in the fused multiply-add, since the difference
// is a multiple of 2^-50 below 4.
__device__ __forceinline__ void cos_sin(int32_t pos, float inv_freq, double mscale, float& c, float& s) {
    const double kTwoPiHi = 6.283185307179586232;      // fl64(2 pi)
    const double kTwoPiLo = 2.4492935982947064e-16;    // 2 pi - fl64(2 pi)
    const double kInvTwoPi = 0.15915494309189533577;   // 1 / (2 pi)
    const double kInvPi = 0.31830988618379067154;      // 1 / pi
    const double a = double(pos) * double(inv_freq);
    const double k = rint(a * kInvTwoPi);
    const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, a));
    double sd, cd;
    sincospi(r * kInvPi, &sd, &cd);
    c = float(cd * mscale);
    s = float(sd * mscale);
}

// Half layout: two pairs, x1 and x2 packed bf16 words.
__device__ __forceinline__ void rotate_half2(uint32_t& x1, uint32_t& x2, float c0, float c1, float s0, float s1) {
    const uint64_t a = pack2(bf16_lo(x1), bf16_hi(x1)), b = pack2(bf16_lo(x2), bf16_hi(x2));
    const uint64_t c = pack2(c0, c1), s = pack2(s0, s1);
    float lo, hi;
    unpack2(sub2(mul2(a, c), mul2(b, s)), lo, hi);
    const __nv_bfloat162 y1 = __floats2bfloat162_rn(lo, hi);
    unpack2(add2(mul2(b, c), mul2(a, s)), lo, hi);
    const __nv_bfloat162 y2 = __floats2bfloat162_rn(lo, hi);
    x1 = *reinterpret_cast<const uint32_t*>(&y1);
    x2 = *reinterpret_cast<const uint32_t*>(&y2);
}

// Interleaved layout: one pair, a packed bf16 word.
__device__ __forceinline__ void rotate_word(uint32_t& x, float c, float s) {
    const float a = bf16_lo(x), b = bf16_hi(x);
    float lo, hi;
    unpack2(add2(mul2(pack2(a, b), pack2(c, c)), mul2(pack2(b, a), pack2(-s, s))), lo, hi);
    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
    x = *reinterpret_cast<const uint32_t*>(&y);
}

// UPR lanes per row, a power of two >= D / 16, two vectors each; ITEMS rows
// per thread and pass, their loads issued first.
template <int UPR, bool INTERLEAVED, int ITEMS>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
rope_store_kernel(const Params p) {
    grid_launch_dependents();
    grid_dependency_wait();  // X may be the previous kernel's output
    extern __shared__ __align__(16) float cs[];  // cosines, then sines, [tokens of the block][rot / 2]
    const int half = p.rot >> 1;
    const int tpt = 1 << p.tpt_shift;
    const int tpb = kThreads >> p.tpt_shift;
    const int tok0 = blockIdx.x * tpb;
    const int tb = int(threadIdx.x) >> p.tpt_shift;  // token within the block
    const int token = tok0 + tb;
    const int j = int(threadIdx.x) & (tpt - 1);
    const int u = j % UPR, h0 = j / UPR, hstep = tpt / UPR;
    const int heads = p.nq + p.nk + p.nv;
    // the two vectors of a row: the same places in both halves, or neighbours
    const int hv = p.rot >> 4;
    const bool turns = u < hv;  // (interleaved: vectors 2u and 2u + 1 lie below rot together)
    const int v0 = INTERLEAVED || half == 0 ? 2 * u : turns ? u : hv + u + (u - hv);
    const int v1 = INTERLEAVED || !turns ? v0 + 1 : v0 + hv;
    const bool live = token < p.T && u < (p.vpr >> 1);
    const uint4* x = p.X + int64_t(token) * p.ldx;

    uint4 a[ITEMS], b[ITEMS];
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int h = base + k * hstep;
            a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
            if (live && h < heads) {
                a[k] = x[int64_t(h) * p.vpr + v0];
                b[k] = x[int64_t(h) * p.vpr + v1];
            }
        }
    };
    load(h0);
    float c[8], s[8];
    if (half > 0) {
        float* cosv = cs;
        float* sinv = cs + tpb * half;
        const int n = min(tpb, p.T - tok0) * half;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int t = i / half, f = i - t * half;
            const int ax = p.axis != nullptr ? min(int(p.axis[f]), p.n_axes - 1) : 0;
            cos_sin(p.pos[int64_t(ax) * p.T + tok0 + t], p.inv_freq[f], p.mscale, cosv[i], sinv[i]);
        }
        __syncthreads();
        if (live && turns) {
#pragma unroll
            for (int q = 0; q < 8; q += 4) {
                const float4 cv = *reinterpret_cast<const float4*>(cosv + tb * half + u * 8 + q);
                const float4 sv = *reinterpret_cast<const float4*>(sinv + tb * half + u * 8 + q);
                c[q] = cv.x, c[q + 1] = cv.y, c[q + 2] = cv.z, c[q + 3] = cv.w;
                s[q] = sv.x, s[q + 1] = sv.y, s[q + 2] = sv.z, s[q + 3] = sv.w;
            }
        }
    }
    // where the token's rows go in the pages
    int64_t place = -1;  // row within its page
    int64_t page = 0;
    if (p.nk + p.nv > 0 && token < p.T) {
        const int64_t slot = p.slot[token];
        if (slot >= p.n_slots) record_device_status(MFP8_ERR_INDEX);
        else if (slot >= 0) {
            page = slot >> p.ps_shift;
            place = slot & ((int64_t(1) << p.ps_shift) - 1);
        }
    }
    // every thread of a warp makes the same number of passes (the shuffles want them all)
    for (int base = h0; base - h0 < heads; base += ITEMS * hstep) {
        if (base != h0) load(base);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int h = base + k * hstep;
            if (h - h0 >= heads) break;  // no thread has a row here
            const bool mine = live && h < heads;
            if (half > 0 && turns && h < p.nq + p.nk) {
                uint32_t* xa = reinterpret_cast<uint32_t*>(&a[k]);
                uint32_t* xb = reinterpret_cast<uint32_t*>(&b[k]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (INTERLEAVED) {
                        rotate_word(xa[q], c[q], s[q]);
                        rotate_word(xb[q], c[q + 4], s[q + 4]);
                    } else {
                        rotate_half2(xa[q], xb[q], c[2 * q], c[2 * q + 1], s[2 * q], s[2 * q + 1]);
                    }
                }
            }
            if (mine && h < p.nq) {
                uint4* y = p.Y + int64_t(token) * p.ldy + int64_t(h) * p.vpr;
                y[v0] = a[k];
                y[v1] = b[k];
            }
            if (p.nk + p.nv > 0) {
                const uint32_t acc = absmax_bits_u4(b[k], absmax_bits_u4(a[k], 0u));
                uint32_t amax = max(acc & 0xffffu, acc >> 16);
#pragma unroll
                for (int off = 1; off < UPR; off <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                if (mine && h >= p.nq && place >= 0) {
                    const bool key = h < p.nq + p.nk;
                    const int hk = key ? h - p.nq : h - p.nq - p.nk;
                    const int64_t r = ((page * (key ? p.nk : p.nv) + hk) << p.ps_shift) + place;
                    const float sc = scale_from_absmax_bits(amax);
                    if (u == 0) (key ? p.k_scale : p.v_scale)[r] = sc;
                    uint2* q = (key ? p.K : p.V) + r * p.vpr;
                    if (sc >= kFmaMinScale) {
                        const float rc = __frcp_rn(sc);
                        q[v0] = quantize8_fast(a[k], sc, rc);
                        q[v1] = quantize8_fast(b[k], sc, rc);
                    } else {
                        q[v0] = quantize8_div_call(a[k], sc);
                        q[v1] = quantize8_div_call(b[k], sc);
                    }
                }
            }
        }
    }
}

// Read back: out[t][h][:] = bf16(fl32(dec(code) * scale)) of slot[t], the
// rounding of mfp8_kv_dequantize; zeros for a negative slot.  A thread takes
// kReadItems vectors of 8 codes, all loads issued first; a row's lanes are
// contiguous.
constexpr int kReadItems = 4;
constexpr int kReadThreads = 256;

template <int LPR>
__global__ void __launch_bounds__(kReadThreads)
page_read_kernel(const uint2* __restrict__ C, const float* __restrict__ S, const int64_t* __restrict__ slot,
                 int64_t n_slots, int ps_shift, int R, int H, int vpr, uint4* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int kRowsPerPass = kReadThreads / LPR;
    const int v = threadIdx.x % LPR;
    const int64_t row0 = int64_t(blockIdx.x) * (kRowsPerPass * kReadItems) + threadIdx.x / LPR;
    uint2 q[kReadItems];
    float s[kReadItems];
#pragma unroll
    for (int k = 0; k < kReadItems; ++k) {
        const int64_t row = row0 + k * kRowsPerPass;
        q[k] = make_uint2(0u, 0u);
        s[k] = 0.0f;
        if (row < R && v < vpr) {
            const int t = int(row) / H, h = int(row) - t * H;
            const int64_t at = __ldg(slot + t);
            if (at >= n_slots) {
                record_device_status(MFP8_ERR_INDEX);
            } else if (at >= 0) {
                const int64_t r = ((((at >> ps_shift) * H) + h) << ps_shift) + (at & ((int64_t(1) << ps_shift) - 1));
                q[k] = __ldcs(C + r * vpr + v);
                s[k] = __ldg(S + r);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kReadItems; ++k) {
        const int64_t row = row0 + k * kRowsPerPass;
        if (row < R && v < vpr)
            __stcs(out + row * vpr + v,
                   make_uint4(dequant2(uint16_t(q[k].x & 0xffffu), s[k]), dequant2(uint16_t(q[k].x >> 16), s[k]),
                              dequant2(uint16_t(q[k].y & 0xffffu), s[k]), dequant2(uint16_t(q[k].y >> 16), s[k])));
    }
}

}  // namespace rope
}  // namespace mfp8
