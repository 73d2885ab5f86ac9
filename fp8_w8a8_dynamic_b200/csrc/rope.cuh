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
// Memory-bound: every value is read once (16-byte vectors) and written once.
// A block takes the rows of one or a few whole tokens, so the cosines and
// sines of a token are computed once (64-bit sincos, about 40 operations per
// pair) and shared through shared memory by all its heads; its rows' loads
// are issued before that arithmetic.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace mfp8 {
namespace rope {

constexpr int kThreads = 256;
constexpr int kItems = 3;       // row vectors per thread and pass, loads issued first
constexpr int kMaxTokens = 16;  // tokens per block
constexpr int kMaxHalf = 128;   // rot / 2 <= D / 2 <= 128

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
    int tokens_per_block;
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

// Two values of a row and their partners' (half layout): fl(x c) + fl(p s),
// the sign of s chosen by the caller.
__device__ __forceinline__ uint32_t rotate2(uint32_t x, uint32_t p, float c0, float c1, float s0, float s1) {
    const uint64_t a = mul2(pack2(bf16_lo(x), bf16_hi(x)), pack2(c0, c1));
    const uint64_t b = mul2(pack2(bf16_lo(p), bf16_hi(p)), pack2(s0, s1));
    float lo, hi;
    unpack2(add2(a, b), lo, hi);
    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&y);
}

// LPR lanes per row, a power of two >= D / 8.
template <int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
rope_store_kernel(const Params p) {
    grid_launch_dependents();
    grid_dependency_wait();  // X may be the previous kernel's output
    extern __shared__ __align__(16) float cs[];  // cosines, then sines, [tokens_per_block][rot / 2]
    const int half = p.rot >> 1;
    const int tok0 = blockIdx.x * p.tokens_per_block;
    const int toks = min(p.tokens_per_block, p.T - tok0);
    const int heads = p.nq + p.nk + p.nv;
    const int rows = toks * heads;
    const int v = threadIdx.x % LPR;
    const int lane = threadIdx.x & 31;
    constexpr int kRowsPerPass = kThreads / LPR;
    float* cosv = cs;
    float* sinv = cs + p.tokens_per_block * half;

    for (int base = 0; base < rows; base += kRowsPerPass * kItems) {
        uint4 x[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int row = base + k * kRowsPerPass + int(threadIdx.x) / LPR;
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows && v < p.vpr) {
                const int t = row / heads;
                x[k] = p.X[int64_t(tok0 + t) * p.ldx + int64_t(row - t * heads) * p.vpr + v];
            }
        }
        if (base == 0 && half > 0) {
            for (int i = threadIdx.x; i < toks * half; i += kThreads) {
                const int t = i / half, f = i - t * half;
                const int ax = p.axis != nullptr ? min(int(p.axis[f]), p.n_axes - 1) : 0;
                cos_sin(p.pos[int64_t(ax) * p.T + tok0 + t], p.inv_freq[f], p.mscale, cosv[i], sinv[i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int row = base + k * kRowsPerPass + int(threadIdx.x) / LPR;
            const bool live = row < rows && v < p.vpr;
            const int t = row < rows ? row / heads : 0;
            const int h = row < rows ? row - t * heads : 0;
            uint4 y = x[k];
            if (half > 0) {
                if (INTERLEAVED) {
                    if (live && h < p.nq + p.nk && v * 8 < p.rot) {
                        const float4 c = *reinterpret_cast<const float4*>(cosv + t * half + v * 4);
                        const float4 s = *reinterpret_cast<const float4*>(sinv + t * half + v * 4);
                        // the pair is one word: (x1, x2) and its swap (x2, x1)
                        y.x = rotate2(x[k].x, __byte_perm(x[k].x, 0u, 0x1032u), c.x, c.x, -s.x, s.x);
                        y.y = rotate2(x[k].y, __byte_perm(x[k].y, 0u, 0x1032u), c.y, c.y, -s.y, s.y);
                        y.z = rotate2(x[k].z, __byte_perm(x[k].z, 0u, 0x1032u), c.z, c.z, -s.z, s.z);
                        y.w = rotate2(x[k].w, __byte_perm(x[k].w, 0u, 0x1032u), c.w, c.w, -s.w, s.w);
                    }
                } else {
                    const int hv = p.rot >> 4;  // vectors in each half
                    const bool first = v < hv;
                    const int src = (lane & ~(LPR - 1)) + (first ? v + hv : v < 2 * hv ? v - hv : v);
                    uint4 q;
                    q.x = __shfl_sync(0xffffffffu, x[k].x, src);
                    q.y = __shfl_sync(0xffffffffu, x[k].y, src);
                    q.z = __shfl_sync(0xffffffffu, x[k].z, src);
                    q.w = __shfl_sync(0xffffffffu, x[k].w, src);
                    if (live && h < p.nq + p.nk && v < 2 * hv) {
                        const int f = t * half + (first ? v : v - hv) * 8;
                        const float4 c0 = *reinterpret_cast<const float4*>(cosv + f);
                        const float4 c1 = *reinterpret_cast<const float4*>(cosv + f + 4);
                        float4 s0 = *reinterpret_cast<const float4*>(sinv + f);
                        float4 s1 = *reinterpret_cast<const float4*>(sinv + f + 4);
                        if (first) {
                            s0 = make_float4(-s0.x, -s0.y, -s0.z, -s0.w);
                            s1 = make_float4(-s1.x, -s1.y, -s1.z, -s1.w);
                        }
                        y.x = rotate2(x[k].x, q.x, c0.x, c0.y, s0.x, s0.y);
                        y.y = rotate2(x[k].y, q.y, c0.z, c0.w, s0.z, s0.w);
                        y.z = rotate2(x[k].z, q.z, c1.x, c1.y, s1.x, s1.y);
                        y.w = rotate2(x[k].w, q.w, c1.z, c1.w, s1.z, s1.w);
                    }
                }
            }
            if (live && h < p.nq) p.Y[int64_t(tok0 + t) * p.ldy + int64_t(h) * p.vpr + v] = y;
            if (p.nk + p.nv > 0) {
                const uint32_t acc = absmax_bits_u4(y, 0u);
                uint32_t amax = max(acc & 0xffffu, acc >> 16);
#pragma unroll
                for (int off = 1; off < LPR; off <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                if (live && h >= p.nq) {
                    const int64_t slot = p.slot[tok0 + t];
                    if (slot >= p.n_slots) {
                        record_device_status(MFP8_ERR_INDEX);
                    } else if (slot >= 0) {
                        const bool key = h < p.nq + p.nk;
                        const int hk = key ? h - p.nq : h - p.nq - p.nk;
                        const int nh = key ? p.nk : p.nv;
                        const int64_t r = ((((slot >> p.ps_shift) * nh) + hk) << p.ps_shift) +
                                          (slot & ((int64_t(1) << p.ps_shift) - 1));
                        const float s = scale_from_absmax_bits(amax);
                        if (v == 0) (key ? p.k_scale : p.v_scale)[r] = s;
                        (key ? p.K : p.V)[r * p.vpr + v] = quantize8(y, s, __frcp_rn(s));
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

template <int LPR>
__global__ void __launch_bounds__(kThreads)
page_read_kernel(const uint2* __restrict__ C, const float* __restrict__ S, const int64_t* __restrict__ slot,
                 int64_t n_slots, int ps_shift, int R, int H, int vpr, uint4* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int kRowsPerPass = kThreads / LPR;
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
