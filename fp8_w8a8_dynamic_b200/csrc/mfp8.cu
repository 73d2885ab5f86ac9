// mfp8.cu — the C ABI declared in include/mfp8.h: argument checks, kernel
// choice, TMA descriptor set-up and launches.  The whole library is this
// one translation unit.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "../../include/mfp8.h"
#include "status.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "gemm_tiled.cuh"
#include "gemm_pair.cuh"
#include "gemm_stream.cuh"
#include "gemm_cluster.cuh"
#include "producer.cuh"
#include "kv8.cuh"
#include "rope.cuh"
#include "attend.cuh"
#include "attend_wide.cuh"

namespace mfp8 {
namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = int64_t(1) << 30;  // rows / columns accepted per dimension

struct DeviceInfo {
    bool ready = false;
    bool supported = false;
    int sm_count = 0;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

mfp8_status current_device(int* dev_out, DeviceInfo* info_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo& d = g_dev[dev];
    if (!d.ready) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return MFP8_ERR_CUDA;
        }
        d.supported = (major == 10 && minor == 0);
        d.sm_count = sms;
        d.ready = true;
    }
    if (!g_encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || fn == nullptr) {
            cudaGetLastError();
            return MFP8_ERR_CUDA;
        }
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    if (!d.supported) return MFP8_ERR_DEVICE;
    *dev_out = dev;
    *info_out = d;
    return MFP8_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// [rows, cols] row-major 8-bit matrix, tiles of box_rows x 128 bytes with
// the 128-byte swizzle.
mfp8_status make_map_u8(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows) {
    cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(cols)};
    cuuint32_t box[2] = {128u, cuuint32_t(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MFP8_OK : MFP8_ERR_CUDA;
}

// Y [rows, cols] bf16 for the TMA-store epilogue: 32 x 32 boxes, 64-byte
// rows with the 64-byte swizzle (cols % 8 == 0, so rows are 16-byte aligned).
mfp8_status make_map_y(CUtensorMap* map, void* base, int64_t rows, int64_t cols) {
    cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(cols) * 2};
    cuuint32_t box[2] = {32u, 32u};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MFP8_OK : MFP8_ERR_CUDA;
}

bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

mfp8_status launch_status() {
    return cudaGetLastError() == cudaSuccess ? MFP8_OK : MFP8_ERR_CUDA;
}

// ------------------------------------------------------------- quantize --

template <class Kern>
mfp8_status launch_quant(Kern kern, bool dependent, int64_t R, const uint4* x, int64_t K, uint2* q, float* S,
                         cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(R));  // one block per row
    cfg.blockDim = dim3(kQuantThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, x, K, q, S) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

// The warp-per-row kernel: `blocks` blocks of 8 rows, R rows in all.
template <class Kern>
mfp8_status launch_quant(Kern kern, bool dependent, int64_t blocks, int64_t R, const uint4* x, int64_t K, uint2* q,
                         float* S, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kQuantThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, x, R, K, q, S) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

template <bool EARLY_TRIGGER>
mfp8_status quantize_rows_t(const void* X, int64_t R, int64_t K, void* Q, float* S, cudaStream_t stream) {
    if (R == 0) return MFP8_OK;
    const int64_t nvec = K / 8;
    const uint4* x = static_cast<const uint4*>(X);
    uint2* q = static_cast<uint2*>(Q);
    // Many rows: 1, 2 or 4 warps per row (8 warps per block) while a row
    // fits in their registers; longer rows get more warps.
    auto blocks = [&](int wpr) { return (R * wpr + kQuantThreads / 32 - 1) / (kQuantThreads / 32); };
    if (R >= 256 && nvec <= 32 * 16 * 4 && blocks(4) <= INT32_MAX) {
        if (nvec <= 32 * 4)
            return launch_quant(quant_rows_warp_kernel<4, 1, EARLY_TRIGGER>, EARLY_TRIGGER, blocks(1), R, x, K, q, S,
                                stream);
        if (nvec <= 32 * 8)
            return launch_quant(quant_rows_warp_kernel<8, 1, EARLY_TRIGGER>, EARLY_TRIGGER, blocks(1), R, x, K, q, S,
                                stream);
        if (nvec <= 32 * 8 * 2)
            return launch_quant(quant_rows_warp_kernel<8, 2, EARLY_TRIGGER>, EARLY_TRIGGER, blocks(2), R, x, K, q, S,
                                stream);
        if (nvec <= 32 * 8 * 4)
            return launch_quant(quant_rows_warp_kernel<8, 4, EARLY_TRIGGER>, EARLY_TRIGGER, blocks(4), R, x, K, q, S,
                                stream);
        if (nvec <= 32 * 12 * 4)
            return launch_quant(quant_rows_warp_kernel<12, 4, EARLY_TRIGGER>, EARLY_TRIGGER, blocks(4), R, x, K, q, S,
                                stream);
        return launch_quant(quant_rows_warp_kernel<16, 4, EARLY_TRIGGER>, EARLY_TRIGGER, blocks(4), R, x, K, q, S,
                            stream);
    }
    if (nvec <= 256) return launch_quant(quant_rows_reg_kernel<1, EARLY_TRIGGER>, EARLY_TRIGGER, R, x, K, q, S, stream);
    if (nvec <= 512) return launch_quant(quant_rows_reg_kernel<2, EARLY_TRIGGER>, EARLY_TRIGGER, R, x, K, q, S, stream);
    if (nvec <= 1024) return launch_quant(quant_rows_reg_kernel<4, EARLY_TRIGGER>, EARLY_TRIGGER, R, x, K, q, S, stream);
    if (nvec <= 1536) return launch_quant(quant_rows_reg_kernel<6, EARLY_TRIGGER>, EARLY_TRIGGER, R, x, K, q, S, stream);
    if (nvec <= 2048) return launch_quant(quant_rows_reg_kernel<8, EARLY_TRIGGER>, EARLY_TRIGGER, R, x, K, q, S, stream);
    return launch_quant(quant_rows_loop_kernel<EARLY_TRIGGER>, EARLY_TRIGGER, R, x, K, q, S, stream);
}

// Activations: the GEMM launched next may start its prologue early.
mfp8_status quantize_act_rows(const void* X, int64_t R, int64_t K, void* Q, float* S, cudaStream_t stream) {
    return quantize_rows_t<true>(X, R, K, Q, S, stream);
}

// Weights: no early start for whatever follows.
mfp8_status quantize_weight_rows(const void* X, int64_t R, int64_t K, void* Q, float* S, cudaStream_t stream) {
    return quantize_rows_t<false>(X, R, K, Q, S, stream);
}

mfp8_status check_quant_args(const void* X, int64_t R, int64_t K, const void* Q, const float* S) {
    if (R < 0 || K < 0) return MFP8_ERR_INVALID_ARG;
    if (K == 0 || K % 16 != 0 || K > kMaxDim || R > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (R == 0) return MFP8_OK;
    if (!X || !Q || !S) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Q) || !aligned16(S)) return MFP8_ERR_MISALIGNED;
    if (ranges_overlap(X, size_t(R * K * 2), Q, size_t(R * K)) ||
        ranges_overlap(X, size_t(R * K * 2), S, size_t(R * 4)) ||
        ranges_overlap(Q, size_t(R * K), S, size_t(R * 4)))
        return MFP8_ERR_INVALID_ARG;
    return MFP8_OK;
}

// ----------------------------------------------------------------- GEMM --


template <class Kern>
mfp8_status set_smem(Kern kern, int bytes, int dev, bool* done) {
    if (done[dev]) return MFP8_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    done[dev] = true;
    return MFP8_OK;
}

template <int BN, int STAGES>
mfp8_status launch_tiled_bn(const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8,
                            const float* s_w, int64_t N, int64_t w_rows, void* Y, bool dependent, int dev,
                            const DeviceInfo& info,
                            cudaStream_t stream) {
    using L = tiled::Layout<BN, STAGES>;
    auto kern = tiled::gemm_tiled_kernel<BN, STAGES>;
    static bool attr_done[kMaxDevices] = {};
    mfp8_status st = set_smem(kern, L::SMEM_BYTES, dev, attr_done);
    if (st != MFP8_OK) return st;
    CUtensorMap tmX, tmW, tmY;
    if ((st = make_map_u8(&tmX, X8, M, K, tiled::BM)) != MFP8_OK) return st;
    if ((st = make_map_u8(&tmW, W8, w_rows, K, BN)) != MFP8_OK) return st;
    if ((st = make_map_y(&tmY, Y, M, N)) != MFP8_OK) return st;
    const int64_t tiles = ((M + tiled::BM - 1) / tiled::BM) * ((N + BN - 1) / BN);
    const unsigned grid = static_cast<unsigned>(tiles < info.sm_count ? tiles : info.sm_count);

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(tiled::kThreads);
    cfg.dynamicSmemBytes = L::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tmX, tmW, tmY, s_a, s_w, static_cast<__nv_bfloat16*>(Y), int(M), int(N),
                           int(K)) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

// The 1-CTA kernel's tile width: 256 when that already gives a CTA to most
// SMs, else the widest of 128, 64, 32 that does (narrower tiles re-read the
// X8 row panel more often from L2, but a mid-sized M with 256-wide tiles
// leaves most SMs idle: M = 128, N = 4096 is 16 tiles).
int tiled_tile_width(int64_t M, int64_t N, const DeviceInfo& info) {
    const int64_t mt = (M + tiled::BM - 1) / tiled::BM;
    for (int bn : {256, 128, 64})
        if (mt * ((N + bn - 1) / bn) * 4 >= int64_t(info.sm_count) * 3) return bn;
    return 32;
}

mfp8_status launch_tiled(const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8,
                         const float* s_w, int64_t N, int64_t w_rows, void* Y, bool dependent, int dev,
                         const DeviceInfo& info,
                         cudaStream_t stream) {
    switch (tiled_tile_width(M, N, info)) {
        case 256: return launch_tiled_bn<256, 4>(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
        case 128: return launch_tiled_bn<128, 6>(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
        case 64: return launch_tiled_bn<64, 8>(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
        default: return launch_tiled_bn<32, 10>(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
    }
}

// Clusters of `S` CTAs of `kern` (with `smem` bytes each) that the device
// keeps resident at once.  Clusters are placed inside one GPC, so this can be
// below (SMs x CTAs per SM) / S.  Cached per device and kernel.
template <class Kern>
int max_active_clusters(Kern kern, int S, int smem, int threads, int dev) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int, int>, int> cache;
    const auto key = std::make_tuple(dev, reinterpret_cast<const void*>(kern), S, smem);
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(S));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    cache[key] = n;
    return n;
}

template <int BN, int STAGES>
mfp8_status launch_pair_bn(const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8, const float* s_w,
                           int64_t N, int64_t w_rows, void* Y, bool dependent, int dev, const DeviceInfo& info,
                           cudaStream_t stream) {
    using L = pair::Layout<BN, STAGES>;
    auto kern = pair::gemm_pair_kernel<BN, STAGES>;
    static bool attr_done[kMaxDevices] = {};
    mfp8_status st = set_smem(kern, L::SMEM_BYTES, dev, attr_done);
    if (st != MFP8_OK) return st;
    CUtensorMap tmX, tmW, tmY;
    if ((st = make_map_u8(&tmX, X8, M, K, pair::HALF)) != MFP8_OK) return st;
    if ((st = make_map_u8(&tmW, W8, w_rows, K, BN / 2)) != MFP8_OK) return st;
    if ((st = make_map_y(&tmY, Y, M, N)) != MFP8_OK) return st;
    const int64_t tiles = ((M + pair::BM - 1) / pair::BM) * ((N + BN - 1) / BN);
    // The grid is persistent: only as many pairs as can be resident at once.
    int64_t max_pairs = max_active_clusters(kern, 2, L::SMEM_BYTES, pair::kThreads, dev);
    if (max_pairs <= 0 || max_pairs > info.sm_count / 2) max_pairs = info.sm_count / 2;
    const int64_t pairs = tiles < max_pairs ? tiles : max_pairs;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * pairs));
    cfg.blockDim = dim3(pair::kThreads);
    cfg.dynamicSmemBytes = L::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tmX, tmW, tmY, s_a, s_w, static_cast<__nv_bfloat16*>(Y), int(M), int(N),
                           int(K)) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

// Tile width for the pair kernel: the one that finishes sooner, counting
// rounds of tiles over the CTA pairs times the time of one tile.  A
// 256 x 128 tile moves 3/4 of the bytes of a 256 x 256 tile for half the
// MACs and measured about 1.45x slower per MAC, so it is chosen only when it
// saves rounds (narrow N, e.g. the k/v projections at M = 2048).
int pair_tile_width(int64_t M, int64_t N, const DeviceInfo& info) {
    const int64_t pairs = info.sm_count / 2;
    const int64_t mt = (M + pair::BM - 1) / pair::BM;
    const int64_t r256 = (mt * ((N + 255) / 256) + pairs - 1) / pairs;
    const int64_t r128 = (mt * ((N + 127) / 128) + pairs - 1) / pairs;
    return double(r128) * 128.0 * 1.45 < double(r256) * 256.0 ? 128 : 256;
}

mfp8_status launch_pair(const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8, const float* s_w,
                        int64_t N, int64_t w_rows, void* Y, bool dependent, int dev, const DeviceInfo& info,
                        cudaStream_t stream) {
    if (pair_tile_width(M, N, info) == 128)
        return launch_pair_bn<128, 8>(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
    return launch_pair_bn<256, 6>(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
}

constexpr int64_t kStreamMaxM = stream::kMaxM;
constexpr int64_t kClusterMaxM = cluster::kMaxM;

int sm_count_for_sizing();

int choose_path(int64_t M, int64_t N, int64_t K) {
    (void)K;
    if (M <= kStreamMaxM) return MFP8_PATH_FUSED;
    // The cluster split-K kernel up to 128 rows (measured ahead of the
    // 128-row tiles there on the layer's shapes); above, its stages of a
    // weight block and up to 256 code rows leave too shallow a ring and the
    // tiles are faster.
    if (M <= 128) return MFP8_PATH_SPLITK;
    if (M < 256) return MFP8_PATH_TILED;
    // Too few 256 x 256 pair tiles to occupy half the CTA pairs (the k/v
    // projections at M = 2048 make 32): narrower single-CTA tiles fill the
    // GPU instead.
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    if (pair_tiles * 4 < sm_count_for_sizing()) return MFP8_PATH_TILED;
    return MFP8_PATH_PAIR;
}

mfp8_status check_gemm_args(int64_t M, int64_t N, int64_t K, const void* W8, const float* s_w, const void* Y) {
    if (M < 0 || N < 0 || K < 0) return MFP8_ERR_INVALID_ARG;
    if (K == 0 || K % 16 != 0 || N == 0 || K > kMaxDim || N > kMaxDim || M > kMaxDim)
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (M > 0 && M * (K > N ? K : N) > (int64_t(1) << 40)) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (!W8 || !s_w || (M > 0 && !Y)) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(W8) || !aligned16(s_w) || !aligned16(Y)) return MFP8_ERR_MISALIGNED;
    if (M > 0 && (ranges_overlap(Y, size_t(M * N * 2), W8, size_t(N * K)) ||
                  ranges_overlap(Y, size_t(M * N * 2), s_w, size_t(N * 4))))
        return MFP8_ERR_INVALID_ARG;
    return MFP8_OK;
}

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// How one call uses the caller's workspace: the activation codes X8 [M, K]
// and scales s_a [M] of the quantize pass, each 256-byte aligned.  Nothing
// in it outlives the call.
struct Plan {
    size_t x8_off = 0, sa_off = 0, total = 0;
};

Plan make_plan(int64_t M, int64_t K, bool codes) {
    Plan p;
    if (!codes) return p;  // nothing to keep: no workspace needed
    p.x8_off = 0;
    p.sa_off = round_up(size_t(M) * size_t(K), 256);
    p.total = p.sa_off + round_up(size_t(M) * 4, 256);
    return p;
}

// N not a multiple of 8: rows of Y are not 16-byte aligned, which the
// kernels' vector stores and the TMA store maps need.  The kernels then run
// on N8 = N rounded up to 8 channels: the weight tensor map keeps N rows
// (rows N .. N8-1 read as zeros), the channel scales are copied into a
// zero-padded [N8] array and the output goes to an [M, N8] scratch, whose
// first N columns a copy kernel writes into Y.  Both scratch arrays follow
// the codes in the workspace.
struct PadPlan {
    int64_t n8 = 0;
    size_t sw_off = 0, y_off = 0, total = 0;
};

PadPlan make_pad_plan(int64_t M, int64_t N, size_t start) {
    PadPlan p;
    p.n8 = N;
    p.total = start;
    if (N % 8 == 0) return p;
    p.n8 = (N + 7) / 8 * 8;
    p.sw_off = round_up(start, 256);
    p.y_off = round_up(p.sw_off + size_t(p.n8) * 4, 256);
    p.total = round_up(p.y_off + size_t(M) * size_t(p.n8) * 2, 256);
    return p;
}

__global__ void pad_scales_kernel(const float* __restrict__ s_w, int64_t N, float* __restrict__ sw8, int64_t N8) {
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < N8; i += int64_t(gridDim.x) * blockDim.x)
        sw8[i] = i < N ? s_w[i] : 0.0f;
}

__global__ void crop_rows_kernel(const uint16_t* __restrict__ Y8, int64_t N8, uint16_t* __restrict__ Y, int64_t M,
                                 int64_t N) {
    const int64_t n = M * N;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t m = i / N;
        Y[i] = Y8[m * N8 + (i - m * N)];
    }
}


// ------------------------------------------- decode: one-kernel Linear --

// Cluster size S (K split) of the one-kernel decode path: the largest power
// of two up to 8 that keeps tiles * S within 1.5 CTAs per SM (two fit on an
// SM; more CTAs keep more weight copies in flight), no more
// than the K blocks, and raised (up to 8) until the codes of one CTA's K
// range fit its code store.  Weight ring: what is left of the shared region.
// Returns false when no S fits (K too long for this path).
bool stream_geometry(int64_t M, int64_t N, int64_t K, int sm_count, stream::Geometry* g) {
    const int64_t tiles = (N + stream::TILE - 1) / stream::TILE;
    const int64_t kb = (K + stream::SUB - 1) / stream::SUB;
    const int mpad = M <= 8 ? 8 : 16;
    // The K split doubles while the grid stays within 1.5 CTAs per SM, and
    // on up to 2 per SM while every CTA keeps at least 8 K blocks (long-K
    // Linears such as down_proj, where more CTAs in flight stream faster).
    int S = 1;
    auto grow = [&](int s) {
        if (s >= stream::kMaxCluster || s * 2 > kb) return false;
        const int64_t ctas = tiles * s * 2;
        return ctas <= sm_count * 3 / 2 || (ctas <= int64_t(sm_count) * 2 && kb / (s * 2) >= 8);
    };
    while (grow(S)) S *= 2;
    auto code_bytes = [&](int s_) {
        const int64_t kbs = (kb + s_ - 1) / s_;
        return (kbs * mpad * stream::SUB + 1023) / 1024 * 1024;
    };
    while (code_bytes(S) > stream::kMaxCodeBytes && S < stream::kMaxCluster && S * 2 <= kb) S *= 2;
    if (code_bytes(S) > stream::kMaxCodeBytes) return false;
    g->S = S;
    g->mpad = mpad;
    g->code_bytes = int(code_bytes(S));
    const int st = (stream::kShared - g->code_bytes) / stream::kWStageBytes;
    g->stages = st > stream::kMaxStages ? stream::kMaxStages : st;
    // K blocks beyond the ring wait in TMEM (up to 7 per CTA).
    const int64_t spare = (kb + S - 1) / S - g->stages;
    g->tm_blocks = spare <= 0 ? 0 : int(spare < stream::kMaxTmemBlocks ? spare : stream::kMaxTmemBlocks);
    return g->stages >= stream::kMinStages;
}

mfp8_status launch_stream(const void* X, int64_t M, int64_t K, const void* W8, const float* s_w, int64_t N,
                          int64_t w_rows,
                          void* Y, bool weights_static, bool dependent, void* x8_out, float* sa_out, int dev,
                          const DeviceInfo& info, cudaStream_t stream) {
    if (M < 1 || M > kStreamMaxM || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    stream::Geometry g;
    if (!stream_geometry(M, N, K, info.sm_count, &g)) return MFP8_ERR_UNSUPPORTED_SHAPE;
    // Eight quantizer warps pay off once a CTA has more than 8 token rows.
    const bool wide = M > 8;
    auto kern = wide ? stream::gemm_stream_kernel<8> : stream::gemm_stream_kernel<4>;
    static bool attr_done4[kMaxDevices] = {}, attr_done8[kMaxDevices] = {};
    mfp8_status st = set_smem(kern, stream::Smem::BYTES, dev, wide ? attr_done8 : attr_done4);
    if (st != MFP8_OK) return st;
    const int64_t tiles = (N + stream::TILE - 1) / stream::TILE;
    const int64_t grid = tiles * g.S;
    if (grid > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    CUtensorMap tmW;
    if ((st = make_map_u8(&tmW, W8, w_rows, K, stream::TILE)) != MFP8_OK) return st;

    stream::Args args;
    args.X = static_cast<const __nv_bfloat16*>(X);
    args.s_w = s_w;
    args.Y = static_cast<__nv_bfloat16*>(Y);
    args.x8_out = static_cast<uint8_t*>(x8_out);
    args.sa_out = sa_out;
    args.M = int(M);
    args.N = int(N);
    args.K = int(K);
    args.weights_static = weights_static ? 1 : 0;
    args.g = g;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(wide ? stream::Warps<8>::kThreads : stream::Warps<4>::kThreads));
    cfg.dynamicSmemBytes = stream::Smem::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(g.S);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tmW, args) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

// ------------------------------ small / middle M: cluster split-K on codes --

// Cluster size S (K split) of the split-K path: the decode kernel's rule (up
// to 1.5 CTAs per SM, or 2 while each CTA keeps 8+ K blocks).  Ring: as many
// weight + code stages as fit.
bool cluster_geometry(int64_t M, int64_t N, int64_t K, int sm_count, cluster::Geometry* g) {
    if (M < 1 || M > cluster::kMaxM) return false;
    const int64_t tiles = (N + cluster::TILE - 1) / cluster::TILE;
    const int64_t kb = (K + cluster::SUB - 1) / cluster::SUB;
    int S = 1;
    auto grow = [&](int s) {
        if (s >= cluster::kMaxCluster || s * 2 > kb) return false;
        const int64_t ctas = tiles * s * 2;
        return ctas <= sm_count * 3 / 2 || (ctas <= int64_t(sm_count) * 2 && kb / (s * 2) >= 8);
    };
    while (grow(S)) S *= 2;
    g->S = S;
    g->mp = int((M + 15) / 16 * 16);
    // A grid of at most one CTA per SM takes the deeper ring (more bytes in
    // flight per CTA, fewer exchange rounds); larger grids keep two CTAs per
    // SM resident.
    g->ring = tiles * S <= sm_count ? cluster::kRingBig : cluster::kRingBytes;
    const int st = g->ring / cluster::stage_bytes(g->mp);
    g->stages = st > cluster::kMaxStages ? cluster::kMaxStages : st;
    // Exchange rounds: as few as the ring allows, of equal width (a multiple
    // of 32 token columns where the round is that wide, else of 16: whole
    // 32-column TMEM loads).
    g->tc = g->mp;
    if (S > 1) {
        int rounds = 1;
        auto width = [&](int r) {
            const int w = (g->mp + r - 1) / r;
            return w > 16 ? (w + 31) / 32 * 32 : 16;
        };
        while (cluster::exchange_bytes(S, width(rounds)) > g->ring) ++rounds;
        g->tc = width(rounds) < g->mp ? width(rounds) : g->mp;
    }
    return g->stages >= cluster::kMinStages;
}

mfp8_status launch_cluster(const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8, const float* s_w,
                           int64_t N, int64_t w_rows, void* Y, bool weights_static, bool dependent, int dev,
                           const DeviceInfo& info,
                           cudaStream_t stream) {
    cluster::Geometry g;
    if (!cluster_geometry(M, N, K, info.sm_count, &g)) return MFP8_ERR_UNSUPPORTED_SHAPE;
    auto kern = cluster::gemm_cluster_kernel;
    static bool attr_done[kMaxDevices] = {};
    mfp8_status st = set_smem(kern, cluster::Smem::MAX_BYTES, dev, attr_done);
    if (st != MFP8_OK) return st;
    const int64_t tiles = (N + cluster::TILE - 1) / cluster::TILE;
    const int64_t grid = tiles * g.S;
    if (grid > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    CUtensorMap tmX, tmW;
    if ((st = make_map_u8(&tmW, W8, w_rows, K, cluster::TILE)) != MFP8_OK) return st;
    if ((st = make_map_u8(&tmX, X8, M, K, g.mp)) != MFP8_OK) return st;

    cluster::Args args;
    args.s_a = s_a;
    args.s_w = s_w;
    args.Y = static_cast<__nv_bfloat16*>(Y);
    args.M = int(M);
    args.N = int(N);
    args.K = int(K);
    args.weights_static = weights_static ? 1 : 0;
    args.g = g;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(cluster::kThreads);
    cfg.dynamicSmemBytes = size_t(cluster::Smem::bytes(g.ring));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(g.S);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tmX, tmW, args) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

// The GEMM on codes already in memory (tiled, pair, or split-K).
mfp8_status run_gemm(const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8, const float* s_w,
                     int64_t N, int64_t w_rows, void* Y, int path, bool weights_static, bool dependent, int dev,
                     const DeviceInfo& info, cudaStream_t stream) {
    // The kernels take M, N, K as 32-bit.
    if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (path == MFP8_PATH_TILED) return launch_tiled(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
    if (path == MFP8_PATH_PAIR) return launch_pair(X8, s_a, M, K, W8, s_w, N, w_rows, Y, dependent, dev, info, stream);
    if (path == MFP8_PATH_SPLITK)
        return launch_cluster(X8, s_a, M, K, W8, s_w, N, w_rows, Y, weights_static, dependent, dev, info, stream);
    return MFP8_ERR_INVALID_ARG;
}

int sm_count_for_sizing() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && sms > 0)
        return sms;
    cudaGetLastError();
    return 148;  // B200
}

// Scratch of mfp8_linear_noalloc: one fixed array per device, part of the
// module's own global memory, so that entry point allocates nothing.  It is
// for callers that cannot call an allocator where they call the Linear: a C
// host with no device allocator of its own, or one whose memory is planned
// in full up front (a fixed budget per GPU).  Every call on a device uses
// the same bytes, so two calls that can be in flight at once race.
constexpr size_t kStaticWsBytes = MFP8_STATIC_WORKSPACE_BYTES;
static __device__ __align__(256) uint8_t g_static_ws[kStaticWsBytes];

// The array's device address, looked up once per device and context.  In
// host code `g_static_ws` names a host-side stand-in, not device memory; the
// address kernels need comes from cudaGetSymbolAddress with the device
// current.  It is cached together with the context's unique ID: a context
// that was destroyed and created again (cudaDeviceReset) reloads the module,
// which may place the array elsewhere, and the new ID forces a new lookup.
struct StaticWs {
    unsigned long long ctx_id = 0;
    void* ptr = nullptr;
};
StaticWs g_static_ws_cache[kMaxDevices];
PFN_cuCtxGetCurrent_v4000 g_ctx_get_current = nullptr;
PFN_cuCtxGetId_v12000 g_ctx_get_id = nullptr;

// Unique ID of the calling thread's current context (0 when none is bound).
mfp8_status current_context_id(unsigned long long* id) {
    if (!g_ctx_get_current || !g_ctx_get_id) {
        void* f1 = nullptr;
        void* f2 = nullptr;
        cudaDriverEntryPointQueryResult q1, q2;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &f1, cudaEnableDefault, &q1) != cudaSuccess ||
            cudaGetDriverEntryPoint("cuCtxGetId", &f2, cudaEnableDefault, &q2) != cudaSuccess ||
            q1 != cudaDriverEntryPointSuccess || q2 != cudaDriverEntryPointSuccess || !f1 || !f2) {
            cudaGetLastError();
            return MFP8_ERR_CUDA;
        }
        g_ctx_get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(f1);
        g_ctx_get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(f2);
    }
    CUcontext ctx = nullptr;
    if (g_ctx_get_current(&ctx) != CUDA_SUCCESS) return MFP8_ERR_CUDA;
    *id = 0;
    if (ctx && g_ctx_get_id(ctx, id) != CUDA_SUCCESS) return MFP8_ERR_CUDA;
    return MFP8_OK;
}

mfp8_status static_workspace(int dev, void** out) {
    std::lock_guard<std::mutex> lock(g_mu);
    unsigned long long id = 0;
    mfp8_status st = current_context_id(&id);
    if (st != MFP8_OK) return st;
    StaticWs& c = g_static_ws_cache[dev];
    if (id == 0 || c.ptr == nullptr || c.ctx_id != id) {
        // cudaGetSymbolAddress also binds the device's primary context to
        // this thread if none was bound yet; the ID is read after it.
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_static_ws) != cudaSuccess || p == nullptr) {
            cudaGetLastError();
            return MFP8_ERR_CUDA;
        }
        if ((st = current_context_id(&id)) != MFP8_OK) return st;
        c.ptr = p;
        c.ctx_id = id;
    }
    *out = c.ptr;
    return MFP8_OK;
}

__global__ void bounded_wait_kernel(uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_u32(&bar), 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // Nothing ever arrives on this barrier: the wait must give up.
        mbar_wait(smem_u32(&bar), 0, &abort_flag, limit_ns);
    }
}

// Launch of a fused producer kernel: one block per row, VPT vectors of 8
// values per thread (rows up to 16384 values), as a programmatic dependent.
template <template <int> class Pick, class... A>
mfp8_status launch_producer(int64_t nvec, int64_t M, cudaStream_t stream, A... args) {
    auto launch = [&](auto kern) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(M));
        cfg.blockDim = dim3(producer::kThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
            cudaGetLastError();
            return MFP8_ERR_CUDA;
        }
        return MFP8_OK;
    };
    if (nvec <= 256) return launch(Pick<1>::kern());
    if (nvec <= 512) return launch(Pick<2>::kern());
    if (nvec <= 1024) return launch(Pick<4>::kern());
    if (nvec <= 1536) return launch(Pick<6>::kern());
    if (nvec <= 2048) return launch(Pick<8>::kern());
    return MFP8_ERR_UNSUPPORTED_SHAPE;
}

// A launch that may begin while the previous kernel on the stream drains
// (programmatic dependent launch); the kernel waits for that kernel's
// results with griddepcontrol.wait before its first global load.
template <typename... KArgs, typename... A>
mfp8_status launch_pdl(void (*kern)(KArgs...), dim3 grid, int threads, cudaStream_t stream, int smem_bytes,
                       A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = size_t(smem_bytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return MFP8_OK;
}

template <int VPT>
struct PickRmsnorm {
    static auto kern() { return producer::rmsnorm_quant_kernel<producer::kThreads, VPT>; }
};
constexpr int64_t kSiluWideFrom = 1024;  // rows above this many 8-value vectors take 512 threads

template <int VPT>
struct PickSiluMul {
    static auto kern() { return producer::silu_mul_quant_kernel<producer::kThreads, VPT>; }
};

// ------------------------------------- rotary positions, paged cache --

// A strided run of T tokens' head rows, in bytes from its start.
size_t strided_bytes(int64_t T, int64_t ld, int64_t width, size_t elem) {
    return T == 0 ? 0 : (size_t(T - 1) * size_t(ld) + size_t(width)) * elem;
}

template <class P>
bool aligned_to(const P* p) {
    return (reinterpret_cast<uintptr_t>(p) & (alignof(P) - 1)) == 0;
}

// page_size -> its log2, or -1.
int page_shift(int64_t page_size) {
    for (int s = 3; s <= 8; ++s)
        if (page_size == int64_t(1) << s) return s;
    return -1;
}

bool page_shape_ok(int64_t n_pages, int64_t H, int64_t page_size, int64_t D) {
    return n_pages >= 0 && n_pages <= INT32_MAX && page_shift(page_size) > 0 &&
           (n_pages == 0 || H * page_size * D <= (int64_t(1) << 44) / n_pages);
}

mfp8_status check_rope_args(const int32_t* pos, int n_axes, const uint8_t* axis, const float* inv_freq, int64_t rot,
                            int64_t D, int layout, double mscale, int64_t T) {
    if (n_axes < 1 || n_axes > 4 || (layout != MFP8_ROPE_HALF && layout != MFP8_ROPE_INTERLEAVED) ||
        !std::isfinite(mscale))
        return MFP8_ERR_INVALID_ARG;
    if (D <= 0 || D % 16 != 0 || D > 256 || rot < 0 || rot % 16 != 0 || rot > D) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T > 0 && rot > 0) {
        if (!pos || !inv_freq || (n_axes > 1 && !axis)) return MFP8_ERR_INVALID_ARG;
        if (!aligned_to(pos) || !aligned_to(inv_freq)) return MFP8_ERR_MISALIGNED;
    }
    return MFP8_OK;
}

// Whether [out, out + n) overlaps the positions or tables of a rotation.
bool over_rope_inputs(const void* out, size_t n, const int32_t* pos, int n_axes, int64_t T, const uint8_t* axis,
                      const float* inv_freq, int64_t rot) {
    if (rot == 0) return false;
    return ranges_overlap(out, n, pos, size_t(n_axes) * size_t(T) * 4) ||
           ranges_overlap(out, n, inv_freq, size_t(rot / 2) * 4) ||
           (n_axes > 1 && ranges_overlap(out, n, axis, size_t(rot / 2)));
}

mfp8_status launch_rope(rope::Params p, int layout, cudaStream_t stream) {
    const int heads = p.nq + p.nk + p.nv;
    const int units = p.vpr / 2;
    const int upr = units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : 16;
    // Threads per token: enough for a vector pair each, but at least a
    // sixteenth of a block; all of a block while there are few tokens.
    int shift = 7;  // kThreads
    while (shift > 3 && (1 << (shift - 1)) >= upr && (1 << (shift - 1)) >= heads * upr &&
           int64_t(p.T) >= int64_t(148) * 8 * (rope::kThreads >> (shift - 1)))
        --shift;
    p.tpt_shift = shift;
    const int tpb = rope::kThreads >> shift;
    const dim3 grid(unsigned((p.T + tpb - 1) / tpb));
    const int smem = tpb * p.rot * int(sizeof(float));
    // Rows per thread and pass: three where that divides a thread's rows and
    // two does not (no pass with places to spare), else two.  Both ways, us for
    // two / three rows, rotation alone and fused store, 134 MB of head rows of
    // 128: 2 rows 41.6 / 44.0 and 54.0 / 57.6; 3 rows 42.8 / 41.4 and 50.3 /
    // 47.5; 4 rows 42.0 / 42.7 and 45.7 / 48.9; 5 rows 41.8 / 42.6 and 46.4 /
    // 46.2; 6 rows 42.3 / 43.2 and 44.2 / 43.7; 8 rows 42.8 / 44.1 and 44.7 /
    // 45.3 (heads of 256 the same).
    const int rows = (heads * upr + (1 << shift) - 1) >> shift;
    const bool three = rows % 3 == 0 && rows % 2 != 0;
    const bool il = layout == MFP8_ROPE_INTERLEAVED;
    auto run = [&](auto kern) { return launch_pdl(kern, grid, rope::kThreads, stream, smem, p); };
    auto pick = [&](auto u) {
        constexpr int U = decltype(u)::value;
        if (il) return three ? run(rope::rope_store_kernel<U, true, 3>) : run(rope::rope_store_kernel<U, true, 2>);
        return three ? run(rope::rope_store_kernel<U, false, 3>) : run(rope::rope_store_kernel<U, false, 2>);
    };
    switch (upr) {
        case 1: return pick(std::integral_constant<int, 1>());
        case 2: return pick(std::integral_constant<int, 2>());
        case 4: return pick(std::integral_constant<int, 4>());
        case 8: return pick(std::integral_constant<int, 8>());
        default: return pick(std::integral_constant<int, 16>());
    }
}

// ------------------------------------- attention over a shared prefix --

// How the work is cut: which kernel takes the prefix and the own tokens, the
// slots of partial outputs per row of each, and their row tiles (of 8 or 16
// rows, or of 256 for the tall kernel).
struct AttendPlan {
    bool wide_p = false, wide_o = false;
    int splits_p = 0, splits_o = 0;
    int64_t tiles_p = 0, tiles_o = 0;
    bool direct = false;
    int row_tile = 16;  // of the row kernel
    size_t lse_off = 0, total = 0;
};

constexpr int kAttendSms = 148;
// Blocks per SM that the row kernel's splits aim at.  Sequences x own tokens
// (8 KV heads of 128), us for 2, 4, 8, 16: 4 x 16384 42, 34, 43, 55; 16 x 16384
// 120, 111, 105, 109; 64 x 64 to 8192 124, 110, 106, 110; 64 x 4096 92, 104,
// 104, 108; 64 x 1024 32, 40, 43, 50; 256 x 128 to 4096 187 with one slot
// each (2 to 8), 201.  Sequences of one length want whole waves, uneven ones
// small pieces; every sequence gets the same number of pieces, whatever its length.
constexpr int kRowBlocks = 4;
constexpr int64_t kAttendMax = int64_t(1) << 20;

// Which kernel takes a part (the prefix, or the own tokens) of `rows` query
// rows per KV head, `units` KV heads (times sequences) and `len` tokens.  One
// 16-row tile is the row kernel's whatever its length (own tokens of 4
// sequences, 8 heads: 16384 tokens 42 us, tall 57).  With more rows the tall
// kernel reads the tokens once for all of them, but its start costs 10 us;
// both sides of the border, row kernel and tall kernel: 2048 prefix tokens,
// 64 rows 12 / 15 us, 128 rows 21 / 15; 8192, 16 rows 14 / 19, 32 rows 22 /
// 19; 65536, 128 rows 223 / 57; own tokens of 4 sequences, 512, 64 rows 12 /
// 15, 128 rows 21 / 16; 2048, 16 rows 12 / 19, 32 rows 21 / 20.
constexpr double kWideWork = 100000;  // 16-row tiles times tokens
// Row tiles of 8 where no part has more rows, or where the call is so short
// that their start (2 us less than of 16 rows) counts for more than reading
// the tokens twice; both sides, 16 and 8 rows per tile: 2048 prefix tokens, 32
// rows 10.5 / 8.7 us, 64 rows 12.3 / 14.0; 8192, 16 rows 14.5 / 16.0; own
// tokens of 4 sequences, 1024, 16 rows 11.4 / 9.1, 32 rows 12.6 / 14.7; 2048,
// 16 rows 12.4 / 14.9.
constexpr double kEightWork = 40000;  // 16-row tiles times tokens
bool attend_wide(int path, int64_t rows, int64_t units, int64_t len) {
    if (path != MFP8_ATTEND_AUTO) return path == MFP8_ATTEND_TALL;
    return rows > attend::kRows && double((rows + attend::kRows - 1) / attend::kRows * units) * double(len) >= kWideWork;
}

// Row kernel: slots for `units` (row tile, KV head) pairs over `len` tokens:
// enough blocks for four per SM, none with less than the smallest chunk.
int attend_splits(int64_t units, int64_t len) {
    int64_t s = (kAttendSms * kRowBlocks + units - 1) / units;
    const int64_t most = (len + attend::kMinChunk - 1) / attend::kMinChunk;
    if (s > most) s = most;
    return int(s < 1 ? 1 : s > 256 ? 256 : s);
}

// Tall kernel, one CTA per SM: the number of slots that ends first.  A wave of
// CTAs takes its tile steps and eight more (Q, the ends of the pipeline, the
// partial output: about 10 us); the row kernel's part of the call, `beside`
// bytes of cache, is read meanwhile by the SMs that the tall kernel leaves
// free, then by all; a slot's outputs are written and joined at 4 TB/s.  64
// sequences over 32768 shared tokens (8 units), slots and us: 12 86, 14 77, 16
// 78, 18 79; 256 over 8192 (32 units), 1 218, 2 228, 3 232, 4 237.  Elsewhere,
// the choice in brackets: 32 sequences with 500 own tokens over 65536, 9 99,
// 14 71, [18 73]; 128 over 16384, 4 99, 6 85, [8 92], 9 91; heads of 64, 64
// over 32768, 9 79, 14 61, [16 64]; 256 over 8192 without own tokens, 3 84,
// [4 80], 6 86; 3010 prompt tokens over 10007, [1 625], 2 688; one prompt of
// 8192, [1 672], 2 815; of 700, [1 26], 2 31.
int attend_wide_splits(int64_t units, int64_t rows, int64_t len, int64_t out_values, double beside) {
    constexpr double kStepUs = 1.2, kFree = 45e3, kFull = 5.4e6;  // bytes per us: one SM of a few, all
    const int64_t tiles = (len + attend::kTile - 1) / attend::kTile;
    const int64_t per_tile = rows > attend::kTile ? 2 : 1;
    int64_t best = 1;
    double best_us = 1e300;
    for (int64_t s = 1; s <= 64 && s <= tiles; ++s) {
        const int64_t waves = (units * s + kAttendSms - 1) / kAttendSms;
        const double tall = double(waves * ((tiles + s - 1) / s * per_tile + 8)) * kStepUs;
        const int64_t idle = waves == 1 ? kAttendSms - units * s : 0;
        const double rate = std::min(double(idle) * kFree, kFull);
        const double us = tall + std::max(0.0, beside - tall * rate) / kFull + double(s * out_values) * 8 / 4e6;
        if (us < best_us) best = s, best_us = us;
    }
    return int(best);
}

bool attend_shape_ok(int64_t T, int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix_len,
                     int64_t max_pages, int64_t page_size) {
    return T >= 0 && T <= kAttendMax && B >= 0 && B <= kAttendMax && max_q >= 1 && max_q <= kAttendMax && Hkv >= 1 &&
           Hq >= Hkv && Hq <= 65536 && Hq % Hkv == 0 && (D == 64 || D == 128) && page_shift(page_size) > 0 &&
           prefix_len >= 0 && prefix_len <= attend::kMaxTokens && max_pages >= 0 &&
           max_pages <= attend::kMaxTokens / page_size && T * Hq <= kMaxDim;
}

AttendPlan attend_plan(int64_t T, int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix_len,
                       int64_t max_pages, int64_t page_size, int path) {
    AttendPlan a;
    const int64_t G = Hq / Hkv, rows_p = T * G, rows_o = (max_q < T ? max_q : T) * G, len_o = max_pages * page_size;
    const bool own = max_pages > 0 || prefix_len == 0;
    a.wide_p = prefix_len > 0 && attend_wide(path, rows_p, Hkv, prefix_len);
    a.wide_o = max_pages > 0 && attend_wide(path, rows_o, Hkv * B, len_o);
    // The row kernel's work in 16-row tiles times tokens.
    auto work = [](int64_t rows, int64_t units, int64_t len) { return double((rows + 15) / 16 * units) * double(len); };
    const bool narrow_p = prefix_len > 0 && !a.wide_p, narrow_o = own && !a.wide_o;
    if ((!narrow_p || rows_p <= 8) && (!narrow_o || rows_o <= 8)) a.row_tile = 8;
    if ((narrow_p ? work(rows_p, Hkv, prefix_len) : 0.0) + (narrow_o ? work(rows_o, Hkv * B, len_o) : 0.0) <= kEightWork)
        a.row_tile = 8;
    const int64_t tile_p = a.wide_p ? attend::kWideRows : a.row_tile;
    const int64_t tile_o = a.wide_o ? attend::kWideRows : a.row_tile;
    if (prefix_len > 0) a.tiles_p = (rows_p + tile_p - 1) / tile_p;
    if (own) a.tiles_o = (rows_o + tile_o - 1) / tile_o;
    // What the row kernel reads; own tokens are taken to fill half of the table.
    const double bytes_p = a.wide_p ? 0.0 : double(a.tiles_p * Hkv) * double(prefix_len * 2 * (D + 4));
    const double bytes_o = a.wide_o ? 0.0 : double(a.tiles_o * Hkv * B) * double(len_o * (D + 4));
    if (prefix_len > 0)
        a.splits_p = a.wide_p ? attend_wide_splits(a.tiles_p * Hkv, rows_p, prefix_len, T * Hq * D, bytes_o)
                              : attend_splits(a.tiles_p * Hkv, prefix_len);
    if (own)
        a.splits_o = a.wide_o ? attend_wide_splits(a.tiles_o * Hkv * B, rows_o, len_o, T * Hq * D, bytes_p)
                              : attend_splits(a.tiles_o * Hkv * B, len_o);
    const int64_t slots = a.splits_p + a.splits_o;
    a.direct = slots == 1;
    if (!a.direct) {
        a.lse_off = size_t(slots) * size_t(T * Hq) * size_t(D) * 4;
        a.total = a.lse_off + (size_t(slots) * size_t(T * Hq) * 4 + 255) / 256 * 256;
    }
    return a;
}

// The codes of a paged cache tensor as rows of D bytes: a copy takes the
// rows of one head in one page, at most a tile of them, D-byte swizzle.
mfp8_status make_map_pages(CUtensorMap* map, const void* base, int64_t rows, int64_t D, int box_rows) {
    cuuint64_t dims[2] = {cuuint64_t(D), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(D)};
    cuuint32_t box[2] = {cuuint32_t(D), cuuint32_t(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MFP8_OK : MFP8_ERR_CUDA;
}

template <int D>
mfp8_status launch_attend(attend::Params p, const AttendPlan& plan, int dev, cudaStream_t stream) {
    using L8 = attend::RowsLayout<D, 8>;
    using L16 = attend::RowsLayout<D, 16>;
    using WL = attend::WideLayout<D>;
    static bool ready[kMaxDevices] = {};
    {
        std::lock_guard<std::mutex> lock(g_mu);
        if (!ready[dev]) {
            if (cudaFuncSetAttribute(attend::attend_rows_kernel<D, 8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     L8::SMEM) != cudaSuccess ||
                cudaFuncSetAttribute(attend::attend_rows_kernel<D, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     L16::SMEM) != cudaSuccess ||
                cudaFuncSetAttribute(attend::attend_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     WL::SMEM_BYTES) != cudaSuccess) {
                cudaGetLastError();
                return MFP8_ERR_CUDA;
            }
            ready[dev] = true;
        }
    }
    const int64_t units_p = plan.tiles_p * plan.splits_p * p.Hkv, units_o = plan.tiles_o * plan.splits_o * p.Hkv * p.B;
    const int64_t wide = (plan.wide_p ? units_p : 0) + (plan.wide_o ? units_o : 0);
    const int64_t narrow = units_p + units_o - wide;
    mfp8_status st = MFP8_OK;
    if (wide > 0) {
        const int ps = 1 << p.ps_shift;
        const int64_t rows = p.n_pages * p.Hkv * ps;
        CUtensorMap tmK, tmV;
        if ((st = make_map_pages(&tmK, p.K, rows, D, ps < attend::kTile ? ps : attend::kTile)) != MFP8_OK) return st;
        if ((st = make_map_pages(&tmV, p.V, rows, D, ps < attend::kTile ? ps : attend::kTile)) != MFP8_OK) return st;
        const attend::WideGrid wg{plan.wide_p ? int(plan.tiles_p) : 0, plan.wide_o ? int(plan.tiles_o) : 0};
        st = launch_pdl(attend::attend_wide_kernel<D>, dim3(unsigned(wide)), attend::kWideThreads, stream,
                        WL::SMEM_BYTES, p, wg, tmK, tmV);
        if (st != MFP8_OK) return st;
    }
    if (narrow > 0) {
        p.tiles_p = plan.wide_p ? 0 : int(plan.tiles_p);
        p.tiles_o = plan.wide_o ? 0 : int(plan.tiles_o);
        p.beside = wide > 0;
        const dim3 grid(unsigned(narrow + (wide > 0)));
        st = plan.row_tile == 8 ? launch_pdl(attend::attend_rows_kernel<D, 8>, grid, attend::kThreads, stream, L8::SMEM, p)
                           : launch_pdl(attend::attend_rows_kernel<D, 16>, grid, attend::kThreads, stream, L16::SMEM, p);
        if (st != MFP8_OK) return st;
    }
    if (p.direct) return MFP8_OK;
    const int64_t rows = int64_t(p.T) * p.Hq;
    return launch_pdl(attend::join_kernel<D>, dim3(unsigned((rows + 7) / 8)), 256, stream, 0, p);
}

// The padded run: scales padded, X quantized (unless FUSED), the kernels on
// N8 channels into the scratch, then the crop.  Every launch here is a plain
// stream-ordered launch, so the scratch scales are complete before any
// kernel reads them.
mfp8_status run_padded(const void* X_bf16, const void* X8, const float* s_a, int64_t M, int64_t K, const void* W8,
                       const float* s_w, int64_t N, void* Y, const PadPlan& pad, uint8_t* base, int path,
                       void* X_fp8_out, float* x_scale_out, int dev, const DeviceInfo& info, cudaStream_t stream) {
    float* sw8 = reinterpret_cast<float*>(base + pad.sw_off);
    void* y8 = base + pad.y_off;
    const int64_t cap = int64_t(info.sm_count) * 8;
    pad_scales_kernel<<<unsigned((pad.n8 + 255) / 256 < cap ? (pad.n8 + 255) / 256 : cap), 256, 0, stream>>>(
        s_w, N, sw8, pad.n8);
    mfp8_status st = launch_status();
    if (st != MFP8_OK) return st;
    if (path == MFP8_PATH_FUSED) {
        st = launch_stream(X_bf16, M, K, W8, sw8, pad.n8, N, y8, /*weights_static=*/false, /*dependent=*/false,
                           X_fp8_out, x_scale_out, dev, info, stream);
    } else {
        // the per-row quantizer without the early trigger: the same codes as
        // mfp8_quantize_act, launched in plain stream order
        if (X_bf16 && (st = quantize_weight_rows(X_bf16, M, K, const_cast<void*>(X8), const_cast<float*>(s_a),
                                                 stream)) != MFP8_OK)
            return st;
        st = run_gemm(X8, s_a, M, K, W8, sw8, pad.n8, N, y8, path, /*weights_static=*/false, /*dependent=*/false,
                      dev, info, stream);
    }
    if (st != MFP8_OK) return st;
    const int64_t nb = (M * N + 255) / 256;
    crop_rows_kernel<<<unsigned(nb < cap ? nb : cap), 256, 0, stream>>>(static_cast<const uint16_t*>(y8), pad.n8,
                                                                        static_cast<uint16_t*>(Y), M, N);
    return launch_status();
}

}  // namespace
}  // namespace mfp8

using namespace mfp8;

extern "C" {

mfp8_status mfp8_quantize_weight(const void* W_bf16, int64_t N, int64_t K, void* W_fp8, float* w_scale,
                                 void* stream) {
    mfp8_status st = check_quant_args(W_bf16, N, K, W_fp8, w_scale);
    if (st != MFP8_OK || N == 0) return st;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    return quantize_weight_rows(W_bf16, N, K, W_fp8, w_scale, static_cast<cudaStream_t>(stream));
}

mfp8_status mfp8_quantize_act(const void* X_bf16, int64_t M, int64_t K, void* X_fp8, float* x_scale,
                              void* stream) {
    mfp8_status st = check_quant_args(X_bf16, M, K, X_fp8, x_scale);
    if (st != MFP8_OK || M == 0) return st;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    return quantize_act_rows(X_bf16, M, K, X_fp8, x_scale, static_cast<cudaStream_t>(stream));
}

size_t mfp8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
    return make_pad_plan(M, N, make_plan(M, K, true).total).total;
}

mfp8_status mfp8_linear_ex(const void* X_bf16, int64_t M, int64_t K, const void* W_fp8, const float* w_scale,
                           int64_t N, void* Y_bf16, void* workspace, size_t workspace_bytes_given, int path,
                           int flags, void* X_fp8_out, float* x_scale_out, void* stream) {
    mfp8_status st = check_gemm_args(M, N, K, W_fp8, w_scale, Y_bf16);
    if (st != MFP8_OK) return st;
    if (path < MFP8_PATH_AUTO || path > MFP8_PATH_FUSED) return MFP8_ERR_INVALID_ARG;
    if ((flags & ~MFP8_FLAG_STATIC_WEIGHTS) != 0) return MFP8_ERR_INVALID_ARG;
    if (path == MFP8_PATH_SPLITK && M > kClusterMaxM) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (path == MFP8_PATH_FUSED && M > kStreamMaxM) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MFP8_OK;
    if (!X_bf16) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(X_bf16)) return MFP8_ERR_MISALIGNED;
    if ((X_fp8_out == nullptr) != (x_scale_out == nullptr)) return MFP8_ERR_INVALID_ARG;
    if (ranges_overlap(X_bf16, size_t(M * K * 2), Y_bf16, size_t(M * N * 2))) return MFP8_ERR_INVALID_ARG;
    if (X_fp8_out) {
        if (!aligned16(X_fp8_out) || !aligned16(x_scale_out)) return MFP8_ERR_MISALIGNED;
        if ((st = check_quant_args(X_bf16, M, K, X_fp8_out, x_scale_out)) != MFP8_OK) return st;
        if (ranges_overlap(X_fp8_out, size_t(M * K), Y_bf16, size_t(M * N * 2)) ||
            ranges_overlap(x_scale_out, size_t(M * 4), Y_bf16, size_t(M * N * 2)))
            return MFP8_ERR_INVALID_ARG;
    }
    if (path == MFP8_PATH_AUTO) path = choose_path(M, (N + 7) / 8 * 8, K);
    const bool weights_static = (flags & MFP8_FLAG_STATIC_WEIGHTS) != 0;
    // FUSED (M <= 16): one kernel quantizes X on chip and streams the
    // weights; it keeps nothing in the workspace.
    const bool fused = path == MFP8_PATH_FUSED;
    const Plan plan = fused ? Plan() : make_plan(M, K, X_fp8_out == nullptr);
    const PadPlan pad = make_pad_plan(M, N, plan.total);
    if (pad.total > 0) {
        if (!workspace || workspace_bytes_given < pad.total) return MFP8_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MFP8_ERR_MISALIGNED;
        if (ranges_overlap(workspace, pad.total, Y_bf16, size_t(M * N * 2)) ||
            ranges_overlap(workspace, pad.total, X_bf16, size_t(M * K * 2)) ||
            (X_fp8_out && (ranges_overlap(workspace, pad.total, X_fp8_out, size_t(M * K)) ||
                           ranges_overlap(workspace, pad.total, x_scale_out, size_t(M * 4)))))
            return MFP8_ERR_INVALID_ARG;
    }

    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    if (pad.n8 != N) {
        const void* X8 = fused ? nullptr : (X_fp8_out ? X_fp8_out : base + plan.x8_off);
        const float* s_a = fused ? nullptr : (x_scale_out ? x_scale_out : reinterpret_cast<float*>(base + plan.sa_off));
        return run_padded(X_bf16, X8, s_a, M, K, W_fp8, w_scale, N, Y_bf16, pad, base, path, X_fp8_out, x_scale_out,
                          dev, info, s);
    }
    if (fused)
        return launch_stream(X_bf16, M, K, W_fp8, w_scale, N, N, Y_bf16, weights_static, /*dependent=*/true,
                             X_fp8_out, x_scale_out, dev, info, s);
    void* X8 = X_fp8_out ? X_fp8_out : base + plan.x8_off;
    float* s_a = x_scale_out ? x_scale_out : reinterpret_cast<float*>(base + plan.sa_off);
    if ((st = quantize_act_rows(X_bf16, M, K, X8, s_a, s)) != MFP8_OK) return st;
    return run_gemm(X8, s_a, M, K, W_fp8, w_scale, N, N, Y_bf16, path, weights_static,
                    /*dependent=*/true, dev, info, s);
}

mfp8_status mfp8_linear(const void* X_bf16, int64_t M, int64_t K, const void* W_fp8, const float* w_scale,
                        int64_t N, void* Y_bf16, void* workspace, size_t workspace_bytes_given, void* stream) {
    return mfp8_linear_ex(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, workspace, workspace_bytes_given,
                          MFP8_PATH_AUTO, 0, nullptr, nullptr, stream);
}

mfp8_status mfp8_linear_noalloc(const void* X_bf16, int64_t M, int64_t K, const void* W_fp8, const float* w_scale,
                               int64_t N, void* Y_bf16, void* stream) {
    mfp8_status st = check_gemm_args(M, N, K, W_fp8, w_scale, Y_bf16);
    if (st != MFP8_OK || M == 0) return st;
    if (mfp8_linear_workspace_bytes(M, N, K) > kStaticWsBytes) return MFP8_ERR_WORKSPACE;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    void* ws = nullptr;
    if ((st = static_workspace(dev, &ws)) != MFP8_OK) return st;
    return mfp8_linear_ex(X_bf16, M, K, W_fp8, w_scale, N, Y_bf16, ws, kStaticWsBytes, MFP8_PATH_AUTO, 0,
                          nullptr, nullptr, stream);
}

int mfp8_choose_path(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return MFP8_PATH_AUTO;
    return choose_path(M, N, K);
}

size_t mfp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
    return make_pad_plan(M, N, 0).total;  // only N % 8 != 0 needs scratch
}

mfp8_status mfp8_gemm(const void* X_fp8, const float* x_scale, int64_t M, int64_t K, const void* W_fp8,
                      const float* w_scale, int64_t N, void* Y_bf16, void* workspace, size_t workspace_bytes_given,
                      int path, void* stream) {
    mfp8_status st = check_gemm_args(M, N, K, W_fp8, w_scale, Y_bf16);
    if (st != MFP8_OK) return st;
    if (path < MFP8_PATH_AUTO || path > MFP8_PATH_PAIR) return MFP8_ERR_INVALID_ARG;
    if (path == MFP8_PATH_SPLITK && M > kClusterMaxM) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MFP8_OK;
    if (!X_fp8 || !x_scale) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(X_fp8) || !aligned16(x_scale)) return MFP8_ERR_MISALIGNED;
    if (ranges_overlap(X_fp8, size_t(M * K), Y_bf16, size_t(M * N * 2)) ||
        ranges_overlap(x_scale, size_t(M * 4), Y_bf16, size_t(M * N * 2)))
        return MFP8_ERR_INVALID_ARG;
    const PadPlan pad = make_pad_plan(M, N, 0);
    if (path == MFP8_PATH_AUTO) path = choose_path(M, pad.n8, K);
    if (path == MFP8_PATH_FUSED) path = MFP8_PATH_SPLITK;  // codes given: the split-K kernel streams them
    if (pad.total > 0) {
        if (!workspace || workspace_bytes_given < pad.total) return MFP8_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MFP8_ERR_MISALIGNED;
        if (ranges_overlap(workspace, pad.total, Y_bf16, size_t(M * N * 2)) ||
            ranges_overlap(workspace, pad.total, X_fp8, size_t(M * K)) ||
            ranges_overlap(workspace, pad.total, x_scale, size_t(M * 4)))
            return MFP8_ERR_INVALID_ARG;
    }
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pad.n8 != N)
        return run_padded(nullptr, X_fp8, x_scale, M, K, W_fp8, w_scale, N, Y_bf16, pad,
                          static_cast<uint8_t*>(workspace), path, nullptr, nullptr, dev, info, s);
    return run_gemm(X_fp8, x_scale, M, K, W_fp8, w_scale, N, N, Y_bf16, path, /*weights_static=*/false,
                    /*dependent=*/false, dev, info, s);
}

mfp8_status mfp8_rmsnorm_quantize(const void* X_bf16, const void* gamma_bf16, float eps, int64_t M, int64_t K,
                                  void* Y_bf16, void* X_fp8, float* x_scale, void* stream) {
    mfp8_status st = check_quant_args(X_bf16, M, K, X_fp8, x_scale);
    if (st != MFP8_OK) return st;
    if (K > 16384) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (!(eps >= 0.0f) || eps > 1.0f) return MFP8_ERR_INVALID_ARG;
    if (M == 0) return MFP8_OK;
    if (!gamma_bf16) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(gamma_bf16) || !aligned16(Y_bf16)) return MFP8_ERR_MISALIGNED;
    if (Y_bf16 && (ranges_overlap(Y_bf16, size_t(M * K * 2), X_bf16, size_t(M * K * 2)) ||
                   ranges_overlap(Y_bf16, size_t(M * K * 2), X_fp8, size_t(M * K)) ||
                   ranges_overlap(Y_bf16, size_t(M * K * 2), x_scale, size_t(M * 4))))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    const int64_t nvec = K / 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint4* xv = static_cast<const uint4*>(X_bf16);
    const uint4* gv = static_cast<const uint4*>(gamma_bf16);
    uint4* yv = static_cast<uint4*>(Y_bf16);
    uint2* qv = static_cast<uint2*>(X_fp8);
    // Rows up to 4096 values: 128 threads per row.
    if (nvec <= 128)
        return launch_pdl(producer::rmsnorm_quant_kernel<128, 1>, dim3(unsigned(M)), 128, s, 0, xv, gv, K, eps, yv,
                          qv, x_scale);
    if (nvec <= 256)
        return launch_pdl(producer::rmsnorm_quant_kernel<128, 2>, dim3(unsigned(M)), 128, s, 0, xv, gv, K, eps, yv,
                          qv, x_scale);
    if (nvec <= 512)
        return launch_pdl(producer::rmsnorm_quant_kernel<128, 4>, dim3(unsigned(M)), 128, s, 0, xv, gv, K, eps, yv,
                          qv, x_scale);
    return launch_producer<PickRmsnorm>(nvec, M, s, xv, gv, K, eps, yv, qv, x_scale);
}

mfp8_status mfp8_silu_mul_quantize(const void* GU_bf16, int64_t M, int64_t I, void* Y_bf16, void* X_fp8,
                                   float* x_scale, void* stream) {
    if (M < 0 || I < 0) return MFP8_ERR_INVALID_ARG;
    if (I == 0 || I % 16 != 0 || I > 16384 || M > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MFP8_OK;
    if (!GU_bf16 || !X_fp8 || !x_scale) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(GU_bf16) || !aligned16(X_fp8) || !aligned16(x_scale) || !aligned16(Y_bf16))
        return MFP8_ERR_MISALIGNED;
    const size_t in_bytes = size_t(M) * size_t(2 * I) * 2;
    if (ranges_overlap(GU_bf16, in_bytes, X_fp8, size_t(M * I)) ||
        ranges_overlap(GU_bf16, in_bytes, x_scale, size_t(M * 4)) ||
        ranges_overlap(X_fp8, size_t(M * I), x_scale, size_t(M * 4)) ||
        (Y_bf16 && (ranges_overlap(Y_bf16, size_t(M * I * 2), GU_bf16, in_bytes) ||
                    ranges_overlap(Y_bf16, size_t(M * I * 2), X_fp8, size_t(M * I)) ||
                    ranges_overlap(Y_bf16, size_t(M * I * 2), x_scale, size_t(M * 4)))))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    const int64_t nvec = I / 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint4* gu = static_cast<const uint4*>(GU_bf16);
    uint4* yv = static_cast<uint4*>(Y_bf16);
    uint2* qv = static_cast<uint2*>(X_fp8);
    // Long rows: 512 threads per row (more warps resident per SM to hide the
    // loads behind the arithmetic).
    if (nvec > kSiluWideFrom && nvec <= 1536)
        return launch_pdl(producer::silu_mul_quant_kernel<512, 3>, dim3(unsigned(M)), 512, s, 0, gu, I, yv, qv, x_scale);
    if (nvec > kSiluWideFrom && nvec <= 2048)
        return launch_pdl(producer::silu_mul_quant_kernel<512, 4>, dim3(unsigned(M)), 512, s, 0, gu, I, yv, qv, x_scale);
    return launch_producer<PickSiluMul>(nvec, M, s, gu, I, yv, qv, x_scale);
}

mfp8_status mfp8_kv_quantize(const void* KV_bf16, int64_t T, int64_t H, int64_t D, void* KV_fp8, float* kv_scale,
                             void* stream) {
    if (T < 0 || H < 0 || D < 0) return MFP8_ERR_INVALID_ARG;
    if (H == 0 || D == 0 || D % 16 != 0 || D > kMaxDim || H > kMaxDim || T > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    const int64_t R = T * H;
    if (R > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    mfp8_status st = check_quant_args(KV_bf16, R, D, KV_fp8, kv_scale);
    if (st != MFP8_OK || R == 0) return st;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D > 256) return quantize_weight_rows(KV_bf16, R, D, KV_fp8, kv_scale, s);  // long rows: the row kernels
    const int vpr = int(D / 8);
    const int lpr = vpr <= 2 ? 2 : vpr <= 4 ? 4 : vpr <= 8 ? 8 : vpr <= 16 ? 16 : 32;
    const int64_t rows_per_block = int64_t(kQuantThreads / 32) * (32 / lpr) * kSmallRowItems;
    const int64_t blocks = (R + rows_per_block - 1) / rows_per_block;
    if (blocks > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    const uint4* x = static_cast<const uint4*>(KV_bf16);
    uint2* q = static_cast<uint2*>(KV_fp8);
    const dim3 grid{static_cast<unsigned>(blocks)};
    switch (lpr) {
        case 2: return launch_pdl(quant_small_rows_kernel<2>, grid, kQuantThreads, s, 0, x, R, int(D), q, kv_scale);
        case 4: return launch_pdl(quant_small_rows_kernel<4>, grid, kQuantThreads, s, 0, x, R, int(D), q, kv_scale);
        case 8: return launch_pdl(quant_small_rows_kernel<8>, grid, kQuantThreads, s, 0, x, R, int(D), q, kv_scale);
        case 16: return launch_pdl(quant_small_rows_kernel<16>, grid, kQuantThreads, s, 0, x, R, int(D), q, kv_scale);
        default: return launch_pdl(quant_small_rows_kernel<32>, grid, kQuantThreads, s, 0, x, R, int(D), q, kv_scale);
    }
}

mfp8_status mfp8_kv_dequantize(const void* KV_fp8, const float* kv_scale, int64_t T, int64_t H, int64_t D,
                               void* KV_bf16, void* stream) {
    if (T < 0 || H < 0 || D < 0) return MFP8_ERR_INVALID_ARG;
    if (H == 0 || D == 0 || D % 16 != 0 || D > kMaxDim || H > kMaxDim || T > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    const int64_t R = T * H;
    if (R > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (R == 0) return MFP8_OK;
    if (!KV_fp8 || !kv_scale || !KV_bf16) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(KV_fp8) || !aligned16(kv_scale) || !aligned16(KV_bf16)) return MFP8_ERR_MISALIGNED;
    if (ranges_overlap(KV_bf16, size_t(R * D * 2), KV_fp8, size_t(R * D)) ||
        ranges_overlap(KV_bf16, size_t(R * D * 2), kv_scale, size_t(R * 4)))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    const int64_t n8 = R * D / 8;
    const int64_t blocks = (n8 + kQuantThreads * kDequantItems - 1) / (kQuantThreads * kDequantItems);
    if (blocks > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    return launch_pdl(kv_dequant_kernel, dim3(unsigned(blocks)), kQuantThreads, static_cast<cudaStream_t>(stream), 0,
                      static_cast<const uint2*>(KV_fp8), kv_scale, n8, int(D), static_cast<uint4*>(KV_bf16));
}

mfp8_status mfp8_kv8_quantize(const void* KV_bf16, int64_t T, int64_t H, int64_t D, void* KV_u8, float* kv_scale,
                              float* kv_zero, void* stream) {
    if (T < 0 || H < 0 || D < 0) return MFP8_ERR_INVALID_ARG;
    if (H == 0 || D == 0 || D % 16 != 0 || T % kv8::kGroup != 0 || D > kMaxDim || H > kMaxDim || T > kMaxDim)
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    const int64_t C = H * D;
    if (C > kMaxDim || (T > 0 && C > (int64_t(1) << 40) / T)) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MFP8_OK;
    if (!KV_bf16 || !KV_u8 || !kv_scale || !kv_zero) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(KV_bf16) || !aligned16(KV_u8) || !aligned16(kv_scale) || !aligned16(kv_zero))
        return MFP8_ERR_MISALIGNED;
    const int64_t G = T / kv8::kGroup;
    const size_t nin = size_t(T * C) * 2, nq = size_t(T * C), nf = size_t(G * C) * 4;
    if (ranges_overlap(KV_bf16, nin, KV_u8, nq) || ranges_overlap(KV_bf16, nin, kv_scale, nf) ||
        ranges_overlap(KV_bf16, nin, kv_zero, nf) || ranges_overlap(KV_u8, nq, kv_scale, nf) ||
        ranges_overlap(KV_u8, nq, kv_zero, nf) || ranges_overlap(kv_scale, nf, kv_zero, nf))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    const int64_t tiles_per_group = (C + kv8::kTileCols - 1) / kv8::kTileCols;
    const int64_t blocks = G * tiles_per_group;
    if (blocks > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    return launch_pdl(kv8::quant_kernel, dim3(unsigned(blocks)), kv8::kQuantThreads, static_cast<cudaStream_t>(stream), 0,
                      static_cast<const uint4*>(KV_bf16), C / 8, tiles_per_group, static_cast<uint2*>(KV_u8), kv_scale,
                      kv_zero);
}

mfp8_status mfp8_kv8_read(const void* KV_u8, const float* kv_scale, const float* kv_zero, int64_t Tq,
                          const void* tail_bf16, int64_t Tr, int64_t H, int64_t D, void* out_bf16, void* stream) {
    if (Tq < 0 || Tr < 0 || H < 0 || D < 0) return MFP8_ERR_INVALID_ARG;
    if (H == 0 || D == 0 || D % 16 != 0 || Tq % kv8::kGroup != 0 || D > kMaxDim || H > kMaxDim || Tq > kMaxDim ||
        Tr > kMaxDim)
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    const int64_t C = H * D, T = Tq + Tr;
    if (C > kMaxDim || (T > 0 && C > (int64_t(1) << 40) / T)) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MFP8_OK;
    if (!out_bf16 || (Tq > 0 && (!KV_u8 || !kv_scale || !kv_zero)) || (Tr > 0 && !tail_bf16))
        return MFP8_ERR_INVALID_ARG;
    if (!aligned16(out_bf16) || !aligned16(KV_u8) || !aligned16(kv_scale) || !aligned16(kv_zero) ||
        !aligned16(tail_bf16))
        return MFP8_ERR_MISALIGNED;
    const size_t nout = size_t(T * C) * 2, nq = size_t(Tq * C), nf = size_t(Tq / kv8::kGroup * C) * 4,
                 nt = size_t(Tr * C) * 2;
    if ((Tq > 0 && (ranges_overlap(out_bf16, nout, KV_u8, nq) || ranges_overlap(out_bf16, nout, kv_scale, nf) ||
                    ranges_overlap(out_bf16, nout, kv_zero, nf))) ||
        (Tr > 0 && ranges_overlap(out_bf16, nout, tail_bf16, nt)))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    const int64_t C8 = C / 8, n_tail16 = Tr * C / 8;
    const int64_t items = Tq / kv8::kReadRows * C8 + n_tail16;
    const int64_t blocks = (items + kv8::kReadThreads - 1) / kv8::kReadThreads;
    if (blocks > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    return launch_pdl(kv8::read_kernel, dim3(unsigned(blocks)), kv8::kReadThreads, static_cast<cudaStream_t>(stream), 0,
                      static_cast<const uint2*>(KV_u8), reinterpret_cast<const float4*>(kv_scale),
                      reinterpret_cast<const float4*>(kv_zero), Tq, C8, static_cast<const uint4*>(tail_bf16),
                      n_tail16, static_cast<uint4*>(out_bf16));
}

int64_t mfp8_kv8_history_tokens(int64_t T) {
    if (T < 0) return -1;
    return T < 128 ? 0 : kv8::kGroup * ((T - 128) / kv8::kGroup);
}

mfp8_status mfp8_rope_frequencies(int64_t rot, double theta, int scaling, double factor, int64_t trained_len,
                                  double beta_fast, double beta_slow, float* inv_freq_host, double* mscale_host) {
    if (rot <= 0 || rot % 16 != 0 || rot > 256) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (!inv_freq_host || scaling < MFP8_ROPE_SCALE_NONE || scaling > MFP8_ROPE_SCALE_YARN || !std::isfinite(theta) ||
        !(theta > 1.0) || (scaling != MFP8_ROPE_SCALE_NONE && (!std::isfinite(factor) || !(factor >= 1.0))))
        return MFP8_ERR_INVALID_ARG;
    const bool yarn = scaling == MFP8_ROPE_SCALE_YARN;
    if (yarn && (trained_len < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) || !(beta_fast > beta_slow)))
        return MFP8_ERR_INVALID_ARG;
    const double n = double(rot);
    if (scaling == MFP8_ROPE_SCALE_NTK) theta *= std::pow(factor, n / (n - 2.0));
    double low = 0.0, high = 0.0;
    if (yarn) {
        // the pair that turns `beta` times within the trained length:
        // trained_len theta^(-2i/rot) = 2 pi beta
        auto pair = [&](double beta) {
            return n * std::log(double(trained_len) / (beta * 6.283185307179586)) / (2.0 * std::log(theta));
        };
        low = std::fmax(std::floor(pair(beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair(beta_slow)), n - 1.0);
        if (high <= low) high = low + 0.001;  // the ramp has some width
    }
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(theta, -2.0 * double(i) / n);
        if (scaling == MFP8_ROPE_SCALE_LINEAR) f /= factor;
        if (yarn) {
            const double ramp = std::fmin(std::fmax((double(i) - low) / (high - low), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        inv_freq_host[i] = float(f);
    }
    if (mscale_host) *mscale_host = yarn ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return MFP8_OK;
}

mfp8_status mfp8_rope(const void* X_bf16, int64_t ldx, int64_t T, int64_t H, int64_t D, const int32_t* pos, int n_axes,
                      const uint8_t* axis, const float* inv_freq, int64_t rot, int layout, double mscale, void* Y_bf16,
                      int64_t ldy, void* stream) {
    if (T < 0 || H < 0 || D < 0 || ldx < 0 || ldy < 0) return MFP8_ERR_INVALID_ARG;
    mfp8_status st = check_rope_args(pos, n_axes, axis, inv_freq, rot, D, layout, mscale, T);
    if (st != MFP8_OK) return st;
    if (H == 0 || H > 65536 || T > kMaxDim || T * H > kMaxDim) return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (ldx < H * D || ldy < H * D || ldx % 8 != 0 || ldy % 8 != 0 || ldx > kMaxDim || ldy > kMaxDim)
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MFP8_OK;
    if (!X_bf16 || !Y_bf16) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(X_bf16) || !aligned16(Y_bf16)) return MFP8_ERR_MISALIGNED;
    const bool in_place = X_bf16 == Y_bf16 && ldx == ldy;
    if (!in_place && ranges_overlap(X_bf16, strided_bytes(T, ldx, H * D, 2), Y_bf16, strided_bytes(T, ldy, H * D, 2)))
        return MFP8_ERR_INVALID_ARG;
    if (over_rope_inputs(Y_bf16, strided_bytes(T, ldy, H * D, 2), pos, n_axes, T, axis, inv_freq, rot))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    rope::Params p = {};
    p.X = static_cast<const uint4*>(X_bf16);
    p.ldx = ldx / 8;
    p.pos = pos;
    p.axis = n_axes > 1 ? axis : nullptr;
    p.inv_freq = inv_freq;
    p.n_axes = n_axes;
    p.rot = int(rot);
    p.mscale = mscale;
    p.T = int(T);
    p.nq = int(H);
    p.vpr = int(D / 8);
    p.Y = static_cast<uint4*>(Y_bf16);
    p.ldy = ldy / 8;
    return launch_rope(p, layout, static_cast<cudaStream_t>(stream));
}

mfp8_status mfp8_kv_page_store(const void* KV_bf16, int64_t ldkv, const int64_t* slot, int64_t T, int64_t H, int64_t D,
                               void* pages, float* scale, int64_t n_pages, int64_t page_size, void* stream) {
    if (T < 0 || H < 0 || D < 0 || ldkv < 0 || n_pages < 0) return MFP8_ERR_INVALID_ARG;
    if (H == 0 || H > 65536 || D == 0 || D % 16 != 0 || D > 256 || T > kMaxDim || T * H > kMaxDim || ldkv < H * D ||
        ldkv % 8 != 0 || ldkv > kMaxDim || !page_shape_ok(n_pages, H, page_size, D))
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MFP8_OK;
    if (!KV_bf16 || !slot || (n_pages > 0 && (!pages || !scale))) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(KV_bf16) || !aligned16(pages) || !aligned16(scale) || !aligned_to(slot)) return MFP8_ERR_MISALIGNED;
    const size_t in = strided_bytes(T, ldkv, H * D, 2), rows = size_t(n_pages) * size_t(H * page_size);
    if (ranges_overlap(KV_bf16, in, pages, rows * size_t(D)) || ranges_overlap(KV_bf16, in, scale, rows * 4) ||
        ranges_overlap(pages, rows * size_t(D), scale, rows * 4) ||
        ranges_overlap(slot, size_t(T) * 8, pages, rows * size_t(D)) || ranges_overlap(slot, size_t(T) * 8, scale, rows * 4))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    rope::Params p = {};
    p.X = static_cast<const uint4*>(KV_bf16);
    p.ldx = ldkv / 8;
    p.n_axes = 1;
    p.T = int(T);
    p.nv = int(H);
    p.vpr = int(D / 8);
    p.slot = slot;
    p.n_slots = n_pages * page_size;
    p.ps_shift = page_shift(page_size);
    p.V = static_cast<uint2*>(pages);
    p.v_scale = scale;
    return launch_rope(p, MFP8_ROPE_HALF, static_cast<cudaStream_t>(stream));
}

mfp8_status mfp8_kv_page_read(const void* pages, const float* scale, int64_t n_pages, int64_t page_size,
                              const int64_t* slot, int64_t T, int64_t H, int64_t D, void* out_bf16, void* stream) {
    if (T < 0 || H < 0 || D < 0 || n_pages < 0) return MFP8_ERR_INVALID_ARG;
    if (H == 0 || H > 65536 || D == 0 || D % 16 != 0 || D > 256 || T > kMaxDim || T * H > kMaxDim ||
        !page_shape_ok(n_pages, H, page_size, D))
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MFP8_OK;
    if (!out_bf16 || !slot || (n_pages > 0 && (!pages || !scale))) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(out_bf16) || !aligned16(pages) || !aligned16(scale) || !aligned_to(slot)) return MFP8_ERR_MISALIGNED;
    const size_t nout = size_t(T * H * D) * 2, rows = size_t(n_pages) * size_t(H * page_size);
    if (ranges_overlap(out_bf16, nout, pages, rows * size_t(D)) || ranges_overlap(out_bf16, nout, scale, rows * 4) ||
        ranges_overlap(out_bf16, nout, slot, size_t(T) * 8))
        return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    const int vpr = int(D / 8);
    const int lpr = vpr <= 2 ? 2 : vpr <= 4 ? 4 : vpr <= 8 ? 8 : vpr <= 16 ? 16 : 32;
    const int64_t R = T * H, per_block = int64_t(rope::kReadThreads / lpr) * rope::kReadItems;
    const dim3 grid(unsigned((R + per_block - 1) / per_block));
    auto run = [&](auto kern) {
        return launch_pdl(kern, grid, rope::kReadThreads, static_cast<cudaStream_t>(stream), 0,
                          static_cast<const uint2*>(pages), scale, slot, n_pages * page_size, page_shift(page_size),
                          int(R), int(H), vpr, static_cast<uint4*>(out_bf16));
    };
    switch (lpr) {
        case 2: return run(rope::page_read_kernel<2>);
        case 4: return run(rope::page_read_kernel<4>);
        case 8: return run(rope::page_read_kernel<8>);
        case 16: return run(rope::page_read_kernel<16>);
        default: return run(rope::page_read_kernel<32>);
    }
}

mfp8_status mfp8_rope_kv_store(const void* QKV_bf16, int64_t ldqkv, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                               const int32_t* pos, int n_axes, const uint8_t* axis, const float* inv_freq, int64_t rot,
                               int layout, double mscale, const int64_t* slot, void* Q_bf16, void* k_pages,
                               float* k_scale, void* v_pages, float* v_scale, int64_t n_pages, int64_t page_size,
                               void* stream) {
    if (T < 0 || Hq < 0 || Hkv < 0 || D < 0 || ldqkv < 0 || n_pages < 0) return MFP8_ERR_INVALID_ARG;
    mfp8_status st = check_rope_args(pos, n_axes, axis, inv_freq, rot, D, layout, mscale, T);
    if (st != MFP8_OK) return st;
    if (Hq > 65536 || Hkv > 65536) return MFP8_ERR_UNSUPPORTED_SHAPE;
    const int64_t H = Hq + 2 * Hkv;
    if (Hq == 0 || Hkv == 0 || T > kMaxDim || T * H > kMaxDim || ldqkv < H * D || ldqkv % 8 != 0 || ldqkv > kMaxDim ||
        !page_shape_ok(n_pages, Hkv, page_size, D))
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MFP8_OK;
    if (!QKV_bf16 || !Q_bf16 || !slot || (n_pages > 0 && (!k_pages || !k_scale || !v_pages || !v_scale)))
        return MFP8_ERR_INVALID_ARG;
    if (!aligned16(QKV_bf16) || !aligned16(Q_bf16) || !aligned16(k_pages) || !aligned16(k_scale) ||
        !aligned16(v_pages) || !aligned16(v_scale) || !aligned_to(slot))
        return MFP8_ERR_MISALIGNED;
    const size_t in = strided_bytes(T, ldqkv, H * D, 2), rows = size_t(n_pages) * size_t(Hkv * page_size);
    const void* const buf[7] = {QKV_bf16, slot, Q_bf16, k_pages, k_scale, v_pages, v_scale};
    const size_t len[7] = {in, size_t(T) * 8, size_t(T * Hq * D) * 2, rows * size_t(D), rows * 4, rows * size_t(D), rows * 4};
    for (int i = 0; i < 7; ++i)
        for (int j = i + 1 > 2 ? i + 1 : 2; j < 7; ++j)
            if (ranges_overlap(buf[i], len[i], buf[j], len[j])) return MFP8_ERR_INVALID_ARG;
    for (int j = 2; j < 7; ++j)
        if (over_rope_inputs(buf[j], len[j], pos, n_axes, T, axis, inv_freq, rot)) return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    if ((st = current_device(&dev, &info)) != MFP8_OK) return st;
    rope::Params p = {};
    p.X = static_cast<const uint4*>(QKV_bf16);
    p.ldx = ldqkv / 8;
    p.pos = pos;
    p.axis = n_axes > 1 ? axis : nullptr;
    p.inv_freq = inv_freq;
    p.n_axes = n_axes;
    p.rot = int(rot);
    p.mscale = mscale;
    p.T = int(T);
    p.nq = int(Hq);
    p.nk = p.nv = int(Hkv);
    p.vpr = int(D / 8);
    p.Y = static_cast<uint4*>(Q_bf16);
    p.ldy = Hq * D / 8;
    p.slot = slot;
    p.n_slots = n_pages * page_size;
    p.ps_shift = page_shift(page_size);
    p.K = static_cast<uint2*>(k_pages);
    p.k_scale = k_scale;
    p.V = static_cast<uint2*>(v_pages);
    p.v_scale = v_scale;
    return launch_rope(p, layout, static_cast<cudaStream_t>(stream));
}

size_t mfp8_prefix_attention_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D,
                                             int64_t prefix_len, int64_t max_pages, int64_t page_size) {
    if (!attend_shape_ok(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, page_size) || T == 0 || B == 0) return 0;
    size_t most = 0;
    for (int path = MFP8_ATTEND_AUTO; path <= MFP8_ATTEND_TALL; ++path) {
        const size_t n = attend_plan(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, page_size, path).total;
        if (n > most) most = n;
    }
    return most;
}

mfp8_status mfp8_prefix_attention(const void* Q_bf16, int64_t ldq, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                  const int32_t* q_start, const int32_t* kv_len, int64_t B, int64_t max_q,
                                  const void* k_pages, const float* k_scale, const void* v_pages, const float* v_scale,
                                  int64_t n_pages, int64_t page_size, const int32_t* prefix_pages, int64_t prefix_len,
                                  const int32_t* page_table, int64_t ld_table, int64_t max_pages, float softmax_scale,
                                  void* O_bf16, float* lse, void* workspace, size_t workspace_bytes_given, int path,
                                  void* stream) {
    if (path < MFP8_ATTEND_AUTO || path > MFP8_ATTEND_TALL) return MFP8_ERR_INVALID_ARG;
    if (T < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0 || ldq < 0 || max_q < 0 || n_pages < 0 || prefix_len < 0 ||
        max_pages < 0 || ld_table < 0 || !std::isfinite(softmax_scale * 1.4426950408889634f) || !(softmax_scale > 0.0f))
        return MFP8_ERR_INVALID_ARG;
    if (!attend_shape_ok(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, page_size) ||
        !page_shape_ok(n_pages, Hkv, page_size, D) || ldq < Hq * D || ldq % 8 != 0 || ldq > kMaxDim ||
        ld_table < max_pages || ld_table > kMaxDim)
        return MFP8_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || B == 0) return MFP8_OK;
    const bool cached = prefix_len > 0 || max_pages > 0;
    if (!Q_bf16 || !O_bf16 || !q_start || !kv_len || (prefix_len > 0 && !prefix_pages) ||
        (max_pages > 0 && !page_table) ||
        (cached && (n_pages == 0 || !k_pages || !k_scale || !v_pages || !v_scale)))
        return MFP8_ERR_INVALID_ARG;
    if (!aligned16(Q_bf16) || !aligned16(O_bf16) || !aligned16(k_pages) || !aligned16(k_scale) || !aligned16(v_pages) ||
        !aligned16(v_scale) || !aligned_to(q_start) || !aligned_to(kv_len) || !aligned_to(prefix_pages) ||
        !aligned_to(page_table) || !aligned_to(lse))
        return MFP8_ERR_MISALIGNED;
    const AttendPlan plan = attend_plan(T, B, max_q, Hq, Hkv, D, prefix_len, max_pages, page_size, path);
    const size_t rows = size_t(n_pages) * size_t(Hkv * page_size);
    // inputs, then what is written
    const void* const buf[12] = {Q_bf16, k_pages, k_scale, v_pages, v_scale, q_start, kv_len, page_table, prefix_pages,
                                 O_bf16, lse, workspace};
    const size_t len[12] = {strided_bytes(T, ldq, Hq * D, 2), rows * size_t(D), rows * 4, rows * size_t(D), rows * 4,
                            size_t(B + 1) * 4, size_t(B) * 4, strided_bytes(B, ld_table, max_pages, 4),
                            size_t((prefix_len + page_size - 1) / page_size) * 4,
                            size_t(T * Hq * D) * 2, lse ? size_t(T * Hq) * 4 : 0, plan.total};
    if (plan.total > 0) {
        if (!workspace || workspace_bytes_given < plan.total) return MFP8_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MFP8_ERR_MISALIGNED;
    }
    for (int j = 9; j < 12; ++j)
        for (int i = 0; i < j; ++i)
            if (len[i] && len[j] && ranges_overlap(buf[i], len[i], buf[j], len[j])) return MFP8_ERR_INVALID_ARG;
    const int64_t np = plan.tiles_p * plan.splits_p * Hkv, no = plan.tiles_o * plan.splits_o * Hkv * B;
    if (np + no >= INT32_MAX || int64_t(rows) > INT32_MAX) return MFP8_ERR_UNSUPPORTED_SHAPE;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    attend::Params p = {};
    p.Q = static_cast<const __nv_bfloat16*>(Q_bf16);
    p.ldq = ldq;
    p.q_start = q_start;
    p.B = int(B);
    p.T = int(T);
    p.Hq = int(Hq);
    p.Hkv = int(Hkv);
    p.G = int(Hq / Hkv);
    p.K = static_cast<const uint8_t*>(k_pages);
    p.k_scale = k_scale;
    p.V = static_cast<const uint8_t*>(v_pages);
    p.v_scale = v_scale;
    p.n_pages = n_pages;
    p.ps_shift = page_shift(page_size);
    p.prefix_pages = prefix_pages;
    p.prefix_len = int(prefix_len);
    p.table = page_table;
    p.ld_table = ld_table;
    p.max_pages = int(max_pages);
    p.kv_len = kv_len;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    p.O = static_cast<__nv_bfloat16*>(O_bf16);
    p.lse = lse;
    p.part = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.lse_off);
    p.splits_p = plan.splits_p;
    p.splits_o = plan.splits_o;
    p.max_q = int(max_q);
    p.direct = plan.direct;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return D == 128 ? launch_attend<128>(p, plan, dev, s) : launch_attend<64>(p, plan, dev, s);
}

mfp8_status mfp8_debug_kv8_code_check(void* out_u64x2, int64_t n_scale_pairs, uint32_t seed, void* stream) {
    if (!out_u64x2 || n_scale_pairs <= 0 || n_scale_pairs > INT32_MAX) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(out_u64x2)) return MFP8_ERR_MISALIGNED;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(out_u64x2, 0, 16, s) != cudaSuccess) return MFP8_ERR_CUDA;
    kv8::code_check_kernel<<<unsigned(n_scale_pairs), 256, 0, s>>>(static_cast<unsigned long long*>(out_u64x2), seed);
    return launch_status();
}

mfp8_status mfp8_e4m3_encode_f32(const float* in, int64_t n, uint8_t* out, void* stream) {
    if (n < 0) return MFP8_ERR_INVALID_ARG;
    if (n == 0) return MFP8_OK;
    if (!in || !out) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(in) || !aligned16(out)) return MFP8_ERR_MISALIGNED;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    const int64_t pairs = (n + 1) / 2;
    int64_t blocks = (pairs + 255) / 256;
    const int64_t cap = int64_t(info.sm_count) * 16;
    if (blocks > cap) blocks = cap;
    e4m3_encode_kernel<<<unsigned(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(in, n, out);
    return launch_status();
}

mfp8_status mfp8_debug_quantize_check(void* out_u64x2, void* stream) {
    if (!out_u64x2) return MFP8_ERR_INVALID_ARG;
    if (!aligned16(out_u64x2)) return MFP8_ERR_MISALIGNED;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(out_u64x2, 0, 16, s) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    quantize_check_kernel<<<0x7f80u, 256, 0, s>>>(static_cast<unsigned long long*>(out_u64x2));
    return launch_status();
}

mfp8_status mfp8_debug_bounded_wait(int64_t timeout_us, void* stream) {
    if (timeout_us < 1 || timeout_us > 100000) return MFP8_ERR_INVALID_ARG;
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    bounded_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(uint64_t(timeout_us) * 1000u);
    return launch_status();
}

mfp8_status mfp8_get_device_status(void* stream) {
    int dev;
    DeviceInfo info;
    mfp8_status st = current_device(&dev, &info);
    if (st != MFP8_OK) return st;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    int word = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&word, g_device_status, sizeof(int)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return MFP8_ERR_CUDA;
    }
    return static_cast<mfp8_status>(word);
}

const char* mfp8_status_string(mfp8_status status) {
    switch (status) {
        case MFP8_OK: return "ok";
        case MFP8_ERR_INVALID_ARG: return "invalid argument";
        case MFP8_ERR_MISALIGNED: return "pointer not 16-byte aligned";
        case MFP8_ERR_UNSUPPORTED_SHAPE: return "unsupported shape (K must be a positive multiple of 16, N of 8)";
        case MFP8_ERR_WORKSPACE: return "workspace missing or too small";
        case MFP8_ERR_CUDA: return "CUDA runtime error";
        case MFP8_ERR_TIMEOUT: return "a kernel's bounded wait ran out";
        case MFP8_ERR_DEVICE: return "device is not compute capability 10.0 (B200)";
        case MFP8_ERR_INDEX: return "a slot, page or length in device memory is out of range";
    }
    return "unknown status";
}

int mfp8_version(void) { return 200; }

}  // extern "C"
