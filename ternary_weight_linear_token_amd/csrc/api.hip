// api.hip -- the extern "C" entry points declared in include/bitnet_w2a8.h.
//
// Every entry point validates its arguments on the host, before any HIP call, and
// returns a bitnet_status code; nothing throws across the ABI.  Work is enqueued on the
// caller's stream; nothing here synchronizes or allocates.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "bitnet_w2a8.h"
#include "kernels.hpp"

// Fewest tokens the fused quant + GEMV entry point sends to the register-quantizing
// kernel (K % 64 == 0); fewer go to the staged kernel.
#ifndef BITNET_FUSED_DIRECT_MIN_M
#define BITNET_FUSED_DIRECT_MIN_M 12
#endif

namespace {

thread_local char g_last_hip_error[256] = "";

int record_hip(hipError_t e) {
    if (e == hipSuccess) return BITNET_OK;
    std::snprintf(g_last_hip_error, sizeof g_last_hip_error, "%s (%d)", hipGetErrorString(e),
                  (int)e);
    return BITNET_ERR_HIP;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Per-device cache of "is this a gfx950": 0 unknown, 1 yes, 2 no.
constexpr int kMaxDevices = 64;
std::atomic<int> g_arch[kMaxDevices];

int check_device() {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return record_hip(e);
    if (dev < 0 || dev >= kMaxDevices) return BITNET_ERR_DEVICE;
    int state = g_arch[dev].load(std::memory_order_acquire);
    if (state == 0) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess) return record_hip(e);
        state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_arch[dev].store(state, std::memory_order_release);
    }
    return state == 1 ? BITNET_OK : BITNET_ERR_DEVICE;
}

// Shared shape checks: M, N >= 0, 4 <= K <= BITNET_MAX_K, K % 4 == 0, sizes that fit the
// kernels' 32-bit indices and grids.
int check_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 1) return BITNET_ERR_INVALID_ARG;
    if (K > BITNET_MAX_K) return BITNET_ERR_INVALID_ARG;
    if (M > INT32_MAX || N > INT32_MAX) return BITNET_ERR_INVALID_ARG;
    if (K % 4 != 0) return BITNET_ERR_UNALIGNED;
    return BITNET_OK;
}

bool valid_dtype(int dt) {
    return dt == BITNET_OUT_F32 || dt == BITNET_OUT_BF16 || dt == BITNET_OUT_I32;
}

bool valid_scale(int s) { return s == BITNET_SCALE_ABSMAX || s == BITNET_SCALE_POW2; }

// Shapes of a gradient: N[g] at most BITNET_MAX_K (the kernels' 32-bit offsets into a block
// of rows), M at most 2^30 (their 32-bit row numbers, padded to a tile).
int check_grad_groups(int64_t M, int64_t K, int64_t groups, const int64_t* N) {
    if (groups < 1 || groups > BITNET_MAX_GROUPS || !N) return BITNET_ERR_INVALID_ARG;
    if (M > BITNET_GRAD_MAX_M) return BITNET_ERR_INVALID_ARG;
    for (int64_t g = 0; g < groups; ++g) {
        const int st = check_shape(M, N[g], K);
        if (st) return st;
        if (N[g] > BITNET_MAX_K) return BITNET_ERR_INVALID_ARG;
    }
    return BITNET_OK;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// int8 product for M <= 16: the kernel that stages the activations in LDS for one to
// three tokens (and for four to seven with large N), the one that reads them straight
// into the matrix-core operands above (K % 64 == 0).  Measured crossover; both give
// identical outputs.
hipError_t launch_small_m(const int8_t* xq, const float* a_scale, const uint8_t* packed,
                          const float* w_scale, int64_t M, int64_t N, int64_t K, void* out,
                          int out_dtype, hipStream_t stream) {
    const bool direct = K % 64 == 0 && (M >= 8 || (M >= 4 && N <= 4096));
    if (direct)
        return bitnet::launch_gemv_direct(xq, a_scale, nullptr, packed, w_scale, M, N, K, out,
                                          out_dtype, nullptr, nullptr, stream);
    return bitnet::launch_skinny(xq, a_scale, nullptr, packed, w_scale, M, N, K, out, out_dtype,
                                 nullptr, nullptr, stream);
}

// The product of bitnet_w2a8_gemm once its arguments are validated.  Auto: the
// weight-streaming kernels while the product is small enough that one round of their
// blocks beats the tiled kernel (whose single-round grids cost about the same for any M
// up to 64): always up to 4 tokens, up to 16 while the weights are at most 16 MB, the
// direct kernel up to 32 tokens while N * K <= 2^25, and the staged kernel's token tiles
// up to 32 while M * N is small; else the tiled kernel, which may split K through the
// workspace.
int gemm_launch(const int8_t* xq, const float* a_scale, const uint8_t* packed,
                const float* w_scale, int64_t M, int64_t N, int64_t K, void* out, int out_dtype,
                int algo, void* workspace, size_t ws_bytes, hipStream_t stream) {
    if (algo == BITNET_ALGO_SKINNY)
        return record_hip(bitnet::launch_skinny(xq, a_scale, nullptr, packed, w_scale, M, N, K,
                                                out, out_dtype, nullptr, nullptr, stream));
    if (algo == BITNET_ALGO_AUTO) {
        if (M <= 4 || (M <= 16 && N * K <= ((int64_t)1 << 26)))
            return record_hip(launch_small_m(xq, a_scale, packed, w_scale, M, N, K, out,
                                             out_dtype, stream));
        // 17 to 32 tokens: the direct kernel's two token tiles while the activations it
        // re-reads per 16-row block (M * K bytes each) stay cheap next to the weights
        if (M <= 32 && K % 64 == 0 && N * K <= ((int64_t)1 << 25))
            return record_hip(bitnet::launch_gemv_direct(xq, a_scale, nullptr, packed, w_scale,
                                                         M, N, K, out, out_dtype, nullptr,
                                                         nullptr, stream));
        if (M <= 32 && M * N <= 131072)
            return record_hip(bitnet::launch_skinny(xq, a_scale, nullptr, packed, w_scale, M, N,
                                                    K, out, out_dtype, nullptr, nullptr, stream));
    }
    return record_hip(bitnet::launch_tiled(xq, a_scale, packed, w_scale, M, N, K, out, out_dtype,
                                           workspace, ws_bytes, stream));
}

// ---- device scratch of the allocation-free product (bitnet_w2a8_gemm_noalloc) ----
// The int32 partial sums of a split-K product live in this file-scope array: one copy on
// every GPU the library runs on, allocated with the code object and held until the
// process ends.  In host code `scratch` names a host-side stand-in, never the device
// memory: its address on a device is taken once per device with hipGetSymbolAddress
// (that device current) and only that address reaches kernels.  Every call on a GPU
// shares its copy, so calls that overlap on one GPU (different streams) race; the
// partials need no clearing, as every call writes each one before reading it.
constexpr size_t kScratchBytes = BITNET_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) int scratch[kScratchBytes / sizeof(int)];

struct ScratchSlot {
    std::mutex lock;
    std::atomic<void*> ptr{nullptr};
};
ScratchSlot g_scratch_slot[kMaxDevices];

// This device's scratch address (dev is the current device), looked up on the first
// call on the device; a failed lookup is retried by the next call.
hipError_t scratch_address(int dev, void** out) {
    ScratchSlot& slot = g_scratch_slot[dev];
    void* p = slot.ptr.load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> guard(slot.lock);
        p = slot.ptr.load(std::memory_order_relaxed);
        if (!p) {
            const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (e != hipSuccess) return e;
            if (!p) return hipErrorInvalidSymbol;
            slot.ptr.store(p, std::memory_order_release);
        }
    }
    *out = p;
    return hipSuccess;
}

}  // namespace

extern "C" {

int bitnet_abi_version(void) { return BITNET_ABI_VERSION; }

const char* bitnet_status_str(int status) {
    switch (status) {
        case BITNET_OK: return "ok";
        case BITNET_ERR_INVALID_ARG: return "invalid argument";
        case BITNET_ERR_UNALIGNED: return "unaligned size or pointer";
        case BITNET_ERR_WORKSPACE: return "workspace too small";
        case BITNET_ERR_HIP: return "HIP runtime error";
        case BITNET_ERR_DEVICE: return "unsupported device (gfx950 required)";
        default: return "unknown status";
    }
}

const char* bitnet_last_hip_error(void) { return g_last_hip_error; }

int bitnet_pack_weights(const float* w, int64_t N, int64_t K, uint8_t* packed, float* w_scale,
                        void* stream) {
    int st = check_shape(0, N, K);
    if (st) return st;
    if (N == 0) return BITNET_OK;
    if (!w || !packed || !w_scale) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(packed) || !aligned16(w_scale)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_pack_weights(w, N, K, packed, w_scale, as_stream(stream)));
}

int bitnet_unpack_weights(const uint8_t* packed, int64_t N, int64_t K, int8_t* codes,
                          void* stream) {
    int st = check_shape(0, N, K);
    if (st) return st;
    if (N == 0) return BITNET_OK;
    if (!packed || !codes) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(packed) || !aligned16(codes)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_unpack_weights(packed, N, K, codes, as_stream(stream)));
}

int bitnet_quant_act(const uint16_t* x, int64_t M, int64_t K, int8_t* xq, float* a_scale,
                     void* stream) {
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!x || !xq || !a_scale) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(a_scale)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_quant_act(x, M, K, xq, a_scale, as_stream(stream)));
}

int bitnet_w2a8_gemv(const int8_t* xq, const float* a_scale, const uint8_t* packed,
                     const float* w_scale, int64_t M, int64_t N, int64_t K, void* out,
                     int out_dtype, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (M > BITNET_GEMV_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!xq || !a_scale || !packed || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(a_scale) || !aligned16(packed) || !aligned16(w_scale) ||
        !aligned16(out))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(launch_small_m(xq, a_scale, packed, w_scale, M, N, K, out, out_dtype,
                                     as_stream(stream)));
}

size_t bitnet_w2a8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (check_shape(M, N, K) != BITNET_OK) return 0;
    return bitnet::tiled_workspace_size(M, N, K);
}

int bitnet_w2a8_gemm(const int8_t* xq, const float* a_scale, const uint8_t* packed,
                     const float* w_scale, int64_t M, int64_t N, int64_t K, void* out,
                     int out_dtype, int algo, void* workspace, size_t ws_bytes, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    if (algo != BITNET_ALGO_AUTO && algo != BITNET_ALGO_SKINNY && algo != BITNET_ALGO_TILED)
        return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (algo == BITNET_ALGO_SKINNY && M > BITNET_SKINNY_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!xq || !a_scale || !packed || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    if (ws_bytes > 0 && !workspace) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(a_scale) || !aligned16(packed) || !aligned16(w_scale) ||
        !aligned16(out) || !aligned16(workspace))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return gemm_launch(xq, a_scale, packed, w_scale, M, N, K, out, out_dtype, algo, workspace,
                       ws_bytes, as_stream(stream));
}

int bitnet_w2a8_gemm_noalloc(const int8_t* xq, const float* a_scale, const uint8_t* packed,
                             const float* w_scale, int64_t M, int64_t N, int64_t K, void* out,
                             int out_dtype, int algo, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    if (algo != BITNET_ALGO_AUTO && algo != BITNET_ALGO_SKINNY && algo != BITNET_ALGO_TILED)
        return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (algo == BITNET_ALGO_SKINNY && M > BITNET_SKINNY_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!xq || !a_scale || !packed || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(a_scale) || !aligned16(packed) || !aligned16(w_scale) ||
        !aligned16(out))
        return BITNET_ERR_UNALIGNED;
    // the planned partials must fit the fixed scratch (never the case below 32 MB: the
    // planner itself keeps partials under 64 MB)
    if (bitnet::tiled_workspace_size(M, N, K) > kScratchBytes) return BITNET_ERR_WORKSPACE;
    if ((st = check_device())) return st;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return record_hip(e);
    void* ws = nullptr;
    if ((e = scratch_address(dev, &ws)) != hipSuccess) return record_hip(e);
    return gemm_launch(xq, a_scale, packed, w_scale, M, N, K, out, out_dtype, algo, ws,
                       kScratchBytes, as_stream(stream));
}

int bitnet_pack_b3(const uint8_t* packed, int64_t N, int64_t K, uint8_t* b3, void* stream) {
    int st = check_shape(0, N, K);
    if (st) return st;
    if (N == 0) return BITNET_OK;
    if (!packed || !b3) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(packed) || !aligned16(b3)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_pack_b3(packed, N, K, b3, as_stream(stream)));
}

int bitnet_quant_gemv_b3(const uint16_t* x, const uint8_t* b3, const float* w_scale, int64_t M,
                         int64_t N, int64_t K, void* out, int out_dtype, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (K % 8 != 0) return BITNET_ERR_UNALIGNED;
    if (M > 1 || K > BITNET_B3_MAX_K) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!x || !b3 || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(b3) || !aligned16(w_scale) || !aligned16(out))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_quant_gemv_b3(x, b3, w_scale, N, K, out, out_dtype,
                                                   as_stream(stream)));
}

int bitnet_w2a8_gemm_grouped(const int8_t* xq, const float* a_scale, int64_t M, int64_t K,
                             int64_t groups, const uint8_t* const* packed,
                             const float* const* w_scale, const int64_t* N, void* const* out,
                             int out_dtype, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    if (groups < 1 || groups > BITNET_MAX_GROUPS) return BITNET_ERR_INVALID_ARG;
    if (!packed || !w_scale || !N || !out) return BITNET_ERR_INVALID_ARG;
    int64_t total_n = 0;
    for (int64_t g = 0; g < groups; ++g) {
        int st = check_shape(M, N[g], K);
        if (st) return st;
        total_n += N[g];
    }
    if (total_n > INT32_MAX) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || total_n == 0) return BITNET_OK;
    if (!xq || !a_scale) return BITNET_ERR_INVALID_ARG;
    for (int64_t g = 0; g < groups; ++g) {
        if (N[g] == 0) continue;
        if (!packed[g] || !w_scale[g] || !out[g]) return BITNET_ERR_INVALID_ARG;
        if (!aligned16(packed[g]) || !aligned16(w_scale[g]) || !aligned16(out[g]))
            return BITNET_ERR_UNALIGNED;
    }
    if (!aligned16(xq) || !aligned16(a_scale)) return BITNET_ERR_UNALIGNED;
    int st = check_device();
    if (st) return st;
    return record_hip(bitnet::launch_tiled_grouped(xq, a_scale, (int)groups, packed, w_scale, N,
                                                   out, M, K, out_dtype, as_stream(stream)));
}

int bitnet_w2a8_gemm_plan(int64_t M, int64_t K, int64_t groups, const int64_t* N, int64_t cus,
                          int32_t* plan) {
    if (groups < 1 || groups > BITNET_MAX_GROUPS || !N || !plan || M < 1)
        return BITNET_ERR_INVALID_ARG;
    int64_t total_n = 0;
    for (int64_t g = 0; g < groups; ++g) {
        int st = check_shape(M, N[g], K);
        if (st) return st;
        total_n += N[g];
    }
    if (total_n == 0 || total_n > INT32_MAX) return BITNET_ERR_INVALID_ARG;
    int p[5];
    bitnet::tiled_plan(M, K, (int)groups, N, cus, p);
    for (int i = 0; i < 5; ++i) plan[i] = p[i];
    return BITNET_OK;
}

int bitnet_quant_gemv(const uint16_t* x, const uint8_t* packed, const float* w_scale,
                      int64_t M, int64_t N, int64_t K, void* out, int out_dtype,
                      int8_t* xq_out, float* a_scale_out, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (M > BITNET_GEMV_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!x || !packed || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(w_scale) || !aligned16(out) ||
        !aligned16(xq_out) || !aligned16(a_scale_out))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    // 12 to 16 tokens: the kernel that quantizes in registers (its whole-row max scan is
    // cheaper there than the staged kernel's LDS copy); fewer: the staged kernel
    if (M >= BITNET_FUSED_DIRECT_MIN_M && K % 64 == 0)
        return record_hip(bitnet::launch_gemv_direct(nullptr, nullptr, x, packed, w_scale, M, N,
                                                     K, out, out_dtype, xq_out, a_scale_out,
                                                     as_stream(stream)));
    return record_hip(bitnet::launch_skinny(nullptr, nullptr, x, packed, w_scale, M, N, K, out,
                                            out_dtype, xq_out, a_scale_out, as_stream(stream)));
}

int bitnet_quant_gemv_grouped(const uint16_t* x, int64_t M, int64_t K, int64_t groups,
                              const uint8_t* const* packed, const float* const* w_scale,
                              const int64_t* N, void* const* out, int out_dtype,
                              int8_t* xq_out, float* a_scale_out, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    if (groups < 1 || groups > BITNET_MAX_GROUPS) return BITNET_ERR_INVALID_ARG;
    if (!packed || !w_scale || !N || !out) return BITNET_ERR_INVALID_ARG;
    int64_t total_n = 0;
    for (int64_t g = 0; g < groups; ++g) {
        int st = check_shape(M, N[g], K);
        if (st) return st;
        total_n += N[g];
    }
    if (M > BITNET_GEMV_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (total_n > INT32_MAX) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || total_n == 0) return BITNET_OK;
    if (!x) return BITNET_ERR_INVALID_ARG;
    for (int64_t g = 0; g < groups; ++g) {
        if (N[g] == 0) continue;
        if (!packed[g] || !w_scale[g] || !out[g]) return BITNET_ERR_INVALID_ARG;
        if (!aligned16(packed[g]) || !aligned16(w_scale[g]) || !aligned16(out[g]))
            return BITNET_ERR_UNALIGNED;
    }
    if (!aligned16(x) || !aligned16(xq_out) || !aligned16(a_scale_out)) return BITNET_ERR_UNALIGNED;
    int st = check_device();
    if (st) return st;
    return record_hip(bitnet::launch_skinny_grouped(nullptr, nullptr, x, (int)groups, packed,
                                                    w_scale, N, out, M, K, out_dtype, xq_out,
                                                    a_scale_out, as_stream(stream)));
}

int bitnet_quant_act_per_tensor(const uint16_t* x, int64_t M, int64_t K, int8_t* xq,
                                float* a_scale, void* stream) {
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!x || !xq || !a_scale) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(a_scale)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_quant_act_per_tensor(x, M, K, xq, a_scale, as_stream(stream)));
}

int bitnet_repack_codes(const uint8_t* in, int64_t N, int64_t K, int from_table, int to_table,
                        uint8_t* out, int32_t* invalid_count, void* stream) {
    const auto valid_table = [](int t) { return t == BITNET_CODES_OFFSET || t == BITNET_CODES_SIGN; };
    if (!valid_table(from_table) || !valid_table(to_table)) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(0, N, K);
    if (st) return st;
    if (N == 0) return BITNET_OK;
    if (!in || !out) return BITNET_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(invalid_count) & 3u) != 0) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_repack_codes(in, N, K, from_table, to_table, out,
                                                  invalid_count, as_stream(stream)));
}

int bitnet_a16_gemv(const uint16_t* x, const uint8_t* packed, const float* w_scale, int64_t M,
                    int64_t N, int64_t K, void* out, int out_dtype, void* stream) {
    if (out_dtype != BITNET_OUT_F32 && out_dtype != BITNET_OUT_BF16) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (K % 64 != 0) return BITNET_ERR_UNALIGNED;
    if (M > BITNET_GEMV_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!x || !packed || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(w_scale) || !aligned16(out))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_a16(x, packed, w_scale, M, N, K, out, out_dtype,
                                         as_stream(stream)));
}

int bitnet_quant_gemv_swiglu(const uint16_t* x, const uint8_t* packed_gate,
                             const float* w_scale_gate, const uint8_t* packed_up,
                             const float* w_scale_up, int64_t M, int64_t N, int64_t K, void* h,
                             int out_dtype, int8_t* xq_out, float* a_scale_out, void* stream) {
    if (out_dtype != BITNET_OUT_F32 && out_dtype != BITNET_OUT_BF16) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, N, K);
    if (st) return st;
    if (M > BITNET_GEMV_MAX_M) return BITNET_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!x || !packed_gate || !w_scale_gate || !packed_up || !w_scale_up || !h)
        return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed_gate) || !aligned16(w_scale_gate) ||
        !aligned16(packed_up) || !aligned16(w_scale_up) || !aligned16(h) || !aligned16(xq_out) ||
        !aligned16(a_scale_out))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_skinny_swiglu(x, packed_gate, w_scale_gate, packed_up,
                                                   w_scale_up, M, N, K, h, out_dtype, xq_out,
                                                   a_scale_out, as_stream(stream)));
}

// ---- the training side of a layer ----

int bitnet_quant_act_pow2(const uint16_t* x, int64_t M, int64_t K, int8_t* xq, float* a_scale,
                          void* stream) {
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!x || !xq || !a_scale) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(a_scale)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_quant_act_pow2(x, M, K, xq, a_scale, as_stream(stream)));
}

int bitnet_dequant_act(const int8_t* xq, const float* a_scale, int64_t M, int64_t K, uint16_t* x,
                       void* stream) {
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!x || !xq || !a_scale) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(a_scale)) return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_dequant_act(xq, a_scale, M, K, x, as_stream(stream)));
}

int bitnet_layernorm(const uint16_t* x, const float* weight, const float* bias, float eps,
                     int64_t M, int64_t K, uint16_t* y, int8_t* xq, float* a_scale, int scale,
                     float* mean, float* rstd, void* stream) {
    if (!valid_scale(scale)) return BITNET_ERR_INVALID_ARG;
    if (!(eps >= FLT_MIN) || eps > FLT_MAX) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!x || (!y && !xq) || (xq != nullptr) != (a_scale != nullptr)) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(weight) || !aligned16(bias) || !aligned16(y) || !aligned16(xq) ||
        !aligned16(a_scale) || !aligned16(mean) || !aligned16(rstd))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_layernorm(x, weight, bias, eps, M, K, y, xq, a_scale,
                                               scale == BITNET_SCALE_POW2, mean, rstd,
                                               as_stream(stream)));
}

size_t bitnet_layernorm_backward_workspace_size(int64_t M, int64_t K) {
    if (check_shape(M, 0, K) != BITNET_OK || M == 0) return 0;
    return bitnet::layernorm_back_workspace_size(M, K);
}

int bitnet_layernorm_backward(const uint16_t* dy, const void* x, const float* x_scale,
                              const float* weight, const float* mean, const float* rstd, int64_t M,
                              int64_t K, uint16_t* dx, float* dweight, float* dbias,
                              void* workspace, size_t ws_bytes, void* stream) {
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0 && !dweight && !dbias) return BITNET_OK;
    if (M > 0 && (!dy || !x || !mean || !rstd || !dx)) return BITNET_ERR_INVALID_ARG;
    if (ws_bytes > 0 && !workspace) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(x_scale) || !aligned16(weight) ||
        !aligned16(mean) || !aligned16(rstd) || !aligned16(dx) || !aligned16(dweight) ||
        !aligned16(dbias) || !aligned16(workspace))
        return BITNET_ERR_UNALIGNED;
    if (M > 0 && (dweight || dbias) && ws_bytes < bitnet::layernorm_back_workspace_size(M, K))
        return BITNET_ERR_WORKSPACE;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_layernorm_back(dy, x, x_scale, weight, mean, rstd, M, K, dx,
                                                    dweight, dbias, workspace, as_stream(stream)));
}

int bitnet_swiglu(const uint16_t* g, const uint16_t* u, int64_t M, int64_t N, uint16_t* h,
                  int8_t* hq, float* h_scale, int scale, int8_t* gq, float* g_scale, int8_t* uq,
                  float* u_scale, void* stream) {
    if (!valid_scale(scale)) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, 0, N);  // N is the K of the product that reads h
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!g || !u || (!h && !hq) || (hq != nullptr) != (h_scale != nullptr))
        return BITNET_ERR_INVALID_ARG;
    const int kept = (gq != nullptr) + (g_scale != nullptr) + (uq != nullptr) + (u_scale != nullptr);
    if (kept != 0 && kept != 4) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(g) || !aligned16(u) || !aligned16(h) || !aligned16(hq) || !aligned16(h_scale) ||
        !aligned16(gq) || !aligned16(g_scale) || !aligned16(uq) || !aligned16(u_scale))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_swiglu(g, u, M, N, h, hq, h_scale, scale == BITNET_SCALE_POW2,
                                            gq, g_scale, uq, u_scale, as_stream(stream)));
}

int bitnet_swiglu_backward(const uint16_t* dh, const void* g, const float* g_scale, const void* u,
                           const float* u_scale, int64_t M, int64_t N, uint16_t* dg, uint16_t* du,
                           void* stream) {
    int st = check_shape(M, 0, N);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!dh || !g || !u || !dg || !du || (g_scale != nullptr) != (u_scale != nullptr))
        return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dh) || !aligned16(g) || !aligned16(g_scale) || !aligned16(u) ||
        !aligned16(u_scale) || !aligned16(dg) || !aligned16(du))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_swiglu_back(dh, g, g_scale, u, u_scale, M, N, dg, du,
                                                 as_stream(stream)));
}

size_t bitnet_grad_input_workspace_size(int64_t M, int64_t K, int64_t groups, const int64_t* N) {
    if (check_grad_groups(M, K, groups, N) != BITNET_OK || M == 0) return 0;
    return bitnet::grad_input_workspace_size(M, K, (int)groups, N);
}

int bitnet_grad_input(int64_t M, int64_t K, int64_t groups, const uint16_t* const* dy,
                      const uint8_t* const* packed, const float* const* w_scale, const int64_t* N,
                      uint16_t* dx, void* workspace, size_t ws_bytes, void* stream) {
    int st = check_grad_groups(M, K, groups, N);
    if (st) return st;
    if (!dy || !packed || !w_scale) return BITNET_ERR_INVALID_ARG;
    if (M == 0) return BITNET_OK;
    if (!dx || (ws_bytes > 0 && !workspace)) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dx) || !aligned16(workspace)) return BITNET_ERR_UNALIGNED;
    for (int64_t g = 0; g < groups; ++g) {
        if (N[g] == 0) continue;
        if (!dy[g] || !packed[g] || !w_scale[g]) return BITNET_ERR_INVALID_ARG;
        if (!aligned16(dy[g]) || !aligned16(packed[g]) || !aligned16(w_scale[g]))
            return BITNET_ERR_UNALIGNED;
    }
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_grad_input(dy, packed, w_scale, N, (int)groups, M, K, dx,
                                                workspace, ws_bytes, as_stream(stream)));
}

static int grad_plan(int weight, int64_t M, int64_t K, int64_t groups, const int64_t* N, int first,
                     int last, int32_t* out) {
    const int st = check_grad_groups(M, K, groups, N);
    if (st) return st;
    if (!out || M < 1 || (weight && (groups != 1 || N[0] < 1))) return BITNET_ERR_INVALID_ARG;
    int p[5];
    if (weight)
        bitnet::grad_plan(0, N[0], K, &M, 1, p);
    else
        bitnet::grad_plan(1, M, K, N, (int)groups, p);
    for (int i = first; i <= last; ++i) out[i - first] = p[i];
    return BITNET_OK;
}

int bitnet_grad_plan(int weight, int64_t M, int64_t K, int64_t groups, const int64_t* N,
                     int32_t* plan) {
    return grad_plan(weight, M, K, groups, N, 0, 3, plan);
}

int bitnet_grad_plan_step(int weight, int64_t M, int64_t K, int64_t groups, const int64_t* N,
                          int32_t* step) {
    return grad_plan(weight, M, K, groups, N, 4, 4, step);
}

size_t bitnet_grad_weight_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (check_grad_groups(M, K, 1, &N) != BITNET_OK || M == 0 || N == 0) return 0;
    return bitnet::grad_weight_workspace_size(M, N, K);
}

int bitnet_grad_weight(const uint16_t* dy, const int8_t* xq, const float* a_scale, int64_t M,
                       int64_t N, int64_t K, void* dw, int out_dtype, void* workspace,
                       size_t ws_bytes, void* stream) {
    if (out_dtype != BITNET_OUT_F32 && out_dtype != BITNET_OUT_BF16) return BITNET_ERR_INVALID_ARG;
    int st = check_grad_groups(M, K, 1, &N);
    if (st) return st;
    if (N == 0) return BITNET_OK;
    if (!dw || (ws_bytes > 0 && !workspace)) return BITNET_ERR_INVALID_ARG;
    if (M > 0 && (!dy || !xq || !a_scale)) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(xq) || !aligned16(a_scale) || !aligned16(dw) ||
        !aligned16(workspace))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_grad_weight(dy, xq, a_scale, M, N, K, dw, out_dtype, workspace,
                                                 ws_bytes, as_stream(stream)));
}

// ---- root-mean-square norm, global norm of the gradients ----

int bitnet_rmsnorm(const uint16_t* x, const uint16_t* residual, const float* weight, float eps,
                   int64_t M, int64_t K, uint16_t* sum, uint16_t* y, int8_t* xq, float* a_scale,
                   int scale, float* rstd, void* stream) {
    if (!valid_scale(scale)) return BITNET_ERR_INVALID_ARG;
    if (!(eps >= FLT_MIN) || eps > FLT_MAX) return BITNET_ERR_INVALID_ARG;
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0) return BITNET_OK;
    if (!x || (!y && !xq) || (xq != nullptr) != (a_scale != nullptr) ||
        (residual != nullptr) != (sum != nullptr))
        return BITNET_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(sum) || !aligned16(y) ||
        !aligned16(xq) || !aligned16(a_scale) || !aligned16(rstd))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_rmsnorm(x, residual, weight, eps, M, K, sum, y, xq, a_scale,
                                             scale == BITNET_SCALE_POW2, rstd, as_stream(stream)));
}

size_t bitnet_rmsnorm_backward_workspace_size(int64_t M, int64_t K) {
    if (check_shape(M, 0, K) != BITNET_OK || M == 0) return 0;
    return bitnet::rmsnorm_back_workspace_size(M, K);
}

int bitnet_rmsnorm_backward(const uint16_t* dy, const void* x, const float* x_scale,
                            const float* weight, const float* rstd, const uint16_t* dresidual,
                            int64_t M, int64_t K, uint16_t* dx, float* dweight, void* workspace,
                            size_t ws_bytes, void* stream) {
    int st = check_shape(M, 0, K);
    if (st) return st;
    if (M == 0 && !dweight) return BITNET_OK;
    if (M > 0 && (!dy || !x || !rstd || !dx)) return BITNET_ERR_INVALID_ARG;
    if (ws_bytes > 0 && !workspace) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(x_scale) || !aligned16(weight) ||
        !aligned16(rstd) || !aligned16(dresidual) || !aligned16(dx) || !aligned16(dweight) ||
        !aligned16(workspace))
        return BITNET_ERR_UNALIGNED;
    if (M > 0 && dweight && ws_bytes < bitnet::rmsnorm_back_workspace_size(M, K))
        return BITNET_ERR_WORKSPACE;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_rmsnorm_back(dy, x, x_scale, weight, rstd, dresidual, M, K, dx,
                                                  dweight, workspace, as_stream(stream)));
}

// The lists of the norm and of clipping: pointers aligned to their values, sizes that 63 bits hold
// in bytes.
static int check_grads(int64_t count, const void* const* grads, const int64_t* n, const int32_t* dtype) {
    if (count < 0 || count > INT32_MAX) return BITNET_ERR_INVALID_ARG;
    if (count > 0 && (!grads || !n || !dtype)) return BITNET_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        if (dtype[i] != BITNET_OUT_F32 && dtype[i] != BITNET_OUT_BF16) return BITNET_ERR_INVALID_ARG;
        if (n[i] < 0 || n[i] > INT64_MAX / 8) return BITNET_ERR_INVALID_ARG;
        if (n[i] == 0) continue;
        if (!grads[i]) return BITNET_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(grads[i]) & (dtype[i] == BITNET_OUT_F32 ? 3u : 1u))
            return BITNET_ERR_UNALIGNED;
    }
    return BITNET_OK;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t bitnet_grad_norm_workspace_size(int64_t count) {
    if (count < 0 || count > INT32_MAX) return 0;
    return bitnet::grad_norm_workspace_size(count > 0 ? count : 1);
}

int bitnet_grad_norm(int64_t count, const void* const* grads, const int64_t* n, const int32_t* dtype,
                     float* norm, void* workspace, size_t ws_bytes, void* stream) {
    int st = check_grads(count, grads, n, dtype);
    if (st) return st;
    if (!norm || (ws_bytes > 0 && !workspace)) return BITNET_ERR_INVALID_ARG;
    if (!aligned4(norm) || !aligned16(workspace)) return BITNET_ERR_UNALIGNED;
    if (ws_bytes < bitnet_grad_norm_workspace_size(count)) return BITNET_ERR_WORKSPACE;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_grad_norm(count, grads, nullptr, n, dtype, false, 0.0f, nullptr,
                                               norm, workspace, as_stream(stream)));
}

// Whether an output overlaps another output, or an input that is not its own (out[i] == grads[i]
// exactly).  In the order of their starts an output may not begin before the furthest end of the spans in
// front of it, nor an input before that of the outputs.  The spans pass in that order through a buffer on
// the stack: all that fit, or the lowest half buffer of those not seen yet, so that longer lists are read
// again for each.
static int check_clip_outputs(int64_t count, const void* const* grads, void* const* out, const int64_t* n,
                              const int32_t* dtype) {
    struct Span {
        uintptr_t begin;
        int64_t i;  // even: output, odd: input of tensor i / 2
        bool operator<(const Span& b) const { return begin != b.begin ? begin < b.begin : i < b.i; }
    };
    constexpr int kSpans = 2048, kKeep = kSpans / 2;
    Span buf[kSpans];
    Span seen = {0, -1};
    uintptr_t any = 0, outs = 0;
    bool more = true;
    while (more) {
        more = false;
        int m = 0;
        Span most = {UINTPTR_MAX, INT64_MAX};
        for (int64_t t = 0; t < count; ++t) {
            if (n[t] == 0) continue;
            for (int64_t i = 2 * t; i < 2 * t + (grads[t] == out[t] ? 1 : 2); ++i) {
                const Span s = {reinterpret_cast<uintptr_t>(i & 1 ? grads[t] : out[t]), i};
                if (!(seen < s) || !(s < most)) continue;
                if (m == kSpans) {
                    std::nth_element(buf, buf + kKeep, buf + m);
                    m = kKeep;
                    most = buf[kKeep];
                    more = true;
                    if (!(s < most)) continue;
                }
                buf[m++] = s;
            }
        }
        std::sort(buf, buf + m, [](const Span& a, const Span& b) { return a.begin < b.begin; });
        for (int k = 0; k < m; ++k) {
            const int64_t t = buf[k].i >> 1;
            const bool is_out = (buf[k].i & 1) == 0;
            if (buf[k].begin < (is_out ? any : outs)) return BITNET_ERR_INVALID_ARG;
            const uintptr_t end = buf[k].begin + (uintptr_t)n[t] * (dtype[t] == BITNET_OUT_F32 ? 4 : 2);
            any = std::max(any, end);
            if (is_out) outs = std::max(outs, end);
        }
        if (more) seen = *std::max_element(buf, buf + m);
    }
    return BITNET_OK;
}

int bitnet_clip_grads(int64_t count, const void* const* grads, void* const* out, const int64_t* n,
                      const int32_t* dtype, float max_norm, const float* norm_in, float* norm_out,
                      void* workspace, size_t ws_bytes, void* stream) {
    int st = check_grads(count, grads, n, dtype);
    if (st) return st;
    if (!(max_norm >= 0.0f) || max_norm > FLT_MAX) return BITNET_ERR_INVALID_ARG;
    if (count > 0 && !out) return BITNET_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        if (n[i] == 0) continue;
        if (!out[i]) return BITNET_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(out[i]) & (dtype[i] == BITNET_OUT_F32 ? 3u : 1u))
            return BITNET_ERR_UNALIGNED;
    }
    if (ws_bytes > 0 && !workspace) return BITNET_ERR_INVALID_ARG;
    if (!aligned4(norm_in) || !aligned4(norm_out) || !aligned16(workspace)) return BITNET_ERR_UNALIGNED;
    if (!norm_in && ws_bytes < bitnet_grad_norm_workspace_size(count)) return BITNET_ERR_WORKSPACE;
    if ((st = check_clip_outputs(count, grads, out, n, dtype))) return st;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_grad_norm(count, grads, out, n, dtype, true, max_norm, norm_in,
                                               norm_out, workspace, as_stream(stream)));
}

// ---- mixture of experts ----

static int check_experts(int64_t P, int64_t E, int64_t K, int64_t groups, const int64_t* N) {
    if (E < 1 || E > BITNET_MAX_EXPERTS) return BITNET_ERR_INVALID_ARG;
    return check_grad_groups(P, K, groups, N);  // P within BITNET_GRAD_MAX_M, N within BITNET_MAX_K
}

// Tokens behind the rows: as many as rows without a gather, else within 31 bits of codes.
static bool valid_tokens(int64_t T, const int32_t* rows, int64_t P, int64_t K) {
    if (T < 0 || T > INT32_MAX) return false;
    return rows ? T * K <= INT32_MAX : T == P;
}

size_t bitnet_expert_order_workspace_size(int64_t P, int64_t E) {
    if (P < 0 || P > BITNET_GRAD_MAX_M || E < 1 || E > BITNET_MAX_EXPERTS) return 0;
    return bitnet::expert_order_workspace_size(P, E);
}

int bitnet_expert_order(const void* ids, int wide, int64_t T, int64_t J, int64_t E, int32_t* rows,
                        int32_t* offsets, int32_t* slots, void* workspace, size_t ws_bytes,
                        void* stream) {
    if (T < 0 || T > BITNET_GRAD_MAX_M || J < 1 || J > BITNET_MAX_EXPERTS || T * J > BITNET_GRAD_MAX_M ||
        E < 1 || E > BITNET_MAX_EXPERTS || (wide != 0 && wide != 1))
        return BITNET_ERR_INVALID_ARG;
    if (!offsets || (T > 0 && (!ids || !rows || !slots)) || (ws_bytes > 0 && !workspace))
        return BITNET_ERR_INVALID_ARG;
    if (!aligned16(ids) || !aligned16(rows) || !aligned16(offsets) || !aligned16(slots) ||
        !aligned16(workspace))
        return BITNET_ERR_UNALIGNED;
    if (ws_bytes < bitnet::expert_order_workspace_size(T * J, E)) return BITNET_ERR_WORKSPACE;
    const int st = check_device();
    if (st) return st;
    return record_hip(bitnet::launch_expert_order(ids, wide, T, J, E, rows, offsets, slots, workspace,
                                                  as_stream(stream)));
}

int bitnet_gemm_experts(const int8_t* xq, const float* a_scale, int64_t T, const int32_t* rows,
                        const int32_t* offsets, int64_t P, int64_t E, int64_t K, int64_t groups,
                        const uint8_t* const* packed, const float* const* w_scale, const int64_t* N,
                        void* const* out, int out_dtype, void* stream) {
    if (!valid_dtype(out_dtype)) return BITNET_ERR_INVALID_ARG;
    int st = check_experts(P, E, K, groups, N);
    if (st) return st;
    if (!valid_tokens(T, rows, P, K)) return BITNET_ERR_INVALID_ARG;
    if (!packed || !w_scale || !out) return BITNET_ERR_INVALID_ARG;
    int64_t total_n = 0;
    for (int64_t g = 0; g < groups; ++g) total_n += N[g];
    if (P == 0 || total_n == 0) return BITNET_OK;
    if (!offsets || (T > 0 && (!xq || !a_scale))) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(a_scale) || !aligned16(rows) || !aligned16(offsets))
        return BITNET_ERR_UNALIGNED;
    for (int64_t g = 0; g < groups; ++g) {
        if (N[g] == 0) continue;
        if (!packed[g] || !w_scale[g] || !out[g]) return BITNET_ERR_INVALID_ARG;
        if (!aligned16(packed[g]) || !aligned16(w_scale[g]) || !aligned16(out[g]))
            return BITNET_ERR_UNALIGNED;
    }
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_gemm_experts(xq, a_scale, T, rows, offsets, P, E, K, (int)groups,
                                                  packed, w_scale, N, out, out_dtype, as_stream(stream)));
}

int bitnet_grad_input_experts(const int32_t* offsets, int64_t P, int64_t E, int64_t K, int64_t groups,
                              const uint16_t* const* dy, const uint8_t* const* packed,
                              const float* const* w_scale, const int64_t* N, uint16_t* dx,
                              void* stream) {
    int st = check_experts(P, E, K, groups, N);
    if (st) return st;
    if (!dy || !packed || !w_scale) return BITNET_ERR_INVALID_ARG;
    if (P == 0) return BITNET_OK;
    if (!offsets || !dx) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(offsets) || !aligned16(dx)) return BITNET_ERR_UNALIGNED;
    for (int64_t g = 0; g < groups; ++g) {
        if (N[g] == 0) continue;
        if (!dy[g] || !packed[g] || !w_scale[g]) return BITNET_ERR_INVALID_ARG;
        if (!aligned16(dy[g]) || !aligned16(packed[g]) || !aligned16(w_scale[g]))
            return BITNET_ERR_UNALIGNED;
    }
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_grad_input_experts(dy, offsets, P, E, packed, w_scale, N,
                                                        (int)groups, K, dx, as_stream(stream)));
}

// Codes in the rows' order, then their scales.
static size_t gathered_codes(int64_t P, int64_t K) { return ((size_t)(P * K) + 15) / 16 * 16; }

size_t bitnet_grad_weight_experts_workspace_size(int64_t P, int64_t K) {
    if (check_shape(P, 0, K) != BITNET_OK || P > BITNET_GRAD_MAX_M || P == 0) return 0;
    return gathered_codes(P, K) + (size_t)P * 4;
}

int bitnet_grad_weight_experts(const uint16_t* dy, const int8_t* xq, const float* a_scale, int64_t T,
                               const int32_t* rows, const int32_t* offsets, int64_t P, int64_t E,
                               int64_t N, int64_t K, void* dw, int out_dtype, void* workspace,
                               size_t ws_bytes, void* stream) {
    if (out_dtype != BITNET_OUT_F32 && out_dtype != BITNET_OUT_BF16) return BITNET_ERR_INVALID_ARG;
    int st = check_experts(P, E, K, 1, &N);
    if (st) return st;
    if (!valid_tokens(T, rows, P, K)) return BITNET_ERR_INVALID_ARG;
    if (N == 0) return BITNET_OK;
    if (!dw || !offsets || (ws_bytes > 0 && !workspace)) return BITNET_ERR_INVALID_ARG;
    if (P > 0 && (!dy || (T > 0 && (!xq || !a_scale)))) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(xq) || !aligned16(a_scale) || !aligned16(rows) ||
        !aligned16(offsets) || !aligned16(dw) || !aligned16(workspace))
        return BITNET_ERR_UNALIGNED;
    if (rows && ws_bytes < bitnet_grad_weight_experts_workspace_size(P, K)) return BITNET_ERR_WORKSPACE;
    if ((st = check_device())) return st;
    if (rows && P > 0) {
        int8_t* const xs = static_cast<int8_t*>(workspace);
        float* const as = reinterpret_cast<float*>(xs + gathered_codes(P, K));
        st = record_hip(bitnet::launch_gather_codes(xq, a_scale, T, rows, P, K, xs, as, as_stream(stream)));
        if (st) return st;
        xq = xs;
        a_scale = as;
    }
    return record_hip(bitnet::launch_grad_weight_experts(dy, xq, a_scale, offsets, P, E, N, K, dw,
                                                         out_dtype, as_stream(stream)));
}

static int check_combine(int64_t T, int64_t J, int64_t P, int64_t D) {
    if (J < 1 || J > BITNET_MAX_EXPERTS || P < 0 || P > BITNET_GRAD_MAX_M || T > BITNET_GRAD_MAX_M)
        return BITNET_ERR_INVALID_ARG;
    return check_shape(T, 0, D);
}

int bitnet_combine_experts(const uint16_t* y, const int32_t* slots, const float* weights, int64_t T,
                           int64_t J, int64_t P, int64_t D, uint16_t* out, void* stream) {
    int st = check_combine(T, J, P, D);
    if (st) return st;
    if (T == 0) return BITNET_OK;
    if (!slots || !out || (P > 0 && !y)) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(y) || !aligned16(slots) || !aligned16(weights) || !aligned16(out))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_combine(y, slots, weights, T, J, P, D, out, as_stream(stream)));
}

int bitnet_combine_experts_backward(const uint16_t* dout, const uint16_t* y, const int32_t* slots,
                                    const float* weights, int64_t T, int64_t J, int64_t P, int64_t D,
                                    uint16_t* dy, float* dweights, void* stream) {
    int st = check_combine(T, J, P, D);
    if (st) return st;
    if (T == 0) return BITNET_OK;
    if (!dout || !slots || (P > 0 && (!dy || (dweights && !y)))) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(dout) || !aligned16(y) || !aligned16(slots) || !aligned16(weights) ||
        !aligned16(dy) || !aligned16(dweights))
        return BITNET_ERR_UNALIGNED;
    if ((st = check_device())) return st;
    return record_hip(bitnet::launch_combine_back(dout, y, slots, weights, T, J, P, D, dy, dweights,
                                                  as_stream(stream)));
}

}  // extern "C"
