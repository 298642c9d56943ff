// clip.hip -- the global norm of many gradient tensors, and their clipping to a largest norm, on
// gfx950.
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),  g <- g c
//
// Bound by HBM: the norm reads every value once, the scaling reads it again and writes it.  Squares
// and sums are fp64, where the square of an fp32 value is exact and neither overflows nor
// vanishes; two fp64 operations a value are below the time of its bytes.
//
// A launch takes up to kList tensors whose pointers and sizes travel as kernel arguments (no table
// has to be copied to the device, so the calls can be captured).  Every tensor is cut into chunks
// of kChunk bytes, a block walks every gridDim-th chunk and finds its tensor by bisection, and
// leaves one partial sum.  The partial sums are added in a fixed order (no atomics: the same
// inputs give the same bits), by one block for the norm alone, and for clipping by each block of
// the scaling kernel itself, which saves a launch between the two passes over the data.  The
// scaling walks the chunks backwards: what the norm read last is still in the caches.
// Measured: 106 million fp32 values (the matrices and vectors of four 6912 x 2560 layers) 102 to 109 us
// for the squares (3.9 to 4.2 TB/s) and 134 to 145 for the scaling (5.9 to 6.4); 16 small tensors 4.3
// and 5.7 us, launch and one memory trip each.
#include "device_common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace bitnet {

namespace {

constexpr int kList = 128;         // tensors of a launch
constexpr int kChunk = 32 * 1024;  // bytes
constexpr int kThreads = 512;
constexpr int kBlocks = 1024;      // most blocks, and partial sums, of a launch

struct GradList {
    const void* p[kList];
    void* out[kList];       // scaling only
    int64_t n[kList];       // values
    int first[kList + 1];   // first chunk of each tensor; the last entry is their number
    uint64_t bf16[kList / 64];
    int count;
};
static_assert(sizeof(GradList) + 64 <= 4096, "kernel arguments");

// Values before the first 16-byte boundary, whole 16-byte vectors behind it, the rest.
struct Span {
    int64_t head, vecs;
};
__host__ __device__ inline Span span_of(const void* p, int64_t n, int size) {
    const int64_t off = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / size;
    const int64_t head = off < n ? off : n;
    return {head, (n - head) * size / 16};
}

// Calls f(tensor, first vector, number of vectors, whether the chunk is the tensor's first) for
// the chunks of this block, from the last to the first with BACK.
template <bool BACK, class F>
__device__ __forceinline__ void for_chunks(const GradList& l, const F& f) {
    const int total = l.first[l.count];
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
        const int c = BACK ? total - 1 - i : i;
        int lo = 0, hi = l.count;  // first[lo] <= c < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (l.first[mid] <= c)
                lo = mid;
            else
                hi = mid;
        }
        f(lo, (int64_t)(c - l.first[lo]) * (kChunk / 16), c == l.first[lo]);
    }
}

__device__ __forceinline__ double square(double acc, float v) {
    return __builtin_fma((double)v, (double)v, acc);
}

// Sum over the block in a fixed order; the result is in every thread.
__device__ __forceinline__ double block_sum(double v, double (&s)[kThreads / 64]) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) v += s[i];
    return v;
}

// Sum of `blocks` partial sums, the same in every block that asks.
__device__ __forceinline__ float norm_of(const double* part, int blocks, double (&s)[kThreads / 64]) {
    double v = 0.0;
    for (int i = threadIdx.x; i < blocks; i += kThreads) v += part[i];
    return (float)__builtin_sqrt(block_sum(v, s));
}

// `norm` not NULL (a single block): the norm itself, else part[blockIdx.x].
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradList l, double* part, float* norm) {
    __shared__ double s[kThreads / 64];
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for_chunks<false>(l, [&](int t, int64_t v0, bool first) {
        const bool bf = l.bf16[t >> 6] >> (t & 63) & 1;
        const int64_t n = l.n[t];
        const Span sp = span_of(l.p[t], n, bf ? 2 : 4);
        const int nv = (int)(sp.vecs - v0 < kChunk / 16 ? sp.vecs - v0 : kChunk / 16);
        auto vec = [&](const uint4& u) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (bf) {
                    acc[j] = square(acc[j], __uint_as_float(w[j] << 16));
                    acc[j] = square(acc[j], __uint_as_float(w[j] & 0xFFFF0000u));
                } else {
                    acc[j] = square(acc[j], __uint_as_float(w[j]));
                }
            }
        };
        const uint4* const p = reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(l.p[t]) + sp.head * (bf ? 2 : 4)) + v0;
        if (nv == kChunk / 16) {
            uint4 u[kChunk / 16 / kThreads];
#pragma unroll
            for (int j = 0; j < kChunk / 16 / kThreads; ++j) u[j] = p[threadIdx.x + j * kThreads];
#pragma unroll
            for (int j = 0; j < kChunk / 16 / kThreads; ++j) vec(u[j]);
        } else {
            for (int i = threadIdx.x; i < nv; i += kThreads) vec(p[i]);
        }
        if (first && threadIdx.x < 16) {  // at most 7 values on either side of the vectors
            const int64_t end = sp.head + sp.vecs * (bf ? 8 : 4);
            const int64_t i = threadIdx.x < 8 ? threadIdx.x : end + threadIdx.x - 8;
            if (threadIdx.x < 8 ? i < sp.head : i < n)
                acc[0] = square(acc[0], bf ? bf16_bits_to_f32(static_cast<const uint16_t*>(l.p[t])[i])
                                           : static_cast<const float*>(l.p[t])[i]);
        }
    });
    const double v = block_sum((acc[0] + acc[1]) + (acc[2] + acc[3]), s);
    if (threadIdx.x == 0) {
        if (norm)
            *norm = (float)__builtin_sqrt(v);
        else
            part[blockIdx.x] = v;
    }
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* part, int blocks, float* norm) {
    __shared__ double s[kThreads / 64];
    const float v = norm_of(part, blocks, s);
    if (threadIdx.x == 0) *norm = v;
}

// The norm is *norm_in, or comes from the partial sums; the first block writes it to *norm_out.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradList l, const double* part, int blocks,
                                                              const float* norm_in, float* norm_out,
                                                              float max_norm) {
    __shared__ double s[kThreads / 64];
    const float norm = norm_in ? *norm_in : norm_of(part, blocks, s);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    float c = max_norm / (norm + 1e-6f);
    c = c > 1.0f ? 1.0f : c;  // NaN stays, and shows in every gradient
    for_chunks<true>(l, [&](int t, int64_t v0, bool first) {
        if (c == 1.0f && l.p[t] == l.out[t]) return;  // nothing to change
        const bool bf = l.bf16[t >> 6] >> (t & 63) & 1;
        const int size = bf ? 2 : 4;
        const int64_t n = l.n[t];
        const Span sp = span_of(l.p[t], n, size);
        const int nv = (int)(sp.vecs - v0 < kChunk / 16 ? sp.vecs - v0 : kChunk / 16);
        auto one = [&](int64_t i) {
            if (bf)
                static_cast<uint16_t*>(l.out[t])[i] =
                    f32_to_bf16_rne(bf16_bits_to_f32(static_cast<const uint16_t*>(l.p[t])[i]) * c);
            else
                static_cast<float*>(l.out[t])[i] = static_cast<const float*>(l.p[t])[i] * c;
        };
        auto vec = [&](const uint4& u) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = bf ? f32x2_to_bf16x2_rne(__uint_as_float(w[j] << 16) * c,
                                                __uint_as_float(w[j] & 0xFFFF0000u) * c)
                          : __float_as_uint(__uint_as_float(w[j]) * c);
            return make_uint4(o[0], o[1], o[2], o[3]);
        };
        const uint8_t* const src = static_cast<const uint8_t*>(l.p[t]) + sp.head * size;
        uint8_t* const dst = static_cast<uint8_t*>(l.out[t]) + sp.head * size;
        if (((uintptr_t)dst & 15) != 0) {  // the two lie differently: value by value
            const int64_t e0 = sp.head + v0 * (16 / size), e1 = e0 + (int64_t)nv * (16 / size);
            for (int64_t i = e0 + threadIdx.x; i < e1; i += kThreads) one(i);
        } else {
            const uint4* const p = reinterpret_cast<const uint4*>(src) + v0;
            uint4* const q = reinterpret_cast<uint4*>(dst) + v0;
            if (nv == kChunk / 16) {
                uint4 u[kChunk / 16 / kThreads];
#pragma unroll
                for (int j = 0; j < kChunk / 16 / kThreads; ++j) u[j] = p[threadIdx.x + j * kThreads];
#pragma unroll
                for (int j = 0; j < kChunk / 16 / kThreads; ++j) q[threadIdx.x + j * kThreads] = vec(u[j]);
            } else {
                for (int i = threadIdx.x; i < nv; i += kThreads) q[i] = vec(p[i]);
            }
        }
        if (first && threadIdx.x < 16) {
            const int64_t end = sp.head + sp.vecs * (16 / size);
            const int64_t i = threadIdx.x < 8 ? threadIdx.x : end + threadIdx.x - 8;
            if (threadIdx.x < 8 ? i < sp.head : i < n) one(i);
        }
    });
}

// Fills the list with tensors from `at` on; returns where the next list starts.
int64_t fill(GradList& l, int64_t at, int64_t count, const void* const* grads, void* const* out,
             const int64_t* n, const int32_t* dtype) {
    l.count = 0;
    l.first[0] = 0;
    for (uint64_t& b : l.bf16) b = 0;
    for (; at < count && l.count < kList; ++at) {
        if (n[at] == 0) continue;
        const bool bf = dtype[at] == BITNET_OUT_BF16;
        const int64_t chunks =
            (span_of(grads[at], n[at], bf ? 2 : 4).vecs * 16 + kChunk - 1) / kChunk;
        const int64_t end = l.first[l.count] + (chunks > 0 ? chunks : 1);
        if (end > INT32_MAX) {  // more than 2^46 bytes
            if (l.count == 0) return -1;
            break;
        }
        l.p[l.count] = grads[at];
        l.out[l.count] = out ? out[at] : nullptr;
        l.n[l.count] = n[at];
        if (bf) l.bf16[l.count >> 6] |= (uint64_t)1 << (l.count & 63);
        l.first[++l.count] = (int)end;
    }
    return at;
}

unsigned blocks_of(const GradList& l) {
    const int c = l.first[l.count];
    return c < kBlocks ? (c > 0 ? c : 1) : kBlocks;
}

}  // namespace

size_t grad_norm_workspace_size(int64_t count) {
    return (size_t)((count + kList - 1) / kList) * kBlocks * sizeof(double);
}

// clip: scale by the norm (norm_in, or the one computed here) into `out`.
hipError_t launch_grad_norm(int64_t count, const void* const* grads, void* const* out, const int64_t* n,
                            const int32_t* dtype, bool clip, float max_norm, const float* norm_in,
                            float* norm_out, void* workspace, hipStream_t stream) {
    GradList l;
    double* const part = static_cast<double*>(workspace);
    int blocks = 0;
    if (!norm_in) {
        int64_t at = 0;
        do {
            const int64_t from = at;
            at = fill(l, at, count, grads, nullptr, n, dtype);
            if (at < 0) return hipErrorInvalidValue;
            const unsigned b = blocks_of(l);
            // one block that has everything writes the norm itself
            const bool alone = !clip && from == 0 && at == count && b == 1;
            hipLaunchKernelGGL(grad_squares_kernel, dim3(b), dim3(kThreads), 0, stream, l, part + blocks,
                               alone ? norm_out : nullptr);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || alone) return e;
            blocks += (int)b;
        } while (at < count);
        if (!clip) {
            hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, part, blocks, norm_out);
            return hipGetLastError();
        }
    }
    int64_t at = 0;
    bool told = false;
    do {
        at = fill(l, at, count, grads, out, n, dtype);
        if (at < 0) return hipErrorInvalidValue;
        hipLaunchKernelGGL(grad_scale_kernel, dim3(blocks_of(l)), dim3(kThreads), 0, stream, l, part, blocks,
                           norm_in, told ? nullptr : norm_out, max_norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        told = true;
    } while (at < count);
    return hipSuccess;
}

}  // namespace bitnet
