// glu.hip -- SwiGLU for training on gfx950: forward with 8-bit codes of its output and 8-bit
// checkpoints of its inputs, backward from the checkpoints or from bf16 inputs.
//
//   forward   h = silu(g) u, silu(g) = g sig(g), sig(g) = 1 / (1 + exp(-g))
//   backward  dg = dh u sig(g) (1 + g (1 - sig(g))),  du = dh g sig(g)
// All in fp32, each output rounded once.
//
// Bound by HBM.  Forward: the scales of a row need its maxima before any code is written, so
// a row is held in the registers of WPR waves (up to four groups of V elements of g, u and h
// per lane), all loads issued together, the maxima of g, u and h reduced behind one barrier;
// longer rows are read again from cache.  Backward: no row reduction, V elements a thread.
// Measured, inputs out of cache: 2048 x 14336 forward with checkpoints 40 us, 5.9 TB/s, backward
// from them 36.8 us, 6.4 TB/s, from bf16 43.8 us, 6.7 TB/s (a copy: 5.3); 32768 x 2560 138, 136 and
// 169 us, 4.9 to 5.0 TB/s; 4096 x 28672 (16 waves, seven registers in scratch) 184, 161 and 203 us,
// 5.1 to 5.8 TB/s.
#include "device_common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace bitnet {

namespace {

struct GluArgs {
    const uint16_t *g, *u;
    int64_t M, N;
    uint16_t* h;  // NULL: not written
    int8_t *hq, *gq, *uq;  // NULL: not wanted
    float *h_scale, *g_scale, *u_scale;
    int h_pow2;
};

__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-g));  // exp -> inf gives 0
}

template <int V>
__device__ __forceinline__ RowVec<V> swiglu_vec(const RowVec<V>& g, const RowVec<V>& u) {
    float a[V], b[V];
    to_f32<V>(g, a);
    to_f32<V>(u, b);
    RowVec<V> h;
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
        h.w[j] = f32x2_to_bf16x2_rne(a[2 * j] * sigmoid(a[2 * j]) * b[2 * j],
                                     a[2 * j + 1] * sigmoid(a[2 * j + 1]) * b[2 * j + 1]);
    return h;
}

// G == 0: rows longer than the registers hold.
template <int V, int WPR, int G>
__global__ __launch_bounds__(64 * WPR) void swiglu_kernel(GluArgs p) {
    constexpr int kStride = 64 * WPR, H = G > 0 ? G : 1;
    __shared__ uint32_t s_max[2][WPR][3];
    const int64_t groups = p.N / V;
    const bool codes = p.hq || p.gq;
    int parity = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, parity ^= 1) {
        const int64_t row = m * p.N;
        RowVec<V> g[H], u[H], h[H];
        uint32_t mg = 0, mu = 0, mh = 0;
        if (G > 0) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int64_t q = threadIdx.x + (int64_t)i * kStride;
                g[i] = u[i] = zero_row_vec<V>();
                if (q < groups) {
                    g[i] = load_row_vec<V>(p.g + row, q);
                    u[i] = load_row_vec<V>(p.u + row, q);
                }
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int64_t q = threadIdx.x + (int64_t)i * kStride;
                h[i] = swiglu_vec<V>(g[i], u[i]);
                if (p.h && q < groups) store_row_vec<V>(p.h + row, q, h[i]);
                mg = max_pairs<V>(g[i], mg);
                mu = max_pairs<V>(u[i], mu);
                mh = max_pairs<V>(h[i], mh);
            }
        } else {
            for (int64_t q = threadIdx.x; q < groups; q += kStride) {
                g[0] = load_row_vec<V>(p.g + row, q);
                u[0] = load_row_vec<V>(p.u + row, q);
                h[0] = swiglu_vec<V>(g[0], u[0]);
                if (p.h) store_row_vec<V>(p.h + row, q, h[0]);
                mg = max_pairs<V>(g[0], mg);
                mu = max_pairs<V>(u[0], mu);
                mh = max_pairs<V>(h[0], mh);
            }
        }
        if (!codes) continue;
        mg = wave_max_u32(max_of_pair(mg));
        mu = wave_max_u32(max_of_pair(mu));
        mh = wave_max_u32(max_of_pair(mh));
        if (WPR > 1) {
            // the slots of row m are written again two rows later, behind the next row's barrier
            uint32_t(&s)[WPR][3] = s_max[parity];
            if ((threadIdx.x & 63) == 0) {
                s[threadIdx.x >> 6][0] = mg;
                s[threadIdx.x >> 6][1] = mu;
                s[threadIdx.x >> 6][2] = mh;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                mg = max(mg, s[i][0]);
                mu = max(mu, s[i][1]);
                mh = max(mh, s[i][2]);
            }
        }
        const float ag = pow2_scale(mg), au = pow2_scale(mu), ah = scale_of(mh, p.h_pow2);
        if (threadIdx.x == 0) {
            if (p.gq) {
                p.g_scale[m] = ag;
                p.u_scale[m] = au;
            }
            if (p.hq) p.h_scale[m] = ah;
        }
        with_clamp(max(max(mg, mu), mh), [&](auto clamp) {
            constexpr bool C = decltype(clamp)::value;
            auto store = [&](int64_t q, const RowVec<V>& gv, const RowVec<V>& uv, const RowVec<V>& hv) {
                if (p.gq) {
                    store_codes<V, C>(p.gq + row, q, gv, ag);
                    store_codes<V, C>(p.uq + row, q, uv, au);
                }
                if (p.hq) store_codes<V, C>(p.hq + row, q, hv, ah);
            };
            if (G > 0) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int64_t q = threadIdx.x + (int64_t)i * kStride;
                    if (q < groups) store(q, g[i], u[i], h[i]);
                }
            } else {
                for (int64_t q = threadIdx.x; q < groups; q += kStride) {
                    g[0] = load_row_vec<V>(p.g + row, q);
                    u[0] = load_row_vec<V>(p.u + row, q);
                    store(q, g[0], u[0], swiglu_vec<V>(g[0], u[0]));
                }
            }
        });
    }
}

struct GluBackArgs {
    const uint16_t* dh;
    const void *g, *u;                // bf16, or int8 codes with scales
    const float *g_scale, *u_scale;   // NULL: bf16
    int64_t groups, blocks_per_row;
    uint16_t *dg, *du;
};

template <int V, bool CODES>
__global__ __launch_bounds__(256) void swiglu_back_kernel(GluBackArgs p) {
    const int64_t m = blockIdx.x / p.blocks_per_row;
    const int64_t q = (blockIdx.x - m * p.blocks_per_row) * 256 + threadIdx.x;
    if (q >= p.groups) return;
    const int64_t row = m * p.groups * V;
    float d[V], g[V], u[V];
    to_f32<V>(load_row_vec<V>(p.dh + row, q), d);
    if constexpr (CODES) {
        const float ig = 1.0f / p.g_scale[m], iu = 1.0f / p.u_scale[m];
        const uint32_t* gp = reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(p.g) + row) + q * (V / 4);
        const uint32_t* up = reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(p.u) + row) + q * (V / 4);
        uint32_t gw[V / 4], uw[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            gw[i] = gp[i];
            uw[i] = up[i];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            g[j] = (float)(int8_t)(gw[j / 4] >> (8 * (j & 3))) * ig;
            u[j] = (float)(int8_t)(uw[j / 4] >> (8 * (j & 3))) * iu;
        }
    } else {
        to_f32<V>(load_row_vec<V>(static_cast<const uint16_t*>(p.g) + row, q), g);
        to_f32<V>(load_row_vec<V>(static_cast<const uint16_t*>(p.u) + row, q), u);
    }
    RowVec<V> a, b;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
        float dg[2], du[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = 2 * j + e;
            const float s = sigmoid(g[k]);
            dg[e] = d[k] * u[k] * (s * __builtin_fmaf(g[k], 1.0f - s, 1.0f));
            du[e] = d[k] * (g[k] * s);
        }
        a.w[j] = f32x2_to_bf16x2_rne(dg[0], dg[1]);
        b.w[j] = f32x2_to_bf16x2_rne(du[0], du[1]);
    }
    store_row_vec<V>(p.dg + row, q, a);
    store_row_vec<V>(p.du + row, q, b);
}

template <int V>
hipError_t launch_swiglu_v(const GluArgs& a, hipStream_t stream) {
    const int64_t lanes = (a.N / V + 3) / 4;  // lanes that hold a row in four groups each
    const unsigned rows = (unsigned)(a.M < 8192 ? a.M : 8192);
    if (lanes <= 64)
        hipLaunchKernelGGL((swiglu_kernel<V, 1, 4>), dim3(rows), dim3(64), 0, stream, a);
    else if (lanes <= 256)
        hipLaunchKernelGGL((swiglu_kernel<V, 4, 4>), dim3(rows), dim3(256), 0, stream, a);
    else if (lanes <= 512)
        hipLaunchKernelGGL((swiglu_kernel<V, 8, 4>), dim3(rows), dim3(512), 0, stream, a);
    else if (lanes <= 1024)
        hipLaunchKernelGGL((swiglu_kernel<V, 16, 4>), dim3(rows), dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((swiglu_kernel<V, 16, 0>), dim3(rows), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* g, const uint16_t* u, int64_t M, int64_t N, uint16_t* h,
                         int8_t* hq, float* h_scale, int h_pow2, int8_t* gq, float* g_scale,
                         int8_t* uq, float* u_scale, hipStream_t stream) {
    const GluArgs a = {g, u, M, N, h, hq, gq, uq, h_scale, g_scale, u_scale, h_pow2};
    return N % 8 == 0 ? launch_swiglu_v<8>(a, stream) : launch_swiglu_v<4>(a, stream);
}

hipError_t launch_swiglu_back(const uint16_t* dh, const void* g, const float* g_scale, const void* u,
                              const float* u_scale, int64_t M, int64_t N, uint16_t* dg, uint16_t* du,
                              hipStream_t stream) {
    const int64_t groups = N / (N % 8 == 0 ? 8 : 4), bpr = (groups + 255) / 256;
    const int64_t step = max_blocks(256) / bpr;  // rows of a launch
    const int64_t size = g_scale ? 1 : 2;        // bytes of an element of g and u
    for (int64_t m = 0; m < M; m += step) {
        const GluBackArgs a = {dh + m * N,
                               static_cast<const uint8_t*>(g) + m * N * size,
                               static_cast<const uint8_t*>(u) + m * N * size,
                               g_scale ? g_scale + m : nullptr,
                               u_scale ? u_scale + m : nullptr,
                               groups,
                               bpr,
                               dg + m * N,
                               du + m * N};
        const dim3 grid((unsigned)((M - m < step ? M - m : step) * bpr)), block(256);
        if (N % 8 == 0) {
            if (g_scale) hipLaunchKernelGGL((swiglu_back_kernel<8, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((swiglu_back_kernel<8, false>), grid, block, 0, stream, a);
        } else {
            if (g_scale) hipLaunchKernelGGL((swiglu_back_kernel<4, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((swiglu_back_kernel<4, false>), grid, block, 0, stream, a);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bitnet
