// grad.hip -- the two gradients of a BitLinear product on gfx950 bf16 matrix cores.
//
// What they compute (straight-through quantizers: the forward is y = x~ (s w)^T with
// x~ = xq / a the dequantized activations, and both roundings pass gradients unchanged):
//   input gradient   dx[m,k] = sum_g sum_n dy_g[m,n] s_g[n] w_g[n,k]      (ternary w, packed)
//   weight gradient  dw[n,k] = sum_m dy[m,n] xq[m,k] / a[m]               (int8 codes)
//
// Both are one product C[i,j] = sum_l A[i,l] B[l,j] in which B has to be expanded from 2 or
// 8 bits, so both run on one kernel, MODE choosing the loaders:
//   MODE 0 (weight): l = m, i = n, j = k.  A = dy rows as they are; B = bf16(xq / a), exact
//          when a is a power of two.
//   MODE 1 (input):  l = n, i = m, j = k.  A = bf16(dy * s / 2); B = 2 w, exact (the scale
//          varies along l, so it has to enter before the sum; rounding dy * s once per
//          element is independent from element to element, while rounding s itself would
//          err the same way in every term of rows with nearly equal scales).
//
// Bound: matrix cores for hundreds of tokens and more, the bytes of the weights or of the
// output below that.
//
// Design:
//  * v_mfma_f32_32x32x16_bf16.  A wave owns WM x 64 outputs; 128 x 64 needs 12 KB of LDS
//    reads per 32 l against 16 KB of 64 x 64 twice over, and the LDS read rate is what a
//    64 x 64 wave tile would be bound by.  8 waves per block: (BM / WM) x (BN / 64) waves
//    for each of G groups; group g takes every G-th step of l, and the groups' sums are
//    joined through LDS at the end, so that small outputs keep large wave tiles.
//  * Operands whose contraction index is the slow one in memory (B always, A in MODE 0) lie
//    in LDS as [l][column] and are read with the transposing ds_read_b64_tr_b16: a group of
//    16 lanes reads 4 rows of 16 columns and lane t gets column t of the 4 rows.  The 32-byte
//    granules of row l are XORed with 2 (l & 3), so the four rows of a read fall in
//    different banks.
//  * Loads go through registers (B is expanded on the way): step t + 1 is loaded while step t
//    is multiplied, then converted and written to the other LDS buffer; one barrier a step.
//  * Few output tiles: l is also split over blocks (slices); every slice writes fp32 partial
//    sums to the workspace and a second launch adds them in a fixed order.
//  * Tails: rows past the end of l read as zeros through the buffer descriptors' bounds or a
//    mask; columns past i or j are computed from whatever lies there and never stored (they
//    only reach their own outputs).
#include "device_common.hpp"
#include "kernels.hpp"

namespace bitnet {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kThreads = 512;
constexpr int kWN = 64;
// high bytes of bf16(2w) by code (w = code - 1): -2, 0, +2, and 0 for the unused code
constexpr uint32_t kHi2w = 0x004000C0u;

struct GradArgs {
    const uint16_t* dy[BITNET_MAX_GROUPS];  // MODE 0: (L, I); MODE 1: (I, L[g])
    const uint8_t* b[BITNET_MAX_GROUPS];    // MODE 0: int8 (L, J); MODE 1: packed (L[g], J / 4)
    const float* scale[BITNET_MAX_GROUPS];  // MODE 0: a (L); MODE 1: s (L[g])
    int L[BITNET_MAX_GROUPS];
    int groups;
    int I, J;
    int tiles_i, tiles_j;
    int steps;   // steps of BL over all groups
    int slices;  // blocks per tile along l
    int out_dtype;
    void* out;    // (I, J)
    float* part;  // (slices, I, J) when slices > 1
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// 8 bf16 values at a 2-byte aligned offset (rows of odd length)
__device__ __forceinline__ u32x4 load8_u16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(r, off + 4 * i, 0, 0);
        const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(r, off + 4 * i + 2, 0, 0);
        v[i] = (lo & 0xFFFFu) | (hi << 16);
    }
    return v;
}

// 16 int8 codes -> 16 bf16 values c * inv (one rounding each; exact for a power of two):
// c + 128 as an unsigned byte is exact in fp32, and so is 128 inv.
__device__ __forceinline__ void codes_to_bf16(u32x4 d, float inv, u32x4 (&o)[2]) {
    const float off = -128.0f * inv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = d[i] ^ 0x80808080u;
        const float f0 = __builtin_fmaf((float)(u & 0xFFu), inv, off);
        const float f1 = __builtin_fmaf((float)((u >> 8) & 0xFFu), inv, off);
        const float f2 = __builtin_fmaf((float)((u >> 16) & 0xFFu), inv, off);
        const float f3 = __builtin_fmaf((float)(u >> 24), inv, off);
        o[i >> 1][2 * (i & 1)] = f32x2_to_bf16x2_rne(f0, f1);
        o[i >> 1][2 * (i & 1) + 1] = f32x2_to_bf16x2_rne(f2, f3);
    }
}

// 16 packed weights -> 16 bf16 values 2w in order: one lookup gives the high bytes of a
// field of all four bytes, and the low bytes of -2, 0, 2 are zero.
__device__ __forceinline__ void weights_to_bf16(uint32_t d, u32x4 (&o)[2]) {
    uint32_t hi[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
        hi[f] = __builtin_amdgcn_perm(kHi2w, kHi2w, (d >> (2 * f)) & 0x03030303u);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t sel = 0x040C000Cu + 0x01000100u * b;
        o[b >> 1][2 * (b & 1)] = __builtin_amdgcn_perm(hi[1], hi[0], sel);
        o[b >> 1][2 * (b & 1) + 1] = __builtin_amdgcn_perm(hi[3], hi[2], sel);
    }
}

// 8 bf16 values times 8 scales, rounded to bf16
__device__ __forceinline__ u32x4 scaled_bf16(u32x4 v, const float (&s)[8]) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = f32x2_to_bf16x2_rne(__uint_as_float(v[i] << 16) * s[2 * i],
                                   __uint_as_float(v[i] & 0xFFFF0000u) * s[2 * i + 1]);
    return o;
}

// Byte offset of 32-byte granule c of row l in an [l][W] bf16 tile.
template <int W>
__device__ __forceinline__ int granule(int l, int c) {
    return l * (2 * W) + ((c ^ (2 * (l & 3))) << 5);
}
// Byte offset of 16-byte chunk c of row i in an [i][BL] bf16 tile (BL = 32 or 64).
template <int BL>
__device__ __forceinline__ int chunk(int i, int c) {
    constexpr int CPR = BL / 8;
    return i * (2 * BL) + ((c ^ (CPR == 8 ? (i & 7) : ((i >> 1) & 3))) << 4);
}

template <int MODE, int BM, int BN, int WM, int G, int BL, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void grad_kernel(GradArgs p) {
    static_assert((BM / WM) * (BN / kWN) * G == 8, "8 waves");
    constexpr int TG = kThreads / G;  // threads of a group
    constexpr int NI = WM / 32, NJ = kWN / 32, KS = BL / 16;
    constexpr int kA = BM * BL * 2, kB = BN * BL * 2;  // bytes of one stage
    constexpr int kBuf = kA + kB;
    constexpr int kJoin = G > 1 ? (G / 2) * (8 / G) * WM * kWN * 4 : 0;
    constexpr int kLds = 2 * G * kBuf > kJoin ? 2 * G * kBuf : kJoin;
    static_assert(kLds <= 160 * 1024, "LDS");
    // loads of 16 bytes (A), 16 codes or 16 weights (B) per thread and step
    constexpr int kAUnits = BM * BL / 8, kBUnits = BN * BL / 16;
    constexpr int NA = (kAUnits + TG - 1) / TG, NB = (kBUnits + TG - 1) / TG;
    __shared__ __align__(1024) uint8_t lds[kLds];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int WPG = 8 / G;
    const int g = wave / WPG, wg = wave % WPG;
    const int wi = wg / (BN / kWN), wj = wg % (BN / kWN);
    const int tg = tid - g * TG;
    uint8_t* const stage = lds + 2 * g * kBuf;

    // tile of this block: consecutive blocks go to different XCDs, so each XCD gets a
    // contiguous run of tiles; runs walk panels of 8 tile rows
    const int tiles = p.tiles_i * p.tiles_j, total = tiles * p.slices;
    int t = blockIdx.x;
    {
        const int xcd = t & 7, q = total >> 3, r = total & 7;
        t = xcd * q + (xcd < r ? xcd : r) + (t >> 3);
    }
    const int slice = t / tiles;
    t -= slice * tiles;
    constexpr int kPanel = 4;
    const int panel = t / (kPanel * p.tiles_j);
    const int ph = p.tiles_i - panel * kPanel < kPanel ? p.tiles_i - panel * kPanel : kPanel;
    const int tp = t - panel * kPanel * p.tiles_j;
    const int ti = panel * kPanel + tp % ph, tj = tp / ph;
    const int i0 = ti * BM, j0 = tj * BN;
    const int I = p.I, J = p.J;

    // steps of this block: [s0, s1), group g takes s0 + g, s0 + g + G, ...
    const int s0 = (int)((int64_t)p.steps * slice / p.slices);
    const int s1 = (int)((int64_t)p.steps * (slice + 1) / p.slices);
    const int nsteps = (s1 - s0 + G - 1) / G;

    u32x4 ra[NA];
    u32x4 rb[NB];   // MODE 0: 16 codes
    uint32_t rw[NB];  // MODE 1: 16 weights
    float rs[MODE == 0 ? NB : 8];

    auto load = [&](int it) {
        int s = s0 + g + G * it;
        if constexpr (MODE == 0) {
            const int l0 = s < s1 ? s * BL : p.L[0];
            const int rows = p.L[0] - l0 < BL ? p.L[0] - l0 : BL;
            const __amdgpu_buffer_rsrc_t ar =
                rsrc(p.dy[0] + (int64_t)l0 * I + i0, ((int64_t)rows * I - i0) * 2);
            const __amdgpu_buffer_rsrc_t br =
                rsrc(p.b[0] + (int64_t)l0 * J + j0, (int64_t)rows * J - j0);
            const __amdgpu_buffer_rsrc_t sr = rsrc(p.scale[0] + l0, (int64_t)rows * 4);
#pragma unroll
            for (int n = 0; n < NA; ++n) {
                const int id = tg + n * TG, l = id / (BM / 8), c = id % (BM / 8);
                const uint32_t off = (uint32_t)(l * I + 8 * c) * 2;
                ra[n] = ALIGNED ? load16(ar, off) : load8_u16(ar, off);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int id = tg + n * TG, l = id / (BN / 16), c = id % (BN / 16);
                rb[n] = load16(br, (uint32_t)(l * J + 16 * c));
                rs[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(sr, 4 * l, 0, 0));
            }
        } else {
            int q = 0;
            if (s >= s1) {
                q = p.groups;
            } else {
                while (s >= (p.L[q] + BL - 1) / BL) s -= (p.L[q++] + BL - 1) / BL;
            }
            const bool live = q < p.groups;
            if (!live) q = 0;
            const int L = p.L[q];
            const int l0 = live ? s * BL : L;
            const int cols = L - l0 < BL ? L - l0 : BL;
            const int row_bytes = J / 4;
            const __amdgpu_buffer_rsrc_t ar =
                rsrc(p.dy[q] + (int64_t)i0 * L, live ? (int64_t)(I - i0 < BM ? I - i0 : BM) * L * 2 : 0);
            const __amdgpu_buffer_rsrc_t br =
                rsrc(p.b[q] + (int64_t)l0 * row_bytes + j0 / 4, (int64_t)cols * row_bytes - j0 / 4);
            const __amdgpu_buffer_rsrc_t sr = rsrc(p.scale[q] + l0, (int64_t)cols * 4);
            {
                const int c = tg % (BL / 8);
                const u32x4 a0 = load16(sr, 32 * c), a1 = load16(sr, 32 * c + 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    rs[e] = 0.5f * __uint_as_float(a0[e]);
                    rs[4 + e] = 0.5f * __uint_as_float(a1[e]);
                }
            }
#pragma unroll
            for (int n = 0; n < NA; ++n) {
                const int id = tg + n * TG, i = id / (BL / 8), c = id % (BL / 8);
                const uint32_t off = (uint32_t)(i * L + l0 + 8 * c) * 2;
                if (kAUnits % TG == 0 || id < kAUnits) ra[n] = ALIGNED ? load16(ar, off) : load8_u16(ar, off);
                if (cols < BL) {  // the last step of a group: columns past the end are zero
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (8 * c + 2 * e >= cols) ra[n][e] = 0u;
                        else if (8 * c + 2 * e + 1 >= cols) ra[n][e] &= 0xFFFFu;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int id = tg + n * TG, l = id / (BN / 16), c = id % (BN / 16);
                const uint32_t off = (uint32_t)(l * row_bytes + 4 * c);
                if (ALIGNED) {
                    rw[n] = __builtin_amdgcn_raw_buffer_load_b32(br, off, 0, 0);
                } else {
                    uint32_t d = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        d |= ((uint32_t)__builtin_amdgcn_raw_buffer_load_b8(br, off + e, 0, 0) & 0xFFu) << (8 * e);
                    rw[n] = d;
                }
            }
        }
    };

    auto store = [&](int it, int buf) {
        uint8_t* const A = stage + buf * kBuf;
        uint8_t* const B = A + kA;
        if constexpr (MODE == 0) {
            const int s = s0 + g + G * it;
            const int rows = s < s1 ? p.L[0] - s * BL : 0;
#pragma unroll
            for (int n = 0; n < NA; ++n) {
                const int id = tg + n * TG, l = id / (BM / 8), c = id % (BM / 8);
                *reinterpret_cast<u32x4*>(A + granule<BM>(l, c >> 1) + 16 * (c & 1)) = ra[n];
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int id = tg + n * TG, l = id / (BN / 16), c = id % (BN / 16);
                u32x4 o[2];
                codes_to_bf16(rb[n], l < rows ? 1.0f / rs[n] : 0.0f, o);
                u32x4* const dst = reinterpret_cast<u32x4*>(B + granule<BN>(l, c));
                dst[0] = o[0];
                dst[1] = o[1];
            }
        } else {
#pragma unroll
            for (int n = 0; n < NA; ++n) {
                const int id = tg + n * TG, i = id / (BL / 8), c = id % (BL / 8);
                if (kAUnits % TG == 0 || id < kAUnits)
                    *reinterpret_cast<u32x4*>(A + chunk<BL>(i, c)) = scaled_bf16(ra[n], rs);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int id = tg + n * TG, l = id / (BN / 16), c = id % (BN / 16);
                u32x4 o[2];
                weights_to_bf16(rw[n], o);
                u32x4* const dst = reinterpret_cast<u32x4*>(B + granule<BN>(l, c));
                dst[0] = o[0];
                dst[1] = o[1];
            }
        }
    };

    f32x16 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // lane's part of a transposed read: row 8 (lane / 32) + (t / 4) of a 16-row step, 8 bytes
    // t % 4 of the granule of its 16 columns
    const int t16 = lane & 15, half = (lane >> 4) & 1, l8 = 8 * (lane >> 5) + (t16 >> 2);
    auto tr_read = [&](const uint8_t* tile, int off, int row_bytes) {
        const uint8_t* a = tile + off;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * row_bytes));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, v);
    };
    int offA[NI], offB[NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if constexpr (MODE == 0)
            offA[i] = granule<BM>(l8, (wi * WM + 32 * i) / 16 + half) + 8 * (t16 & 3);
        else
            offA[i] = 0;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        offB[j] = granule<BN>(l8, (wj * kWN + 32 * j) / 16 + half) + 8 * (t16 & 3);

    auto multiply = [&](int buf) {
        const uint8_t* const A = stage + buf * kBuf;
        const uint8_t* const B = A + kA;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            bf16x8 a[NI], b[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) b[j] = tr_read(B, offB[j] + ks * 16 * 2 * BN, 2 * BN);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                if constexpr (MODE == 0)
                    a[i] = tr_read(A, offA[i] + ks * 16 * 2 * BM, 2 * BM);
                else
                    a[i] = *reinterpret_cast<const bf16x8*>(
                        A + chunk<BL>(wi * WM + 32 * i + (lane & 31), 2 * ks + (lane >> 5)));
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    };

    if (nsteps > 0) {
        load(0);
        store(0, 0);
    }
    __syncthreads();
    for (int it = 0; it < nsteps; ++it) {
        const bool more = it + 1 < nsteps;
        if (more) load(it + 1);
        multiply(it & 1);
        if (more) store(it + 1, (it + 1) & 1);
        __syncthreads();
    }

    // join the groups: the upper half of the remaining groups hands its sums to the lower
    if (G > 1) {
        float* const x = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int h = G / 2; h >= 1; h /= 2) {
            if (g >= h && g < 2 * h) {
                float* const w = x + ((g - h) * WPG + wg) * (WM * kWN) + lane;
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r) w[((i * NJ + j) * 16 + r) * 64] = acc[i][j][r];
            }
            __syncthreads();
            if (g < h) {
                const float* const w = x + (g * WPG + wg) * (WM * kWN) + lane;
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[i][j][r] += w[((i * NJ + j) * 16 + r) * 64];
            }
            __syncthreads();
        }
        if (g > 0) return;
    }

    // lane l, register r of a 32x32 accumulator: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int col = j0 + wj * kWN + 32 * j + (lane & 31);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = i0 + wi * WM + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (row < I && col < J) {
                    const int64_t o = (int64_t)row * J + col;
                    if (p.slices > 1)
                        p.part[(int64_t)slice * I * J + o] = acc[i][j][r];
                    else if (p.out_dtype == BITNET_OUT_F32)
                        static_cast<float*>(p.out)[o] = acc[i][j][r];
                    else
                        static_cast<uint16_t*>(p.out)[o] = f32_to_bf16_rne(acc[i][j][r]);
                }
            }
        }
}

// Sum of the slices' partials, in order; four outputs a thread (J % 4 == 0).
__global__ __launch_bounds__(256) void grad_join_kernel(const float* __restrict__ part, int slices,
                                                        int64_t n, int out_dtype, void* out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    float4 s = *reinterpret_cast<const float4*>(part + i);
    for (int k = 1; k < slices; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(part + k * n + i);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    if (out_dtype == BITNET_OUT_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = s;
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) =
            make_uint2(f32x2_to_bf16x2_rne(s.x, s.y), f32x2_to_bf16x2_rne(s.z, s.w));
}

// ------------------------------------------------------------------------------ plan
struct GradPlan {
    int cfg, slices, steps;
};
struct GradCfg {
    int bm, bn, wm, g, bl;
};
constexpr GradCfg kCfg[] = {{256, 256, 128, 1, 64}, {256, 128, 128, 2, 32}, {128, 128, 128, 4, 32}, {32, 256, 32, 2, 32}};

GradPlan plan(int mode, int64_t I, int64_t J, const int64_t* L, int groups) {
    GradPlan best = {0, 1, 0};
    double best_t = 1e300;
    for (int c = 0; c < 4; ++c) {
        const GradCfg& k = kCfg[c];
        if (mode == 0 && c == 3) continue;
        int64_t steps = 0;
        for (int q = 0; q < groups; ++q) steps += (L[q] + k.bl - 1) / k.bl;
        const int64_t tiles = ((I + k.bm - 1) / k.bm) * ((J + k.bn - 1) / k.bn);
        for (int64_t s = 1; s <= 32; ++s) {
            if (s > 1 && (steps < 2 * s * k.g || s * I * J * 4 > ((int64_t)64 << 20))) break;
            const int64_t rounds = (tiles * s + 255) / 256;
            const int64_t per = ((steps + s - 1) / s + k.g - 1) / k.g;  // steps of a group
            // a step costs its matrix products (8 waves at about half of the peak rate) or a
            // fixed latency; a block its prologue and epilogue; a join its bytes
            const double step_us = 0.45 * k.bl / 32.0 * (k.wm / 128.0) + 0.35;
            const double t = rounds * (per * step_us + 3.0 + k.wm / 64.0) +
                             (s > 1 ? 3.0 + (s + 1) * I * J * 4.0 / 3e6 : 0.0);
            if (t < best_t) {
                best_t = t;
                best = {c, (int)s, (int)steps};
            }
        }
    }
    return best;
}

template <int MODE, int C>
void launch_cfg(const GradArgs& a, bool aligned, hipStream_t stream) {
    constexpr GradCfg k = kCfg[C];
    const dim3 grid((unsigned)((int64_t)a.tiles_i * a.tiles_j * a.slices)), block(kThreads);
    if (aligned)
        hipLaunchKernelGGL((grad_kernel<MODE, k.bm, k.bn, k.wm, k.g, k.bl, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((grad_kernel<MODE, k.bm, k.bn, k.wm, k.g, k.bl, false>), grid, block, 0, stream, a);
}

hipError_t launch_grad(int mode, GradArgs a, const int64_t* L, bool aligned, void* workspace,
                       size_t ws_bytes, hipStream_t stream) {
    const int64_t n = (int64_t)a.I * a.J;
    GradPlan pl = plan(mode, a.I, a.J, L, a.groups);
    if ((size_t)pl.slices * n * 4 > ws_bytes) pl.slices = 1;
    const GradCfg& k = kCfg[pl.cfg];
    const int64_t ti = (a.I + k.bm - 1) / k.bm, tj = (a.J + k.bn - 1) / k.bn;
    if (ti * tj * pl.slices > INT32_MAX / 8) return hipErrorInvalidValue;
    a.tiles_i = (int)ti;
    a.tiles_j = (int)tj;
    a.steps = pl.steps;
    a.slices = pl.slices;
    a.part = static_cast<float*>(workspace);
    if (mode == 0) {
        if (pl.cfg == 0) launch_cfg<0, 0>(a, aligned, stream);
        else if (pl.cfg == 1) launch_cfg<0, 1>(a, aligned, stream);
        else launch_cfg<0, 2>(a, aligned, stream);
    } else {
        if (pl.cfg == 0) launch_cfg<1, 0>(a, aligned, stream);
        else if (pl.cfg == 1) launch_cfg<1, 1>(a, aligned, stream);
        else if (pl.cfg == 2) launch_cfg<1, 2>(a, aligned, stream);
        else launch_cfg<1, 3>(a, aligned, stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || pl.slices == 1) return e;
    hipLaunchKernelGGL(grad_join_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream,
                       a.part, a.slices, n, a.out_dtype, a.out);
    return hipGetLastError();
}

}  // namespace

void grad_plan(int mode, int64_t I, int64_t J, const int64_t* L, int groups, int* out) {
    const GradPlan pl = plan(mode, I, J, L, groups);
    const GradCfg& k = kCfg[pl.cfg];
    out[0] = k.bm;
    out[1] = k.bn;
    out[2] = k.g;
    out[3] = pl.slices;
}

size_t grad_input_workspace_size(int64_t M, int64_t K, int groups, const int64_t* N) {
    const GradPlan pl = plan(1, M, K, N, groups);
    return pl.slices > 1 ? (size_t)pl.slices * M * K * 4 : 0;
}

size_t grad_weight_workspace_size(int64_t M, int64_t N, int64_t K) {
    const GradPlan pl = plan(0, N, K, &M, 1);
    return pl.slices > 1 ? (size_t)pl.slices * N * K * 4 : 0;
}

hipError_t launch_grad_input(const uint16_t* const* dy, const uint8_t* const* packed,
                             const float* const* w_scale, const int64_t* N, int groups, int64_t M,
                             int64_t K, uint16_t* dx, void* workspace, size_t ws_bytes,
                             hipStream_t stream) {
    GradArgs a = {};
    int64_t L[BITNET_MAX_GROUPS];
    bool aligned = K % 16 == 0;
    for (int q = 0; q < groups; ++q) {
        if (N[q] == 0) continue;  // adds nothing
        a.dy[a.groups] = dy[q];
        a.b[a.groups] = packed[q];
        a.scale[a.groups] = w_scale[q];
        a.L[a.groups] = (int)N[q];
        L[a.groups++] = N[q];
        aligned = aligned && N[q] % 2 == 0;
    }
    a.I = (int)M;
    a.J = (int)K;
    a.out = dx;
    a.out_dtype = BITNET_OUT_BF16;
    return launch_grad(1, a, L, aligned, workspace, ws_bytes, stream);
}

hipError_t launch_grad_weight(const uint16_t* dy, const int8_t* xq, const float* a_scale, int64_t M,
                              int64_t N, int64_t K, void* dw, int out_dtype, void* workspace,
                              size_t ws_bytes, hipStream_t stream) {
    GradArgs a = {};
    a.dy[0] = dy;
    a.b[0] = reinterpret_cast<const uint8_t*>(xq);
    a.scale[0] = a_scale;
    a.L[0] = (int)M;
    a.groups = 1;
    a.I = (int)N;
    a.J = (int)K;
    a.out = dw;
    a.out_dtype = out_dtype;
    return launch_grad(0, a, &M, N % 2 == 0, workspace, ws_bytes, stream);
}

}  // namespace bitnet
