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
//   MODE 1 (input):  l = n, i = m, j = k.  A = bf16(dy * s); B = 2 w, exact, and the sum
//          is halved at the end (the scale varies along l, so it has to enter before the sum;
//          rounding dy * s once per element is independent from element to element, while
//          rounding s itself would err the same way in every term of rows with nearly equal
//          scales).
//
// Bound: matrix cores for hundreds of tokens and more, the bytes of the weights or of the
// output below that.
//
// Design:
//  * v_mfma_f32_32x32x16_bf16; a wave owns WM x WN outputs, (BM / WM) x (BN / WN) waves make a
//    group, and G groups share a tile: group g takes every G-th step of BL values of l, and
//    the groups' sums are joined through LDS at the end (in halves, a fixed order), so that
//    small outputs keep the chip busy with large wave tiles.
//  * Operands whose contraction index is the slow one in memory lie in LDS as [l][column] and
//    are read transposed: bf16 rows (MODE 0) with ds_read_b64_tr_b16 (a group of 16 lanes reads
//    4 rows of 16 columns, lane t gets column t), packed weights (MODE 1) as they are, 2 bits
//    each, with ds_read_b64_tr_b8 (8 rows of 16 bytes, lane t gets byte column t: four weights
//    of each of 8 rows), expanded in registers by byte lookups.  Rows are XOR-swizzled so that
//    the rows of a read fall in different banks.
//  * Loads go through registers, since one operand is converted on the way.  Every matrix
//    instruction is a slot that also carries its share of the conversion (see the main loop);
//    descriptors move on by scalar adds, because the instruction issue of a wave counts: 129
//    scalar instructions a step cost 8% at 8192^3.
//  * Few output tiles: l is also split over blocks (slices); every slice writes fp32 partial
//    sums to the workspace and a second launch adds them in a fixed order.
//  * Tails: what lies past the end of l reads as zeros through the buffer descriptors' bounds
//    or a mask.  Rows that start off a dword are put together from the dwords around them; the
//    last of these may hold one value more than the tensor, which must not enter as the start
//    of the next row (a zero in the other operand is not enough, 0 x NaN is NaN): see Rows.
//    Columns past i or j are computed from whatever lies there and never stored (they only
//    reach their own outputs).
// Measured in one run (bf16 out; beside it a library's bf16 product, 1399 TFLOP/s at 8192^3 and
// 1223 on a transposed left operand like dw's): dx 8192^3 806 us, 1364 TFLOP/s, the matrix cores
// busy 58% of the cycles at 4096^3 (the chip holds about 1.8 GHz under such a load, where the peak
// is 1.9 PFLOP/s); dw 8192^3 884 us, 1244 TFLOP/s, busy 55%: both operands of dw are read
// transposed as bf16, 192 KB of LDS reads a step against 132 KB.  What is left is the vector
// instructions of the conversion, which the matrix instructions hide in part.
// One token to dozens: dx 4 x 2560 x 2560 6.1 us and 3.1 for the join (medians, from HBM), launch
// and latency; 512 x 3840 x 2560 24 us against 7.3 at the rate of a large product: 160 tiles on
// 256 CUs, one block on each, and a chain of 30 short steps.  dw 512 x 6912 x 2560 fp32 33 to 36 us
// against 16.3 for its 79 MB: 1080 tiles on 1024 places leave a last round of 56 (the kernel is
// held to 128 registers for them and keeps up to six in scratch).
#include <cmath>
#include <type_traits>
#include <utility>

#include "device_common.hpp"
#include "kernels.hpp"

namespace bitnet {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

// high bytes of bf16(2w) by code (w = code - 1): -2, 0, +2, and 0 for the unused code
constexpr uint32_t kHi2w = 0x004000C0u;

// How the rows of an operand lie.  kOddEnd: kOdd with an odd number of rows in a single column
// of tiles (MODE 0), where the tile that needs the last row's half dword also has the column
// that the other half would enter; there the rows past the end are masked by their number.
// (Masking wherever rows are odd took registers: dw 512 x 6911 x 2560 46 -> 60 us.)
enum Rows { kWhole, kOdd, kOddEnd };

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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes > 0 ? bytes : 0,
                                             0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// 8 bf16 values at a 2-byte aligned offset (rows of odd length): the aligned dwords around
// them, shifted together.  The descriptors end on a whole dword.
__device__ __forceinline__ u32x4 load8_half(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff) {
    const u32x4 v =
        __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off & ~3u, soff, 0));
    const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(r, (off & ~3u) + 16, soff, 0);
    const uint32_t sh = 8 * (off & 2);
    u32x4 o;
    o[0] = __builtin_amdgcn_alignbit(v[1], v[0], sh);
    o[1] = __builtin_amdgcn_alignbit(v[2], v[1], sh);
    o[2] = __builtin_amdgcn_alignbit(v[3], v[2], sh);
    o[3] = __builtin_amdgcn_alignbit(x, v[3], sh);
    return o;
}

// Byte offset of 32-byte granule c of row l in an [l][W] bf16 tile.
template <int W>
__device__ __forceinline__ int granule(int l, int c) {
    return l * (2 * W) + ((c ^ (2 * (l & 3))) << 5);
}
// Byte offset of 16-byte column c of row l in an [l][W / 4] tile of packed weights.
template <int W>
__device__ __forceinline__ int packed_at(int l, int c) {
    return l * (W / 4) + ((c ^ ((l >> 2) & (W / 64 - 1))) << 4);
}
// Byte offset of 16-byte chunk c of row i in an [i][BL] bf16 tile (BL = 32 or 64).
template <int BL>
__device__ __forceinline__ int chunk(int i, int c) {
    constexpr int CPR = BL / 8;
    return i * (2 * BL) + ((c ^ (CPR == 8 ? (i & 7) : ((i >> 1) & 3))) << 4);
}

template <int MODE, int BM, int BN, int WM, int WN, int G, int BL, int D, int W, Rows ROWS>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN) * G, W) void grad_kernel(GradArgs p) {
    constexpr int WPG = (BM / WM) * (BN / WN);  // waves of a group
    constexpr int TG = 64 * WPG;                // threads of a group
    constexpr bool ALIGNED = ROWS == kWhole;
    constexpr int NI = WM / 32, NJ = WN / 32, KS = BL / 16;
    constexpr int kBRow = MODE == 0 ? 2 * BN : BN / 4;   // bytes of a row of B in LDS
    constexpr int kA = BM * BL * 2, kB = kBRow * BL;      // bytes of one stage
    constexpr int kBuf = kA + kB;
    constexpr int kJoin = G > 1 ? (G / 2) * WPG * WM * WN * 4 : 0;
    constexpr int kLds = 2 * G * kBuf > kJoin ? 2 * G * kBuf : kJoin;
    static_assert(kLds <= 160 * 1024, "LDS");
    static_assert(WN == 64, "a wave's 64 columns are 16 byte columns of packed weights");
    static_assert(KS % 2 == 0, "operand sets alternate");
    // 16-byte loads of A, 16 codes or 16 weights of B per thread and step
    constexpr int kAUnits = BM * BL / 8, kBUnits = BN * BL / 16;
    constexpr int NA = (kAUnits + TG - 1) / TG, NB = (kBUnits + TG - 1) / TG;
    constexpr bool kAFull = kAUnits % TG == 0;
    static_assert(kBUnits % TG == 0, "B units");
    static_assert(TG % (BL / 8) == 0, "a thread keeps its chunk column");
    __shared__ __align__(1024) uint8_t lds[kLds];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = wave / WPG, wg = wave % WPG;
    const int wi = wg / (BN / WN), wj = wg % (BN / WN);
    const int tg = tid - g * TG;
    uint8_t* const stage = lds + 2 * g * kBuf;

    // tile of this block: consecutive blocks go to different XCDs, so each XCD gets a
    // contiguous run of tiles; runs walk panels of kPanel tile rows
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

    // steps of this block: [s0, s1), group g takes s0 + g, s0 + g + G, ...; every group runs
    // nsteps steps and multiplies zeros past its last one
    const int s0 = (int)((int64_t)p.steps * slice / p.slices);
    const int s1 = (int)((int64_t)p.steps * (slice + 1) / p.slices);
    const int nsteps = (s1 - s0 + G - 1) / G;

    // ---- loads: the step to load next ----
    // Its descriptors move on by scalar adds.  left: rows (MODE 0) or columns (MODE 1) of l from
    // the step's start to the end of what the block sums of them; at or below zero past the
    // end, where the descriptors are empty and read as zeros.
    int left, end;  // MODE 1: end of the block's share, from the start of group q (padded)
    int l0 = (s0 + g) * BL, q = 0, L = p.L[0];
    const int row_bytes = J / 4;
    const int rows_a = I - i0 < BM ? I - i0 : BM;  // MODE 1
    const int step_l = G * BL;
    const uint8_t *pa, *pb, *ps;
    uint32_t voff_a[NA], voff_b[NB];
    auto padded = [](int l) { return (l + BL - 1) / BL * BL; };
    // The last element of rows at odd places may lie in the lower half of a dword.  The
    // descriptor covers that dword for the tiles that hold the last column; in MODE 0 it ends
    // before it for the others, of which the first has the column behind the last element.
    const int up = MODE == 1 || i0 + BM >= I ? 3 : 0;
    auto whole = [&](int bytes) { return ALIGNED ? bytes : (bytes + up) & ~3; };
    auto enter = [&]() {  // at l0 of group q
        const int stop = L < end ? L : end;
        left = stop - l0;
        pa = reinterpret_cast<const uint8_t*>(
            p.dy[q] + (MODE == 0 ? (int64_t)l0 * I + i0 : (int64_t)i0 * L));
        pb = p.b[q] + (MODE == 0 ? (int64_t)l0 * J + j0 : (int64_t)l0 * row_bytes + j0 / 4);
        ps = reinterpret_cast<const uint8_t*>(p.scale[q] + l0);
#pragma unroll
        for (int n = 0; n < NA; ++n) {
            const int id = tg + n * TG;
            if constexpr (MODE == 0)
                voff_a[n] = (uint32_t)(id / (BM / 8) * I + 8 * (id % (BM / 8))) * 2;
            else
                voff_a[n] = kAFull || id < kAUnits
                                ? (uint32_t)(id / (BL / 8) * L + 8 * (id % (BL / 8))) * 2
                                : 0x80000000u;
        }
    };
    end = s1 * BL;
    if constexpr (MODE == 1) {
        while (q + 1 < p.groups && l0 >= padded(L)) {
            l0 -= padded(L);
            end -= padded(L);
            L = p.L[++q];
        }
    }
    enter();
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int id = tg + n * TG, l = id / (BN / 16), c = id % (BN / 16);
        voff_b[n] = MODE == 0 ? (uint32_t)(l * J + 16 * c) : (uint32_t)(l * row_bytes + 4 * c);
    }
    __amdgpu_buffer_rsrc_t ra, rb, rs;
    auto describe = [&]() {
        // sizes of at most 256 rows of 2^20 elements: 32 bits hold them
        const bool live = left > 0;
        const int rows = left < BL ? left : BL;
        if constexpr (MODE == 0) {
            ra = rsrc(pa, live ? whole((rows * I - i0) * 2) : 0);
            rb = rsrc(pb, live ? rows * J - j0 : 0);
        } else {
            ra = rsrc(pa, live ? whole(rows_a * L * 2) : 0);
            rb = rsrc(pb, live ? whole(rows * row_bytes - j0 / 4) : 0);
        }
        rs = rsrc(ps, live ? rows * 4 : 0);
    };
    auto advance = [&]() {
        l0 += step_l;
        left -= step_l;
        if (MODE == 0) pa += (int64_t)step_l * I * 2;
        pb += (int64_t)step_l * (MODE == 0 ? J : row_bytes);
        ps += step_l * 4;
        if (MODE == 1 && left <= 0 && q + 1 < p.groups && l0 < end) {  // on to the next group
            while (q + 1 < p.groups && l0 >= padded(L)) {
                l0 -= padded(L);
                end -= padded(L);
                L = p.L[++q];
            }
            enter();
        }
        describe();
    };

    struct Loads {
        u32x4 a[NA];
        u32x4 b[MODE == 0 ? NB : 1];     // 16 codes each
        uint32_t w[MODE == 1 ? NB : 1];  // 16 weights each
        float s[MODE == 0 ? NB : 8];
        int left;  // MODE 1: elements of the row chunks that are inside their rows
    };
    Loads ld[D];
    auto load_a = [&](Loads& v, int n) {
        if constexpr (MODE == 0) {
            if (ALIGNED) {
                v.a[n] = load16(ra, voff_a[n]);
            } else {
                const bool in = ROWS == kOdd || (tg + n * TG) / (BM / 8) < left;
                v.a[n] = load8_half(ra, in ? voff_a[n] : 0x80000000u, 0);
            }
        } else {
            if (ALIGNED) {  // whole chunks: those past the row's end read as zeros
                const bool in = 8 * (tg % (BL / 8)) < left;
                v.a[n] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? voff_a[n] : 0x80000000u, 2 * l0, 0));
            } else {
                v.a[n] = load8_half(ra, voff_a[n], 2 * l0);
            }
        }
    };
    auto load_b = [&](Loads& v, int n) {
        if constexpr (MODE == 0) {
            v.b[n] = load16(rb, voff_b[n]);
            v.s[n] = __builtin_bit_cast(
                float, __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * ((tg + n * TG) / (BN / 16)), 0, 0));
        } else if (ALIGNED) {
            v.w[n] = __builtin_amdgcn_raw_buffer_load_b32(rb, voff_b[n], 0, 0);
        } else {
            // rows at any byte: the two dwords around the four bytes
            const auto d = __builtin_amdgcn_raw_buffer_load_b64(rb, voff_b[n] & ~3u, 0, 0);
            v.w[n] = __builtin_amdgcn_alignbit(d[1], d[0], 8 * (voff_b[n] & 3));
        }
    };
    auto load_s = [&](Loads& v) {
        if constexpr (MODE == 1) {
            const u32x4 a0 = load16(rs, 32 * (tg % (BL / 8))), a1 = load16(rs, 32 * (tg % (BL / 8)) + 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v.s[e] = __uint_as_float(a0[e]);
                v.s[4 + e] = __uint_as_float(a1[e]);
            }
            v.left = left - 8 * (tg % (BL / 8));
        }
    };

    // ---- conversion into an LDS stage, in slices of a few vector instructions ----
    // MODE 0: unit n of B in nine slices, the row's 1 / a and then two codes of each dword at a
    // time; A goes to LDS as it is.  MODE 1: one dword of a chunk of A per slice; B as it is.
    constexpr int kSlices = MODE == 0 ? NB * 9 : NA * 4;
    float inv = 0.0f;      // MODE 0
    u32x4 half_out[2];     // MODE 0: the unit's 16 values
    auto write_a = [&](const Loads& v, int n, uint8_t* A) {
        const int id = tg + n * TG;
        if constexpr (MODE == 0) {
            const int l = id / (BM / 8), c = id % (BM / 8);
            *reinterpret_cast<u32x4*>(A + granule<BM>(l, c >> 1) + 16 * (c & 1)) = v.a[n];
        } else if (kAFull || id < kAUnits) {
            *reinterpret_cast<u32x4*>(A + chunk<BL>(id / (BL / 8), id % (BL / 8))) = v.a[n];
        }
    };
    auto convert_slice = [&](Loads& v, int i, uint8_t* A) {
        if constexpr (MODE == 0) {
            const int n = i / 9, h = i % 9 - 1;
            if (h < 0) {
                // 1 / a: the reciprocal (1 ulp) and one Newton step, which leaves 2^-46 before its
                // rounding and keeps powers of two exact, in a third of a division's
                // instructions.  NaN, the scale of a token with a NaN, stays NaN; 0, of one with
                // an infinity, gives 2^127, under which the infinity's code of +-127 is infinite
                // and zeros stay zeros: rows past the end have this scale and only zeros.
                const float a = v.s[n], r = __builtin_fminf(__builtin_amdgcn_rcpf(a), 0x1p126f);
                inv = __builtin_fmaf(__builtin_fmaf(-a, r, 1.0f), r, r);
            } else {
                // each value rounded once (not at all for a power of two)
                const uint32_t u = v.b[n][h >> 1];
                const float f0 = (float)(int8_t)(u >> (16 * (h & 1)));
                const float f1 = (float)(int8_t)(u >> (16 * (h & 1) + 8));
                half_out[h >> 2][h & 3] = f32x2_to_bf16x2_rne(f0 * inv, f1 * inv);
            }
            if (h == 7) {
                const int id = tg + n * TG;
                u32x4* const dst = reinterpret_cast<u32x4*>(A + kA + granule<BN>(id / (BN / 16), id % (BN / 16)));
                dst[0] = half_out[0];
                dst[1] = half_out[1];
            }
        } else {
            const int n = i / 4, e = i % 4;
            uint32_t x = v.a[n][e];
            if (!ALIGNED) x &= v.left >= 2 * e + 2 ? 0xFFFFFFFFu : (v.left == 2 * e + 1 ? 0xFFFFu : 0u);
            v.a[n][e] = f32x2_to_bf16x2_rne(__uint_as_float(x << 16) * v.s[2 * e],
                                            __uint_as_float(x & 0xFFFF0000u) * v.s[2 * e + 1]);
            if (e == 3) write_a(v, n, A);
        }
    };
    auto write_w = [&](const Loads& v, int n, uint8_t* A) {  // MODE 1
        const int id = tg + n * TG, l = id / (BN / 16), c = id % (BN / 16);
        *reinterpret_cast<uint32_t*>(A + kA + packed_at<BN>(l, c >> 2) + 4 * (c & 3)) = v.w[n];
    };

    // ---- operands ----
    const int t16 = lane & 15, half = (lane >> 4) & 1, l8 = 8 * (lane >> 5);
    int off_a[MODE == 0 ? NI : KS], off_b[NJ];
    if constexpr (MODE == 0) {
        // 16-bit transposed reads: row l8 + t16 / 4, 8 bytes t16 % 4 of the granule
#pragma unroll
        for (int i = 0; i < NI; ++i)
            off_a[i] = granule<BM>(l8 + (t16 >> 2), (wi * WM + 32 * i) / 16 + half) + 8 * (t16 & 3);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            off_b[j] = granule<BN>(l8 + (t16 >> 2), (wj * WN + 32 * j) / 16 + half) + 8 * (t16 & 3);
    } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            off_a[ks] = chunk<BL>(wi * WM + (lane & 31), 2 * ks + (lane >> 5));
        // 8-bit transposed reads: row l8 + t16 / 2, 8 bytes t16 % 2 of the wave's 16 byte columns,
        // the same for both halves of the lanes (they take other fields of them)
        off_b[0] = packed_at<BN>(l8 + (t16 >> 1), wj) + 8 * (t16 & 1);
    }
    auto tr16 = [&](const uint8_t* a, int rows4) {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + rows4));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    struct Operands {
        bf16x8 a[NI], b[NJ];
        i32x2 w;  // MODE 1: the byte column that b comes from
    };
    // Part r of the reads of 16 rows (kReads of them, one LDS instruction each, two for tr16).
    constexpr int kReads = MODE == 0 ? NI + NJ : NI + 1;
    auto read = [&](const uint8_t* A, int ks, int r, Operands& o) {
        const uint8_t* const B = A + kA;
        if constexpr (MODE == 0) {
            if (r < NJ)
                o.b[r] = tr16(B + off_b[r] + ks * 16 * kBRow, 4 * kBRow);
            else
                o.a[r - NJ] = tr16(A + off_a[r - NJ] + ks * 16 * 2 * BM, 8 * BM);
        } else {
            if (r == 0)
                o.w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(B + off_b[0] + ks * 16 * kBRow));
            else
                o.a[r - 1] = *reinterpret_cast<const bf16x8*>(A + off_a[ks] + (r - 1) * 32 * 2 * BL);
        }
    };
    // MODE 1: four of the eight weights of b[j] (field 2 j + half of the byte column), the 2 NJ
    // parts of a step's 16 rows: a lookup gives the high bytes of bf16(2w), whose low bytes
    // are zero.
    auto expand = [&](Operands& o, int part) {
        const int j = part >> 1, i = part & 1;
        const uint32_t hi = __builtin_amdgcn_perm(
            kHi2w, kHi2w, ((uint32_t)o.w[i] >> (4 * j + 2 * half)) & 0x03030303u);
        u32x4 x = __builtin_bit_cast(u32x4, o.b[j]);
        x[2 * i] = __builtin_amdgcn_perm(0u, hi, 0x010C000Cu);
        x[2 * i + 1] = __builtin_amdgcn_perm(0u, hi, 0x030C020Cu);
        o.b[j] = __builtin_bit_cast(bf16x8, x);
    };
    f32x16 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // Step it multiplies stage it % 2 while step it + 1, in registers, is converted into the
    // other stage, and its registers are refilled for step it + 1 + D as soon as they are free.
    // Vector instructions of a wave wait for its matrix instructions in order, so with both
    // in runs the SIMD's waves stand behind one unit and then behind the other (measured:
    // the times of the two added up).  So each product is a slot that also carries a few
    // vector instructions of the conversion, of the expansion of the next weights, or an
    // LDS or memory access, and nothing is moved across slots.  One barrier before the last
    // 16 rows of the step, whose operands are already in registers; the first operands of
    // step it + 1 are read behind it.
    constexpr int NM = NI * NJ;
    constexpr int S = (KS - 1) * NM;  // slots that convert
    auto convert = [&](Loads& v, int slot, uint8_t* A, bool all) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
            if (MODE == 1 && (all || n * S / NB == slot)) {
                write_w(v, n, A);
                load_b(v, n);
            }
#pragma unroll
        for (int n = 0; n < NA; ++n)
            if (MODE == 0 && (all || n * S / NA == slot)) {
                write_a(v, n, A);
                load_a(v, n);
            }
#pragma unroll
        for (int i = 0; i < kSlices; ++i)
            if (all || i * S / kSlices == slot) {
                convert_slice(v, i, A);
                if (MODE == 0 && i % 9 == 8) load_b(v, i / 9);
                if (MODE == 1 && i % 4 == 3) load_a(v, i / 4);
            }
        if (all || slot == S - 1) load_s(v);
    };
    // operands of the 16 rows after the current ones: reads in the first slots, expansion in
    // the last
    auto next_operands = [&](const uint8_t* A, int ks, int slot, Operands& o) {
#pragma unroll
        for (int r = 0; r < kReads; ++r)
            if (r * ((NM + 1) / 2) / kReads == slot) read(A, ks, r, o);
        if (MODE == 1) {
#pragma unroll
            for (int e = 0; e < 2 * NJ; ++e)
                if (NM / 2 + e * (NM - NM / 2) / (2 * NJ) == slot) expand(o, e);
        }
    };
    Operands op[2];
    describe();
#pragma unroll
    for (int d = 0; d < D; ++d) {
        if (d > 0) advance();
#pragma unroll
        for (int n = 0; n < NA; ++n) load_a(ld[d], n);
#pragma unroll
        for (int n = 0; n < NB; ++n) load_b(ld[d], n);
        load_s(ld[d]);
    }
    advance();
    convert(ld[0], 0, stage, true);
    __syncthreads();
#pragma unroll
    for (int slot = 0; slot < NM; ++slot) next_operands(stage, 0, slot, op[0]);
    for (int it = 0; it < nsteps; it += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (D > 1 && it + d >= nsteps) break;
            uint8_t* const cur = stage + ((it + d) & 1) * kBuf;
            uint8_t* const nxt = stage + ((it + d + 1) & 1) * kBuf;
            advance();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const bool last = ks == KS - 1;
                if (last) __syncthreads();
                Operands& o = op[ks & 1];
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    acc[m % NI][m / NI] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        o.a[m % NI], o.b[m / NI], acc[m % NI][m / NI], 0, 0, 0);
                    next_operands(last ? nxt : cur, last ? 0 : ks + 1, m, op[(ks + 1) & 1]);
                    if (!last) convert(ld[(d + 1) % D], ks * NM + m, nxt, false);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }

    // join the groups: the upper half of the remaining groups hands its sums to the lower
    if constexpr (G > 1) {
        float* const x = reinterpret_cast<float*>(lds);
        __syncthreads();
#pragma unroll
        for (int h = G / 2; h >= 1; h /= 2) {
            if (g >= h && g < 2 * h) {
                float* const w = x + ((g - h) * WPG + wg) * (WM * WN) + lane;
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r) w[((i * NJ + j) * 16 + r) * 64] = acc[i][j][r];
            }
            __syncthreads();
            if (g < h) {
                const float* const w = x + (g * WPG + wg) * (WM * WN) + lane;
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

    // lane l, register r of a 32x32 accumulator: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
    // MODE 0: block j holds columns 32 j + l % 32.  MODE 1: byte column l % 16 of the wave, its
    // weight 2 j + half.
    // The kind of output and whether the tile lies inside it are the same for the whole block,
    // so they are asked once; 32-bit offsets reach over a tile's rows (256 rows of 2^20).
    // (The empty asm keeps the offsets from being computed, and held in registers, before the
    // main loop.)
    int pitch = J, tid_out = lane;
    asm volatile("" : "+s"(pitch), "+v"(tid_out));
    const int64_t base = (int64_t)(i0 + wi * WM) * pitch + j0 + wj * WN;
    const int rows = I - i0 - wi * WM, cols = J - j0 - wj * WN;
    const bool inside = rows >= WM && cols >= WN;
    auto emit = [&](auto all, auto put) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = 32 * i + 8 * (r >> 2) + 4 * (tid_out >> 5) + (r & 3);
                if constexpr (MODE == 0) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int col = 32 * j + (tid_out & 31);
                        if (decltype(all)::value || (row < rows && col < cols))
                            put((uint32_t)(row * pitch + col), acc[i][j][r], 0.0f);
                    }
                } else {
                    // lanes l and l + 16 hold columns 4 t + (0, 2) and 4 t + (1, 3): exchange, so
                    // that a lane has two neighbours, 4 t + 2 half + (0, 1)
                    const auto x = __builtin_amdgcn_permlane16_swap(
                        __float_as_uint(acc[i][0][r]), __float_as_uint(acc[i][1][r]), false, false);
                    const int col = 4 * (tid_out & 15) + 2 * ((tid_out >> 4) & 1);
                    if (decltype(all)::value || (row < rows && col < cols))
                        put((uint32_t)(row * pitch + col), 0.5f * __uint_as_float(x[0]),
                            0.5f * __uint_as_float(x[1]));
                }
            }
    };
    auto output = [&](auto put) {
        if (inside)
            emit(std::true_type(), put);
        else
            emit(std::false_type(), put);
    };
    if (p.slices > 1) {
        float* const out = p.part + (int64_t)slice * I * J + base;
        output([&](uint32_t o, float v0, float v1) {
            if constexpr (MODE == 0)
                out[o] = v0;
            else
                *reinterpret_cast<float2*>(out + o) = make_float2(v0, v1);
        });
    } else if (MODE == 0 && p.out_dtype == BITNET_OUT_F32) {
        float* const out = static_cast<float*>(p.out) + base;
        output([&](uint32_t o, float v0, float) { out[o] = v0; });
    } else {
        uint16_t* const out = static_cast<uint16_t*>(p.out) + base;
        output([&](uint32_t o, float v0, float v1) {
            if constexpr (MODE == 0)
                out[o] = f32_to_bf16_rne(v0);
            else
                *reinterpret_cast<uint32_t*>(out + o) = f32x2_to_bf16x2_rne(v0, v1);
        });
    }
}

// Sum of the slices' partials, in order; four outputs a thread (J % 4 == 0).
__global__ __launch_bounds__(256) void grad_join_kernel(const float* __restrict__ part, int slices,
                                                        int64_t n, int out_dtype, void* out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    float4 s = *reinterpret_cast<const float4*>(part + i);
#pragma unroll 4
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
// A tile configuration and what it costs: d steps of loads in flight, at least w waves per
// SIMD (4: at most 128 registers), blocks per CU, and the microseconds of a block's
// prologue and epilogue and of a step of a group, alone on its CU and among `blocks` of them
// (measured at 512 to 2048 tokens on 2B and 8B layers; full chip, so at its clocks).
struct GradCfg {
    int mode, bm, bn, wm, wn, g, bl, d, w, blocks;
    double base, step_alone, step_full;
};
constexpr GradCfg kCfg[] = {
    // weight gradient.  256 x 256 is the fastest per flop (2048 x 4096 x 14336: 232 us, 128 x 128
    // tiles 278 and 284); its 256 blocks at a time leave most of the chip idle in a short last
    // round (2048 x 6912 x 2560, 270 tiles: 107 us), which 128 x 128 tiles, two or four blocks
    // per CU, fill better (96 and 109; of 512 tokens 33 and 35 against 40); four share a CU only
    // at half the rows per step.  The costs below are from before the epilogue lost its
    // branches, 10 to 15% too high alike; the tile they pick was within 8% of the best of the
    // three at six sizes measured since.
    {0, 256, 256, 128, 64, 1, 64, 1, 1, 1, 13, 1.8, 1.8},
    {0, 128, 128, 64, 64, 1, 64, 1, 1, 2, 8, 0.73, 1.15},
    {0, 128, 128, 64, 64, 1, 32, 1, 4, 4, 8, 0.43, 1.25},
    // input gradient.  256 x 256 for the largest (2048 x 28672 x 4096 in two slices: 370 us,
    // 256 x 128 457); 256 x 128 where that makes one round of the chip (2048 x 4096 x 4096: 72 us
    // against 77); 64 x 128 with the sum over four groups of waves for hundreds of tokens (512 x
    // 3840 x 2560: 25 us, 256 x 128 in four slices 33); 32 x 128 below (4 x 2560 x 2560 in ten
    // slices with the join: 8.4 us).
    {1, 256, 256, 128, 64, 1, 64, 1, 1, 1, 8, 1.7, 1.7},
    {1, 256, 128, 128, 64, 2, 32, 1, 1, 1, 9, 1.0, 1.0},
    {1, 64, 128, 64, 64, 4, 32, 2, 1, 1, 7, 0.59, 0.59},
    {1, 32, 128, 32, 64, 4, 32, 2, 1, 2, 6, 0.45, 0.67},
};
constexpr int kCfgs = sizeof(kCfg) / sizeof(kCfg[0]);
constexpr int kCUs = 256;

// The configuration and number of slices with the least estimated time.
GradPlan plan(int mode, int64_t I, int64_t J, const int64_t* L, int groups) {
    GradPlan best = {0, 1, 0};
    double best_t = 1e300;
    for (int c = 0; c < kCfgs; ++c) {
        const GradCfg& k = kCfg[c];
        if (k.mode != mode) continue;
        int64_t steps = 0;
        for (int q = 0; q < groups; ++q) steps += (L[q] + k.bl - 1) / k.bl;
        const int64_t tiles = ((I + k.bm - 1) / k.bm) * ((J + k.bn - 1) / k.bn);
        for (int64_t s = 1; s <= 16; ++s) {
            // at least two steps per group of a slice, at most 64 MB of partial sums
            if (s > 1 && (steps < 2 * s * k.g || s * I * J * 4 > ((int64_t)64 << 20))) break;
            const double per = (double)(((steps + s - 1) / s + k.g - 1) / k.g);
            const double x = (double)(tiles * s) / (kCUs * k.blocks);
            double t;
            if (tiles * s <= kCUs)
                t = k.base + per * k.step_alone;
            else if (x <= 1)
                t = k.base + per * k.step_full;
            else  // blocks of a CU do not end together: half of a last round's raggedness
                t = (k.blocks > 1 ? 0.5 * (x + std::ceil(x)) : std::ceil(x)) * (k.base + per * k.step_full);
            if (s > 1) t += 3.0 + (s + 1) * I * J * 4.0 / 5e6;  // the join: a launch, its bytes
            if (t < best_t) {
                best_t = t;
                best = {c, (int)s, (int)steps};
            }
        }
    }
    return best;
}

template <int C, Rows ROWS>
void launch_rows(const GradArgs& a, hipStream_t stream) {
    constexpr GradCfg k = kCfg[C];
    const dim3 grid((unsigned)((int64_t)a.tiles_i * a.tiles_j * a.slices));
    const dim3 block(64 * (k.bm / k.wm) * (k.bn / k.wn) * k.g);
    hipLaunchKernelGGL((grad_kernel<k.mode, k.bm, k.bn, k.wm, k.wn, k.g, k.bl, k.d, k.w, ROWS>), grid, block, 0,
                       stream, a);
}

template <int C>
void launch_cfg(const GradArgs& a, bool aligned, hipStream_t stream) {
    if (aligned)
        launch_rows<C, kWhole>(a, stream);
    else if (kCfg[C].mode == 0 && a.tiles_i == 1 && a.L[0] % 2 != 0)
        launch_rows<C, kCfg[C].mode == 0 ? kOddEnd : kOdd>(a, stream);
    else
        launch_rows<C, kOdd>(a, stream);
}

template <size_t... C>
void launch_any(int cfg, const GradArgs& a, bool aligned, hipStream_t stream, std::index_sequence<C...>) {
    ((cfg == (int)C ? launch_cfg<(int)C>(a, aligned, stream) : (void)0), ...);
}

hipError_t launch_grad(int mode, GradArgs a, const int64_t* L, bool aligned, void* workspace,
                       size_t ws_bytes, hipStream_t stream) {
    const int64_t n = (int64_t)a.I * a.J;
    GradPlan pl = plan(mode, a.I, a.J, L, a.groups);
    if ((size_t)pl.slices * n * 4 > ws_bytes) pl.slices = 1;
    const GradCfg& k = kCfg[pl.cfg];
    const int64_t ti = (a.I + k.bm - 1) / k.bm, tj = (a.J + k.bn - 1) / k.bn;
    // (millions of tokens make 256 x 256 tiles, so that what fits the card fits a launch)
    if (ti * tj * pl.slices > max_blocks(64 * (k.bm / k.wm) * (k.bn / k.wn) * k.g)) return hipErrorInvalidValue;
    a.tiles_i = (int)ti;
    a.tiles_j = (int)tj;
    a.steps = pl.steps;
    a.slices = pl.slices;
    a.part = static_cast<float*>(workspace);
    launch_any(pl.cfg, a, aligned, stream, std::make_index_sequence<kCfgs>());
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
    out[4] = k.bl;
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
        aligned = aligned && N[q] % 8 == 0;
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
