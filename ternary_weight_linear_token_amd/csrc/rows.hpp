// rows.hpp -- helpers of the kernels that work on whole rows (quantization, the norms, SwiGLU, sums of
// experts' rows): groups of V bf16 elements, reductions over the waves of one row, int8 codes and their scales.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace bitnet {

// V bf16 values, two per word, low half first.
template <int V>
struct RowVec {
    uint32_t w[V / 2];
};

template <int V>
__device__ __forceinline__ RowVec<V> zero_row_vec() {
    RowVec<V> v;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v.w[i] = 0u;
    return v;
}
template <int V>
__device__ __forceinline__ RowVec<V> load_row_vec(const uint16_t* row, int64_t g) {
    RowVec<V> v;
    if constexpr (V == 8) {
        const uint4 t = reinterpret_cast<const uint4*>(row)[g];
        v.w[0] = t.x;
        v.w[1] = t.y;
        v.w[2] = t.z;
        v.w[3] = t.w;
    } else {
        const uint2 t = reinterpret_cast<const uint2*>(row)[g];
        v.w[0] = t.x;
        v.w[1] = t.y;
    }
    return v;
}
template <int V>
__device__ __forceinline__ void store_row_vec(uint16_t* row, int64_t g, const RowVec<V>& v) {
    if constexpr (V == 8)
        reinterpret_cast<uint4*>(row)[g] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    else
        reinterpret_cast<uint2*>(row)[g] = make_uint2(v.w[0], v.w[1]);
}
template <int V>
__device__ __forceinline__ void to_f32(const RowVec<V>& v, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = __uint_as_float(v.w[i] << 16);
        f[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
    }
}
// Running max of |x| as bf16 magnitude bits (monotone for finite values), one in each half of
// the word: one packed 16-bit max per two values.
template <int V>
__device__ __forceinline__ uint32_t max_pairs(const RowVec<V>& v, uint32_t mx) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = __builtin_bit_cast(u16x2, mx);
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v.w[i] & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, m);
}
__device__ __forceinline__ uint32_t max_of_pair(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

__device__ __forceinline__ float wave_sum_f32(float v) {
    return __uint_as_float(wave_reduce_dpp(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// Sum / max over the WPR waves of a block that share a row; slot: WPR words of LDS that the
// block reuses no earlier than after another of its barriers.
template <int WPR>
__device__ __forceinline__ float team_sum(float v, float* slot) {
    v = wave_sum_f32(v);
    if (WPR > 1) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i) v += slot[i];
    }
    return v;
}
template <int WPR>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* slot) {
    v = wave_max_u32(v);
    if (WPR > 1) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i) v = max(v, slot[i]);
    }
    return v;
}

// The largest power of two a with a * amax <= 127 (at most 2^23, the power below
// 127 / 1e-5) for amax given as bf16 bits 1.f * 2^e: 127 = 1.984375 * 2^6, so the exponent
// is 6 - e, and one less for the one fraction above, f = 127/128.
__device__ __forceinline__ float pow2_scale(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 7) - 127;
    int p = 6 - e - ((amax_bits & 0x7Fu) == 0x7Fu ? 1 : 0);
    p = p > 23 ? 23 : p;
    return __uint_as_float((uint32_t)(127 + p) << 23);
}

// f(whether codes of rows with this max |x|, the same in every lane, need the clamp).
template <class F>
__device__ __forceinline__ void with_clamp(uint32_t amax_bits, const F& f) {
    if (__builtin_amdgcn_readfirstlane(amax_bits) >= 0x7F80u)
        f(std::true_type());
    else
        f(std::false_type());
}

// Activation scale of a row whose max |x| has these bf16 bits: 127 / max(amax, 1e-5), or
// the power of two above.
__device__ __forceinline__ float scale_of(uint32_t amax_bits, bool pow2) {
    if (pow2) return pow2_scale(amax_bits);
    float amax = bf16_bits_to_f32(amax_bits);
    amax = amax < 1e-5f ? 1e-5f : amax;
    return 127.0f / amax;
}

// rne(x * a) of V elements as int8, every code of the library: adding 1.5 * 2^23 to fl(x * a)
// rounds it to an integer, ties to even, and the sum's low byte is that integer.  Finite rows
// need no clamp, |fl(x * a)| <= 127 (1 + 2^-23) < 127.5 for both kinds of scale; an infinity
// becomes +-127 (and, restored by the scale 2^-122 of such a row, infinite again), NaN -127.
// CLAMP may be false for finite rows (for every row it costs SwiGLU 4096 x 28672 170 -> 179 us).
template <int V, bool CLAMP>
__device__ __forceinline__ void store_codes(int8_t* row, int64_t g, const RowVec<V>& v, float a) {
    constexpr float kMagic = 12582912.0f;
    float f[V];
    to_f32<V>(v, f);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = CLAMP ? __builtin_amdgcn_fmed3f(f[j] * a, -127.0f, 127.0f) : f[j] * a;
    uint32_t p[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(f[4 * i + j] + kMagic);
        p[i] = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u) | __builtin_amdgcn_perm(q[3], q[2], 0x04000c0cu);
    }
    if constexpr (V == 8)
        reinterpret_cast<uint2*>(row)[g] = make_uint2(p[0], p[1]);
    else
        reinterpret_cast<uint32_t*>(row)[g] = p[0];
}

constexpr int kTeamGroups = 2;  // groups of V elements a lane of a norm's team holds

// V values of an fp32 vector, or `missing` where there is none.
template <int V>
__device__ __forceinline__ void load_f32(const float* p, int64_t g, float missing, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 t = p ? reinterpret_cast<const float4*>(p)[(g * V + i) / 4]
                           : make_float4(missing, missing, missing, missing);
        v[i] = t.x;
        v[i + 1] = t.y;
        v[i + 2] = t.z;
        v[i + 3] = t.w;
    }
}

// V elements of a row that is bf16, or int8 codes.
template <int V, bool CODES>
struct XVec {
    RowVec<V> v;
};
template <int V>
struct XVec<V, true> {
    uint32_t q[V / 4];
};
template <int V, bool CODES>
__device__ __forceinline__ XVec<V, CODES> load_x(const void* x, int64_t row, int64_t g) {
    XVec<V, CODES> r;
    if constexpr (CODES) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(x) + row) + g * (V / 4);
        if constexpr (V == 8) {
            const uint2 t = *reinterpret_cast<const uint2*>(p);
            r.q[0] = t.x;
            r.q[1] = t.y;
        } else {
            r.q[0] = *p;
        }
    } else {
        r.v = load_row_vec<V>(static_cast<const uint16_t*>(x) + row, g);
    }
    return r;
}
// The bf16 values or the codes as fp32, exactly.
template <int V, bool CODES>
__device__ __forceinline__ void x_to_f32(const XVec<V, CODES>& v, float (&x)[V]) {
    if constexpr (CODES) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = (float)(int8_t)(v.q[j / 4] >> (8 * (j & 3)));
    } else {
        to_f32<V>(v.v, x);
    }
}

// Waves per row whose lanes hold the row in two groups each; 0: too long.
inline int team_waves(int64_t K, int V) {
    for (int w = 1; w <= 16; w *= 2)
        if (K <= (int64_t)w * 64 * kTeamGroups * V) return w;
    return 0;
}

// Waves per row of the backward pass, one group a lane up to 16 waves, then two; 0: too long.
inline int back_waves(int64_t K, int V) {
    for (int w = 1; w <= 16; w *= 2)
        if (K <= (int64_t)w * 64 * V) return w;
    return K <= (int64_t)16 * 64 * 2 * V ? 16 : 0;
}

}  // namespace bitnet
