// norm.hip -- layer norm in front of a BitLinear layer (forward, optionally with the int8
// codes of its output; backward), and the values 8-bit codes stand for, on gfx950.
//
//   forward   mu = mean_k x, r = 1 / sqrt(mean_k (x - mu)^2 + eps), y = (x - mu) r w + b
//             codes: those bitnet_quant_act (or _pow2) gives for the bf16 y
//   backward  xh = (x - mu) r, g = dy w:
//             dx = r (g - mean_k g - xh mean_k (g xh)),  dw = sum_m dy xh,  db = sum_m dy
//             x as bf16 or as an 8-bit checkpoint xq / a.
//
// Bound by HBM: x is read once and every output written once.  A row is taken by WPR waves
// (a "team") of which each lane keeps up to two groups of V elements in registers, so the
// second pass of the variance and the outputs need no second read; a lane keeps its columns
// for all rows of its team, so the norm's weight and bias are read once per block and the
// backward's column sums stay in registers until the block's last row.  Sums are fp32; the
// variance is the sum of squared differences from the mean (no cancellation).  The column
// sums are joined block by block in a fixed order by a second launch (no atomics: the same
// inputs give the same bits).
//
// Measured, inputs out of cache (a copy of the same sizes: 5.3 to 5.8 TB/s): forward 8192 x 8192
// 45.8 us, 5.9 TB/s, with codes instead of y 42.7 us, 4.7 TB/s (the vector instructions of the
// statistics and codes, about 290 per 16 columns a lane and row, are then as long as the
// bytes); 4096 x 14336 47 us, 5.0 TB/s, with codes 51 us; over 16384 columns the row is read up to
// four times, 2048 x 28672 57 us, 4.1 TB/s.  Backward from a checkpoint 8192 x 4096 41.2 us, 4.1
// TB/s, its column sums 4.2 of them; from bf16 65536 x 1024 77 us, 5.2 TB/s; rows over 8192 columns
// (16 waves, two groups a lane, 24 to 32 registers in scratch) 4096 x 14336 112 us, 3.1 TB/s, and
// over 16384 (two launches that read everything twice over) 2048 x 28672 162 us, 2.2 TB/s.  One
// row of 2560: 2.4 us warm, 4.7 cold, latency.
#include "device_common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace bitnet {

namespace {

constexpr int kTeamGroups = 2;  // groups of V elements a lane holds

struct NormArgs {
    const uint16_t* x;
    const float *w, *b;  // NULL: 1 and 0
    float eps;
    int64_t M, K;
    uint16_t* y;     // NULL: not written
    int8_t* xq;      // NULL: no codes
    float* a_scale;  // with xq
    int pow2;
    float *mean, *rstd;  // NULL: not written
};

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

template <int V, int WPR>
__global__ __launch_bounds__(64 * WPR) void layernorm_kernel(NormArgs p) {
    constexpr int G = kTeamGroups, kStride = 64 * WPR;
    __shared__ float s_red[2][WPR];
    __shared__ uint32_t s_max[WPR];
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    float w[G][V], b[G][V];
    bool in[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int64_t g = threadIdx.x + (int64_t)i * kStride;
        in[i] = g < groups;
        load_f32<V>(p.w, in[i] ? g : 0, 1.0f, w[i]);
        load_f32<V>(p.b, in[i] ? g : 0, 0.0f, b[i]);
    }
    auto load = [&](int64_t m, RowVec<V> (&v)[G]) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            v[i] = zero_row_vec<V>();
            if (in[i] && m < p.M) v[i] = load_row_vec<V>(p.x + m * p.K, threadIdx.x + (int64_t)i * kStride);
        }
    };
    RowVec<V> cur[G], nxt[G];
    load(blockIdx.x, cur);
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        load(m + gridDim.x, nxt);
        float x[G][V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            to_f32<V>(cur[i], x[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) sum += x[i][j];
        }
        const float mean = team_sum<WPR>(sum, s_red[0]) * inv_k;
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i)
            if (in[i]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    x[i][j] -= mean;
                    sq = __builtin_fmaf(x[i][j], x[i][j], sq);
                }
            }
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(team_sum<WPR>(sq, s_red[1]), inv_k, p.eps));
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
                cur[i].w[j] =
                    f32x2_to_bf16x2_rne(__builtin_fmaf(x[i][2 * j] * rstd, w[i][2 * j], b[i][2 * j]),
                                        __builtin_fmaf(x[i][2 * j + 1] * rstd, w[i][2 * j + 1], b[i][2 * j + 1]));
            if (in[i]) {
                if (p.y) store_row_vec<V>(p.y + m * p.K, threadIdx.x + (int64_t)i * kStride, cur[i]);
                mx = max_pairs<V>(cur[i], mx);
            }
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[m] = mean;
            if (p.rstd) p.rstd[m] = rstd;
        }
        if (p.xq) {
            const uint32_t amax = team_max<WPR>(max_of_pair(mx), s_max);
            const float a = scale_of(amax, p.pow2);
            if (threadIdx.x == 0) p.a_scale[m] = a;
            with_clamp(amax, [&](auto clamp) {
#pragma unroll
                for (int i = 0; i < G; ++i)
                    if (in[i])
                        store_codes<V, decltype(clamp)::value>(p.xq + m * p.K, threadIdx.x + (int64_t)i * kStride,
                                                               cur[i], a);
            });
        }
#pragma unroll
        for (int i = 0; i < G; ++i) cur[i] = nxt[i];
    }
}

// Rows too long for a team's registers: one block of 16 waves per row reads it up to four
// times (the later ones from cache).
template <int V>
__global__ __launch_bounds__(1024) void layernorm_long_kernel(NormArgs p) {
    constexpr int WPR = 16;
    __shared__ float s_red[2][WPR];
    __shared__ uint32_t s_max[WPR];
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const uint16_t* row = p.x + m * p.K;
        float x[V], sum = 0.0f, sq = 0.0f;
        for (int64_t g = threadIdx.x; g < groups; g += 1024) {
            to_f32<V>(load_row_vec<V>(row, g), x);
#pragma unroll
            for (int j = 0; j < V; ++j) sum += x[j];
        }
        const float mean = team_sum<WPR>(sum, s_red[0]) * inv_k;
        for (int64_t g = threadIdx.x; g < groups; g += 1024) {
            to_f32<V>(load_row_vec<V>(row, g), x);
#pragma unroll
            for (int j = 0; j < V; ++j) sq = __builtin_fmaf(x[j] - mean, x[j] - mean, sq);
        }
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(team_sum<WPR>(sq, s_red[1]), inv_k, p.eps));
        auto output = [&](int64_t g) {
            float w[V], b[V];
            load_f32<V>(p.w, g, 1.0f, w);
            load_f32<V>(p.b, g, 0.0f, b);
            to_f32<V>(load_row_vec<V>(row, g), x);
            RowVec<V> y;
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
                y.w[j] = f32x2_to_bf16x2_rne(
                    __builtin_fmaf((x[2 * j] - mean) * rstd, w[2 * j], b[2 * j]),
                    __builtin_fmaf((x[2 * j + 1] - mean) * rstd, w[2 * j + 1], b[2 * j + 1]));
            return y;
        };
        uint32_t mx = 0;
        for (int64_t g = threadIdx.x; g < groups; g += 1024) {
            const RowVec<V> y = output(g);
            if (p.y) store_row_vec<V>(p.y + m * p.K, g, y);
            mx = max_pairs<V>(y, mx);
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[m] = mean;
            if (p.rstd) p.rstd[m] = rstd;
        }
        if (p.xq) {
            const uint32_t amax = team_max<WPR>(max_of_pair(mx), s_max);
            const float a = scale_of(amax, p.pow2);
            if (threadIdx.x == 0) p.a_scale[m] = a;
            with_clamp(amax, [&](auto clamp) {
                for (int64_t g = threadIdx.x; g < groups; g += 1024)
                    store_codes<V, decltype(clamp)::value>(p.xq + m * p.K, g, output(g), a);
            });
        }
    }
}

// ------------------------------------------------------------------------- backward
struct NormBackArgs {
    const uint16_t* dy;
    const void* x;         // bf16, or int8 codes with x_scale
    const float* x_scale;  // NULL: x is bf16
    const float *w, *mean, *rstd;
    int64_t M, K;
    uint16_t* dx;
    float* part;  // (blocks, 2, K) column sums, NULL: not wanted
};

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

// xh = (x - mean) rstd, each step rounded relative to xh itself however far the row lies from
// zero; from codes c = a x it is (c - a mean) (rstd / a), the difference in one fused
// multiply-add, which 1 / a would not leave exact.  (x rstd - mean rstd in one instruction
// instead of two errs by u |mean| rstd: for a mean of 500 spreads dw was 8e-6 off.)
template <bool CODES>
__device__ __forceinline__ float normalized(float x, float mean, float a, float scale) {
    return (CODES ? __builtin_fmaf(-mean, a, x) : x - mean) * scale;
}

// Blocks of TEAMS teams; the teams of a block walk the rows in step (every wave reaches
// every barrier; a team past the last row works on zeros).
// A lane holds one group of V columns where 16 waves cover the row so: with two, the column
// sums, the weight and two rows in flight take 146 registers and one block fills a CU
// (8192 x 4096 from the checkpoint, both launches: 59 us against 44).
template <int V, int WPR, int G, bool CODES>
__global__ __launch_bounds__(WPR == 16 ? 1024 : 512) void layernorm_back_kernel(NormBackArgs p) {
    constexpr int kStride = 64 * WPR, TEAMS = WPR == 16 ? 1 : 8 / WPR;
    __shared__ float s_red[2][TEAMS][WPR][2];
    __shared__ float s_join[TEAMS > 1 ? kStride * G * V : 1];
    const int team = threadIdx.x / kStride, lr = threadIdx.x % kStride;
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    float w[G][V], dw[G][V], db[G][V];
    bool in[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int64_t g = lr + (int64_t)i * kStride;
        in[i] = g < groups;
        load_f32<V>(p.w, in[i] ? g : 0, 1.0f, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.0f;
    }
    struct Row {
        RowVec<V> dy[G];
        XVec<V, CODES> x[G];
        float mean, rstd, a;
    };
    auto load = [&](int64_t m, Row& r) {
        const bool live = m < p.M;
        r.mean = live ? p.mean[m] : 0.0f;
        r.rstd = live ? p.rstd[m] : 0.0f;
        r.a = 1.0f;
        if (CODES && live) r.a = p.x_scale[m];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            r.dy[i] = zero_row_vec<V>();
            r.x[i] = XVec<V, CODES>{};
            if (live && in[i]) {
                const int64_t g = lr + (int64_t)i * kStride;
                r.dy[i] = load_row_vec<V>(p.dy + m * p.K, g);
                r.x[i] = load_x<V, CODES>(p.x, m * p.K, g);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    Row cur, nxt;
    load((int64_t)blockIdx.x * TEAMS + team, cur);
    int parity = 0;
    for (int64_t m0 = (int64_t)blockIdx.x * TEAMS; m0 < p.M; m0 += step, parity ^= 1) {
        const int64_t m = m0 + team;
        load(m + step, nxt);
        const float scale = CODES ? cur.rstd / cur.a : cur.rstd;
        float xh[G][V], g[G][V], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            float d[V];
            to_f32<V>(cur.dy[i], d);
            x_to_f32<V, CODES>(cur.x[i], xh[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // columns past the row have dy = 0 and add nothing below
                xh[i][j] = normalized<CODES>(xh[i][j], cur.mean, cur.a, scale);
                dw[i][j] = __builtin_fmaf(d[j], xh[i][j], dw[i][j]);
                db[i][j] += d[j];
                g[i][j] = d[j] * w[i][j];
                s1 += g[i][j];
                s2 = __builtin_fmaf(g[i][j], xh[i][j], s2);
            }
        }
        s1 = wave_sum_f32(s1);
        s2 = wave_sum_f32(s2);
        if (WPR > 1) {
            float(&red)[WPR][2] = s_red[parity][team];
            if ((threadIdx.x & 63) == 0) {
                red[lr >> 6][0] = s1;
                red[lr >> 6][1] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                s1 += red[i][0];
                s2 += red[i][1];
            }
        }
        const float c1 = -cur.rstd * (s1 * inv_k), c2 = -cur.rstd * (s2 * inv_k);
        if (m < p.M) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                RowVec<V> o;
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                    o.w[j] = f32x2_to_bf16x2_rne(
                        __builtin_fmaf(c2, xh[i][2 * j], __builtin_fmaf(cur.rstd, g[i][2 * j], c1)),
                        __builtin_fmaf(c2, xh[i][2 * j + 1], __builtin_fmaf(cur.rstd, g[i][2 * j + 1], c1)));
                if (in[i]) store_row_vec<V>(p.dx + m * p.K, lr + (int64_t)i * kStride, o);
            }
        }
        cur = nxt;
    }
    if (!p.part) return;
    float* const part = p.part + (int64_t)blockIdx.x * 2 * p.K;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float(&acc)[G][V] = which ? db : dw;
        for (int tm = 1; tm < TEAMS; ++tm) {
            __syncthreads();
            if (team == tm) {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) s_join[(i * V + j) * kStride + lr] = acc[i][j];
            }
            __syncthreads();
            if (team == 0) {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[i][j] += s_join[(i * V + j) * kStride + lr];
            }
        }
        if (team == 0) {
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (in[i]) {
#pragma unroll
                    for (int j = 0; j < V; j += 4)
                        *reinterpret_cast<float4*>(part + which * p.K + (lr + (int64_t)i * kStride) * V + j) =
                            make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
                }
        }
    }
}

// dx of rows too long for a team's registers: one block per row, two reads.
template <int V, bool CODES>
__global__ __launch_bounds__(1024) void layernorm_back_long_kernel(NormBackArgs p) {
    constexpr int WPR = 16;
    __shared__ float s_red[2][WPR];
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const float mean = p.mean[m], rstd = p.rstd[m];
        const float a = CODES ? p.x_scale[m] : 1.0f, scale = CODES ? rstd / a : rstd;
        float xh[V], g[V], s1 = 0.0f, s2 = 0.0f;
        auto read = [&](int64_t i) {
            float d[V], w[V];
            to_f32<V>(load_row_vec<V>(p.dy + m * p.K, i), d);
            x_to_f32<V, CODES>(load_x<V, CODES>(p.x, m * p.K, i), xh);
            load_f32<V>(p.w, i, 1.0f, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[j] = normalized<CODES>(xh[j], mean, a, scale);
                g[j] = d[j] * w[j];
            }
        };
        for (int64_t i = threadIdx.x; i < groups; i += 1024) {
            read(i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1 += g[j];
                s2 += g[j] * xh[j];
            }
        }
        const float c1 = team_sum<WPR>(s1, s_red[0]) * inv_k, c2 = team_sum<WPR>(s2, s_red[1]) * inv_k;
        for (int64_t i = threadIdx.x; i < groups; i += 1024) {
            read(i);
            RowVec<V> o;
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
                o.w[j] = f32x2_to_bf16x2_rne(rstd * (g[2 * j] - c1 - xh[2 * j] * c2),
                                             rstd * (g[2 * j + 1] - c1 - xh[2 * j + 1] * c2));
            store_row_vec<V>(p.dx + m * p.K, i, o);
        }
    }
}

// Column sums of such rows: block (c, s) takes 256 columns of every gridDim.y-th row.
template <bool CODES>
__global__ __launch_bounds__(256) void layernorm_cols_kernel(NormBackArgs p) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= p.K) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        const float d = bf16_bits_to_f32(p.dy[m * p.K + k]);
        float x, a = 1.0f, scale = p.rstd[m];
        if (CODES) {
            x = (float)static_cast<const int8_t*>(p.x)[m * p.K + k];
            a = p.x_scale[m];
            scale /= a;
        } else {
            x = bf16_bits_to_f32(static_cast<const uint16_t*>(p.x)[m * p.K + k]);
        }
        dw = __builtin_fmaf(d, normalized<CODES>(x, p.mean[m], a, scale), dw);
        db += d;
    }
    float* const part = p.part + (int64_t)blockIdx.y * 2 * p.K;
    part[k] = dw;
    part[p.K + k] = db;
}

// out[k] = sum_b part[b][which][k]: 64 columns per block, 64 rows of 16 threads that each add
// every 64th partial of four columns, then the 64 sums of a column in order.
__global__ __launch_bounds__(1024) void layernorm_join_kernel(const float* __restrict__ part, int blocks,
                                                              int64_t K, float* dweight, float* dbias) {
    __shared__ float s[64][68];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int64_t k = (int64_t)blockIdx.x * 64 + 4 * c;
    float* const out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (k < K) {
#pragma unroll 4
        for (int b = r; b < blocks; b += 64) {
            const float4 v = *reinterpret_cast<const float4*>(part + ((int64_t)b * 2 + blockIdx.y) * K + k);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
        }
    }
    *reinterpret_cast<float4*>(&s[r][4 * c]) = sum;
    __syncthreads();
    const int col = threadIdx.x & 63, q = threadIdx.x >> 6;  // 16 waves, four sums each
    float t = (s[4 * q][col] + s[4 * q + 1][col]) + (s[4 * q + 2][col] + s[4 * q + 3][col]);
    __syncthreads();
    s[q][col] = t;
    __syncthreads();
    const int64_t kc = (int64_t)blockIdx.x * 64 + col;
    if (q == 0 && kc < K) {
#pragma unroll
        for (int i = 1; i < 16; ++i) t += s[i][col];
        out[kc] = t;
    }
}

// ------------------------------------------------------------------------- dequantize
// bf16(c * (1 / a)): V codes a thread, blocks of 256 groups along a row.  HBM-bound: 16 codes a
// thread 8192 x 8192 34 us, 5.9 TB/s (8 codes and a division per value: 49 us).
template <int V>
__global__ __launch_bounds__(256) void dequant_kernel(const int8_t* __restrict__ xq,
                                                      const float* __restrict__ a_scale, int64_t groups,
                                                      int64_t blocks_per_row, uint16_t* __restrict__ x) {
    constexpr int P = V == 4 ? 4 : 8;  // codes per store
    const int64_t m = blockIdx.x / blocks_per_row;
    const int64_t g = (blockIdx.x - m * blocks_per_row) * 256 + threadIdx.x;
    if (g >= groups) return;
    XVec<P, true> q[V / P];
    const uint32_t* src = reinterpret_cast<const uint32_t*>(xq + m * groups * V) + g * (V / 4);
    if constexpr (V == 16) {
        const uint4 t = *reinterpret_cast<const uint4*>(src);
        q[0].q[0] = t.x;
        q[0].q[1] = t.y;
        q[1].q[0] = t.z;
        q[1].q[1] = t.w;
    } else {
        q[0] = load_x<V, true>(xq, m * groups * V, g);
    }
    const float inv = 1.0f / a_scale[m];
#pragma unroll
    for (int i = 0; i < V / P; ++i) {
        float f[P];
        x_to_f32<P, true>(q[i], f);
        RowVec<P> o;
#pragma unroll
        for (int j = 0; j < P / 2; ++j) o.w[j] = f32x2_to_bf16x2_rne(f[2 * j] * inv, f[2 * j + 1] * inv);
        store_row_vec<P>(x + m * groups * V, g * (V / P) + i, o);
    }
}

// Waves per row whose lanes hold the row in two groups each; 0: too long.
int team_waves(int64_t K, int V) {
    for (int w = 1; w <= 16; w *= 2)
        if (K <= (int64_t)w * 64 * kTeamGroups * V) return w;
    return 0;
}

// Waves per row of the backward pass, one group a lane up to 16 waves, then two; 0: too long.
int back_waves(int64_t K, int V) {
    for (int w = 1; w <= 16; w *= 2)
        if (K <= (int64_t)w * 64 * V) return w;
    return K <= (int64_t)16 * 64 * 2 * V ? 16 : 0;
}

// Blocks of the backward pass.
int64_t back_blocks(int64_t M, int64_t K) {
    const int w = back_waves(K, K % 8 == 0 ? 8 : 4);
    if (w == 0) return M < 64 * 32 ? (M + 31) / 32 : 64;
    const int64_t teams = w == 16 ? 1 : 8 / w;
    const int64_t b = (M + 2 * teams - 1) / (2 * teams);
    return b < 512 ? b : 512;
}

template <int V>
hipError_t launch_layernorm_v(const NormArgs& a, hipStream_t stream) {
    const unsigned rows = (unsigned)a.M;
    switch (team_waves(a.K, V)) {
        case 1:
            hipLaunchKernelGGL((layernorm_kernel<V, 1>), dim3(rows < 8192 ? rows : 8192), dim3(64), 0, stream, a);
            break;
        case 2:
            hipLaunchKernelGGL((layernorm_kernel<V, 2>), dim3(rows < 4096 ? rows : 4096), dim3(128), 0, stream, a);
            break;
        case 4:
            hipLaunchKernelGGL((layernorm_kernel<V, 4>), dim3(rows < 2048 ? rows : 2048), dim3(256), 0, stream, a);
            break;
        case 8:
            hipLaunchKernelGGL((layernorm_kernel<V, 8>), dim3(rows < 1024 ? rows : 1024), dim3(512), 0, stream, a);
            break;
        case 16:
            hipLaunchKernelGGL((layernorm_kernel<V, 16>), dim3(rows < 512 ? rows : 512), dim3(1024), 0, stream, a);
            break;
        default:
            hipLaunchKernelGGL((layernorm_long_kernel<V>), dim3(rows < 1024 ? rows : 1024), dim3(1024), 0, stream, a);
    }
    return hipGetLastError();
}

template <int V, bool CODES>
hipError_t launch_back_v(const NormBackArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)back_blocks(a.M, a.K));
    switch (back_waves(a.K, V)) {
        case 1:
            hipLaunchKernelGGL((layernorm_back_kernel<V, 1, 1, CODES>), grid, dim3(512), 0, stream, a);
            break;
        case 2:
            hipLaunchKernelGGL((layernorm_back_kernel<V, 2, 1, CODES>), grid, dim3(512), 0, stream, a);
            break;
        case 4:
            hipLaunchKernelGGL((layernorm_back_kernel<V, 4, 1, CODES>), grid, dim3(512), 0, stream, a);
            break;
        case 8:
            hipLaunchKernelGGL((layernorm_back_kernel<V, 8, 1, CODES>), grid, dim3(512), 0, stream, a);
            break;
        case 16:
            if (a.K <= (int64_t)16 * 64 * V)
                hipLaunchKernelGGL((layernorm_back_kernel<V, 16, 1, CODES>), grid, dim3(1024), 0, stream, a);
            else
                hipLaunchKernelGGL((layernorm_back_kernel<V, 16, 2, CODES>), grid, dim3(1024), 0, stream, a);
            break;
        default: {
            const unsigned rows = (unsigned)(a.M < 1024 ? a.M : 1024);
            hipLaunchKernelGGL((layernorm_back_long_kernel<V, CODES>), dim3(rows), dim3(1024), 0, stream, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || !a.part) return e;
            hipLaunchKernelGGL((layernorm_cols_kernel<CODES>), dim3((unsigned)((a.K + 255) / 256), grid.x),
                               dim3(256), 0, stream, a);
        }
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layernorm(const uint16_t* x, const float* w, const float* b, float eps, int64_t M,
                            int64_t K, uint16_t* y, int8_t* xq, float* a_scale, int pow2, float* mean,
                            float* rstd, hipStream_t stream) {
    const NormArgs a = {x, w, b, eps, M, K, y, xq, a_scale, pow2, mean, rstd};
    return K % 8 == 0 ? launch_layernorm_v<8>(a, stream) : launch_layernorm_v<4>(a, stream);
}

size_t layernorm_back_workspace_size(int64_t M, int64_t K) {
    return (size_t)back_blocks(M, K) * 2 * K * 4;
}

hipError_t launch_layernorm_back(const uint16_t* dy, const void* x, const float* x_scale, const float* w,
                                 const float* mean, const float* rstd, int64_t M, int64_t K, uint16_t* dx,
                                 float* dweight, float* dbias, void* workspace, hipStream_t stream) {
    const bool sums = dweight || dbias;
    if (M > 0) {
        const NormBackArgs a = {dy, x, x_scale, w, mean, rstd, M, K, dx,
                                sums ? static_cast<float*>(workspace) : nullptr};
        hipError_t e;
        if (x_scale)
            e = K % 8 == 0 ? launch_back_v<8, true>(a, stream) : launch_back_v<4, true>(a, stream);
        else
            e = K % 8 == 0 ? launch_back_v<8, false>(a, stream) : launch_back_v<4, false>(a, stream);
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    hipLaunchKernelGGL(layernorm_join_kernel, dim3((unsigned)((K + 63) / 64), 2), dim3(1024), 0, stream,
                       static_cast<const float*>(workspace), M > 0 ? (int)back_blocks(M, K) : 0, K, dweight,
                       dbias);
    return hipGetLastError();
}

hipError_t launch_dequant_act(const int8_t* xq, const float* a_scale, int64_t M, int64_t K, uint16_t* x,
                              hipStream_t stream) {
    const int V = K % 16 == 0 ? 16 : (K % 8 == 0 ? 8 : 4);
    const int64_t groups = K / V, bpr = (groups + 255) / 256;
    const int64_t step = max_blocks(256) / bpr;  // rows of a launch
    for (int64_t m = 0; m < M; m += step) {
        const dim3 grid((unsigned)((M - m < step ? M - m : step) * bpr)), block(256);
        const int8_t* const q = xq + m * K;
        const float* const a = a_scale + m;
        uint16_t* const out = x + m * K;
        if (V == 16)
            hipLaunchKernelGGL(dequant_kernel<16>, grid, block, 0, stream, q, a, groups, bpr, out);
        else if (V == 8)
            hipLaunchKernelGGL(dequant_kernel<8>, grid, block, 0, stream, q, a, groups, bpr, out);
        else
            hipLaunchKernelGGL(dequant_kernel<4>, grid, block, 0, stream, q, a, groups, bpr, out);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bitnet
