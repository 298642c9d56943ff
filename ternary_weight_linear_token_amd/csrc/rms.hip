// rms.hip -- root-mean-square norm in front of a BitLinear layer, with the residual stream's
// addition and the int8 codes of its output in the same pass, and its backward, on gfx950.
//
//   forward   s = bf16(x + res) (or x), r = 1 / sqrt(mean_k s^2 + eps), y = bf16(s r w)
//             codes: those bitnet_quant_act (or _pow2) gives for the bf16 y
//   backward  z = s r, g = dy w:  dx = r (g - z mean_k(g z)) + dres,  dw = sum_m dy z
//             s as bf16 or as an 8-bit checkpoint
//
// Bound by HBM: every input is read once and every output written once.  The norm is of the
// rounded sum, the value that the next layer and the backward read, so s is rounded before it is
// squared.  Rows are taken by teams of waves as in the layer norm (rows.hpp): a lane keeps its
// elements in registers between the sum of squares and the outputs, and the next row of the
// block is on its way meanwhile.  Sums are fp32 in a fixed order.
// Measured: 2048 x 4096 with residual, codes and statistics 11.2 us (58.7 MB, 5.2 TB/s of which part
// stays in a cache); 1 x 2560 2.6 us; backward 8191 x 4100 from a checkpoint 38 to 41 us (235 MB, 5.9
// TB/s) and 4.7 for the join of the 512 partial column sums.  From bf16 with the residual's gradient, join
// included, replayed: 4096 x 8192 57 us (4.7 TB/s); 2048 x 12288 54 (3.7; from a checkpoint 53, 3.3), where a
// lane keeps 8 (16) of its values in scratch; 2048 x 16388, whose rows no block holds and which are read
// three times, 110 (2.4).
#include "device_common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace bitnet {

namespace {

struct RmsArgs {
    const uint16_t *x, *res;  // res NULL: nothing is added
    const float* w;           // NULL: 1
    float eps;
    int64_t M, K;
    uint16_t* sum;  // with res; may be x or res itself
    uint16_t* y;    // NULL: not written
    int8_t* xq;     // NULL: no codes
    float* a_scale;
    int pow2;
    float* rstd;  // NULL: not written
};

// x + res of V elements, each rounded to bf16 once.
template <int V>
__device__ __forceinline__ RowVec<V> add_rows(const RowVec<V>& x, const RowVec<V>& res) {
    float a[V], b[V];
    to_f32<V>(x, a);
    to_f32<V>(res, b);
    RowVec<V> s;
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
        s.w[j] = f32x2_to_bf16x2_rne(a[2 * j] + b[2 * j], a[2 * j + 1] + b[2 * j + 1]);
    return s;
}

// bf16(s r w) of V elements.
template <int V>
__device__ __forceinline__ RowVec<V> rms_output(const RowVec<V>& s, float r, const float (&w)[V]) {
    float f[V];
    to_f32<V>(s, f);
    RowVec<V> y;
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
        y.w[j] = f32x2_to_bf16x2_rne(f[2 * j] * r * w[2 * j], f[2 * j + 1] * r * w[2 * j + 1]);
    return y;
}

template <int V, int WPR, bool RES>
__global__ __launch_bounds__(64 * WPR) void rmsnorm_kernel(RmsArgs p) {
    constexpr int G = kTeamGroups, kStride = 64 * WPR;
    __shared__ float s_red[2][WPR];  // by the parity of the row: one barrier a row without codes
    __shared__ uint32_t s_max[WPR];
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    float w[G][V];
    bool in[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int64_t g = threadIdx.x + (int64_t)i * kStride;
        in[i] = g < groups;
        load_f32<V>(p.w, in[i] ? g : 0, 1.0f, w[i]);
    }
    RowVec<V> cur[G], res[G], nxt[G], nres[G];
    auto load = [&](int64_t m, RowVec<V> (&v)[G], RowVec<V> (&r)[G]) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            v[i] = zero_row_vec<V>();
            r[i] = zero_row_vec<V>();
            if (in[i] && m < p.M) {
                const int64_t g = threadIdx.x + (int64_t)i * kStride;
                v[i] = load_row_vec<V>(p.x + m * p.K, g);
                if (RES) r[i] = load_row_vec<V>(p.res + m * p.K, g);
            }
        }
    };
    load(blockIdx.x, cur, res);
    int parity = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, parity ^= 1) {
        load(m + gridDim.x, nxt, nres);
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            if (RES) {
                cur[i] = add_rows<V>(cur[i], res[i]);
                if (in[i]) store_row_vec<V>(p.sum + m * p.K, threadIdx.x + (int64_t)i * kStride, cur[i]);
            }
            float f[V];
            to_f32<V>(cur[i], f);
#pragma unroll
            for (int j = 0; j < V; ++j) sq = __builtin_fmaf(f[j], f[j], sq);
        }
        const float rstd =
            __builtin_amdgcn_rsqf(__builtin_fmaf(team_sum<WPR>(sq, s_red[parity]), inv_k, p.eps));
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            cur[i] = rms_output<V>(cur[i], rstd, w[i]);
            if (in[i]) {
                if (p.y) store_row_vec<V>(p.y + m * p.K, threadIdx.x + (int64_t)i * kStride, cur[i]);
                mx = max_pairs<V>(cur[i], mx);
            }
        }
        if (threadIdx.x == 0 && p.rstd) p.rstd[m] = rstd;
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
        for (int i = 0; i < G; ++i) {
            cur[i] = nxt[i];
            res[i] = nres[i];
        }
    }
}

// Rows too long for a team's registers: one block of 16 waves per row.  The first pass writes the
// sum, which the later ones read (a thread reads what it wrote itself, so the sum may take the
// place of x or of the residual).
template <int V, bool RES>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(RmsArgs p) {
    constexpr int WPR = 16;
    __shared__ float s_red[2][WPR];
    __shared__ uint32_t s_max[WPR];
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    int parity = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, parity ^= 1) {
        const uint16_t* row = p.x + m * p.K;
        float f[V], sq = 0.0f;
        for (int64_t g = threadIdx.x; g < groups; g += 1024) {
            RowVec<V> v = load_row_vec<V>(row, g);
            if (RES) {
                v = add_rows<V>(v, load_row_vec<V>(p.res + m * p.K, g));
                store_row_vec<V>(p.sum + m * p.K, g, v);
            }
            to_f32<V>(v, f);
#pragma unroll
            for (int j = 0; j < V; ++j) sq = __builtin_fmaf(f[j], f[j], sq);
        }
        if (RES) row = p.sum + m * p.K;
        const float rstd =
            __builtin_amdgcn_rsqf(__builtin_fmaf(team_sum<WPR>(sq, s_red[parity]), inv_k, p.eps));
        auto output = [&](int64_t g) {
            float w[V];
            load_f32<V>(p.w, g, 1.0f, w);
            return rms_output<V>(load_row_vec<V>(row, g), rstd, w);
        };
        uint32_t mx = 0;
        for (int64_t g = threadIdx.x; g < groups; g += 1024) {
            const RowVec<V> y = output(g);
            if (p.y) store_row_vec<V>(p.y + m * p.K, g, y);
            mx = max_pairs<V>(y, mx);
        }
        if (threadIdx.x == 0 && p.rstd) p.rstd[m] = rstd;
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
struct RmsBackArgs {
    const uint16_t* dy;
    const void* x;         // bf16, or int8 codes with x_scale
    const float* x_scale;  // NULL: x is bf16
    const float *w, *rstd;
    const uint16_t* dres;  // NULL: nothing is added
    int64_t M, K;
    uint16_t* dx;
    float* part;  // (blocks, K) column sums (of a single block: dweight itself), NULL: not wanted
};

// Blocks of TEAMS teams; the teams of a block walk the rows in step (every wave reaches every
// barrier; a team past the last row works on zeros).  From codes c = a s the norm is z =
// c (r / a).
template <int V, int WPR, int G, bool CODES, bool RES>
__global__ __launch_bounds__(WPR == 16 ? 1024 : 512) void rmsnorm_back_kernel(RmsBackArgs p) {
    constexpr int kStride = 64 * WPR, TEAMS = WPR == 16 ? 1 : 8 / WPR;
    __shared__ float s_red[2][TEAMS][WPR];
    __shared__ float s_join[TEAMS > 1 ? kStride * G * V : 1];
    const int team = threadIdx.x / kStride, lr = threadIdx.x % kStride;
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    float w[G][V], dw[G][V];
    bool in[G], some[G];  // of this lane, of this wave
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int64_t g = lr + (int64_t)i * kStride;
        in[i] = g < groups;
        some[i] = i == 0 || __builtin_amdgcn_readfirstlane((int)(__ballot(in[i]) != 0)) != 0;
        load_f32<V>(p.w, in[i] ? g : 0, 1.0f, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.0f;
    }
    struct Row {
        RowVec<V> dy[G], dres[RES ? G : 1];
        XVec<V, CODES> x[G];
        float rstd, a;
    };
    auto load = [&](int64_t m, Row& r) {
        const bool live = m < p.M;
        r.rstd = live ? p.rstd[m] : 0.0f;
        r.a = 1.0f;
        if (CODES && live) r.a = p.x_scale[m];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            r.dy[i] = zero_row_vec<V>();
            r.x[i] = XVec<V, CODES>{};
            if (RES) r.dres[i] = zero_row_vec<V>();
            if (live && in[i]) {
                const int64_t g = lr + (int64_t)i * kStride;
                r.dy[i] = load_row_vec<V>(p.dy + m * p.K, g);
                r.x[i] = load_x<V, CODES>(p.x, m * p.K, g);
                if (RES) r.dres[i] = load_row_vec<V>(p.dres + m * p.K, g);
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
        float z[G][V], g[G][V], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            if (!some[i]) continue;
            float d[V];
            to_f32<V>(cur.dy[i], d);
            x_to_f32<V, CODES>(cur.x[i], z[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                z[i][j] *= scale;
                dw[i][j] = __builtin_fmaf(d[j], z[i][j], dw[i][j]);
                g[i][j] = d[j] * w[i][j];
                dot = __builtin_fmaf(g[i][j], z[i][j], dot);
            }
        }
        dot = wave_sum_f32(dot);
        if (WPR > 1) {
            float(&red)[WPR] = s_red[parity][team];
            if ((threadIdx.x & 63) == 0) red[lr >> 6] = dot;
            __syncthreads();
            dot = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) dot += red[i];
        }
        const float c = -cur.rstd * (dot * inv_k);
        if (m < p.M) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (!some[i]) continue;
                float r[V];
                if (RES) to_f32<V>(cur.dres[RES ? i : 0], r);
                RowVec<V> o;
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float v0 = __builtin_fmaf(c, z[i][2 * j], cur.rstd * g[i][2 * j]);
                    const float v1 = __builtin_fmaf(c, z[i][2 * j + 1], cur.rstd * g[i][2 * j + 1]);
                    o.w[j] = RES ? f32x2_to_bf16x2_rne(v0 + r[2 * j], v1 + r[2 * j + 1])
                                 : f32x2_to_bf16x2_rne(v0, v1);
                }
                if (in[i]) store_row_vec<V>(p.dx + m * p.K, lr + (int64_t)i * kStride, o);
            }
        }
        cur = nxt;
    }
    if (!p.part) return;
    for (int tm = 1; tm < TEAMS; ++tm) {
        __syncthreads();
        if (team == tm) {
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s_join[(i * V + j) * kStride + lr] = dw[i][j];
        }
        __syncthreads();
        if (team == 0) {
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) dw[i][j] += s_join[(i * V + j) * kStride + lr];
        }
    }
    if (team == 0) {
        float* const part = p.part + (int64_t)blockIdx.x * p.K;
#pragma unroll
        for (int i = 0; i < G; ++i)
            if (in[i]) {
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    *reinterpret_cast<float4*>(part + (lr + (int64_t)i * kStride) * V + j) =
                        make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
            }
    }
}

// dx of rows too long for a team's registers: one block per row, two reads.
template <int V, bool CODES>
__global__ __launch_bounds__(1024) void rmsnorm_back_long_kernel(RmsBackArgs p) {
    constexpr int WPR = 16;
    __shared__ float s_red[2][WPR];
    const int64_t groups = p.K / V;
    const float inv_k = 1.0f / (float)p.K;
    int parity = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, parity ^= 1) {
        const float rstd = p.rstd[m], scale = CODES ? rstd / p.x_scale[m] : rstd;
        float z[V], g[V], dot = 0.0f;
        auto read = [&](int64_t i) {
            float d[V], w[V];
            to_f32<V>(load_row_vec<V>(p.dy + m * p.K, i), d);
            x_to_f32<V, CODES>(load_x<V, CODES>(p.x, m * p.K, i), z);
            load_f32<V>(p.w, i, 1.0f, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                z[j] *= scale;
                g[j] = d[j] * w[j];
            }
        };
        for (int64_t i = threadIdx.x; i < groups; i += 1024) {
            read(i);
#pragma unroll
            for (int j = 0; j < V; ++j) dot = __builtin_fmaf(g[j], z[j], dot);
        }
        const float c = -rstd * (team_sum<WPR>(dot, s_red[parity]) * inv_k);
        for (int64_t i = threadIdx.x; i < groups; i += 1024) {
            read(i);
            float r[V] = {};
            if (p.dres) to_f32<V>(load_row_vec<V>(p.dres + m * p.K, i), r);
            RowVec<V> o;
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
                o.w[j] = f32x2_to_bf16x2_rne(
                    __builtin_fmaf(c, z[2 * j], rstd * g[2 * j]) + r[2 * j],
                    __builtin_fmaf(c, z[2 * j + 1], rstd * g[2 * j + 1]) + r[2 * j + 1]);
            store_row_vec<V>(p.dx + m * p.K, i, o);
        }
    }
}

// Column sums of such rows: block (c, s) takes 256 columns of every gridDim.y-th row.
template <bool CODES>
__global__ __launch_bounds__(256) void rmsnorm_cols_kernel(RmsBackArgs p) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= p.K) return;
    float dw = 0.0f;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        const float d = bf16_bits_to_f32(p.dy[m * p.K + k]);
        float z;
        if (CODES)
            z = (float)static_cast<const int8_t*>(p.x)[m * p.K + k] * (p.rstd[m] / p.x_scale[m]);
        else
            z = bf16_bits_to_f32(static_cast<const uint16_t*>(p.x)[m * p.K + k]) * p.rstd[m];
        dw = __builtin_fmaf(d, z, dw);
    }
    p.part[(int64_t)blockIdx.y * p.K + k] = dw;
}

// dweight[k] = sum_b part[b][k]: 64 columns per block, 64 rows of 16 threads that each add every
// 64th partial of four columns, then the 64 sums of a column in order.
__global__ __launch_bounds__(1024) void rmsnorm_join_kernel(const float* __restrict__ part, int blocks,
                                                            int64_t K, float* dweight) {
    __shared__ float s[64][68];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int64_t k = (int64_t)blockIdx.x * 64 + 4 * c;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (k < K) {
#pragma unroll 4
        for (int b = r; b < blocks; b += 64) {
            const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)b * K + k);
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
        dweight[kc] = t;
    }
}

// Blocks of the backward pass.
int64_t rms_back_blocks(int64_t M, int64_t K) {
    const int w = back_waves(K, K % 8 == 0 ? 8 : 4);
    if (w == 0) return M < 64 * 32 ? (M + 31) / 32 : 64;
    const int64_t teams = w == 16 ? 1 : 8 / w;
    // few rows: one block, whose column sums are dweight, costs no second launch and no workspace (a call
    // of 8 rows of 2560 columns 9.8 us against 14.1, replayed in a graph 6.9 against 5.3; 32 of 512 9.8
    // against 14.1, 6.6 against 5.3; 4 of 8192 9.9 against 14.0, 6.1 against 6.5)
    if (M <= (w == 16 ? 4 : 8) * teams) return 1;
    const int64_t b = (M + 2 * teams - 1) / (2 * teams);
    return b < 512 ? b : 512;
}

template <int V, bool RES>
hipError_t launch_rmsnorm_v(const RmsArgs& a, hipStream_t stream) {
    const unsigned rows = (unsigned)a.M;
    auto grid = [&](unsigned most) { return dim3(rows < most ? rows : most); };
    switch (team_waves(a.K, V)) {
        case 1: hipLaunchKernelGGL((rmsnorm_kernel<V, 1, RES>), grid(8192), dim3(64), 0, stream, a); break;
        case 2: hipLaunchKernelGGL((rmsnorm_kernel<V, 2, RES>), grid(4096), dim3(128), 0, stream, a); break;
        case 4: hipLaunchKernelGGL((rmsnorm_kernel<V, 4, RES>), grid(2048), dim3(256), 0, stream, a); break;
        case 8: hipLaunchKernelGGL((rmsnorm_kernel<V, 8, RES>), grid(1024), dim3(512), 0, stream, a); break;
        case 16: hipLaunchKernelGGL((rmsnorm_kernel<V, 16, RES>), grid(512), dim3(1024), 0, stream, a); break;
        default: hipLaunchKernelGGL((rmsnorm_long_kernel<V, RES>), grid(1024), dim3(1024), 0, stream, a);
    }
    return hipGetLastError();
}

template <int V, bool CODES, bool RES>
hipError_t launch_rms_back_v(const RmsBackArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)rms_back_blocks(a.M, a.K));
    switch (back_waves(a.K, V)) {
        case 1: hipLaunchKernelGGL((rmsnorm_back_kernel<V, 1, 1, CODES, RES>), grid, dim3(512), 0, stream, a); break;
        case 2: hipLaunchKernelGGL((rmsnorm_back_kernel<V, 2, 1, CODES, RES>), grid, dim3(512), 0, stream, a); break;
        case 4: hipLaunchKernelGGL((rmsnorm_back_kernel<V, 4, 1, CODES, RES>), grid, dim3(512), 0, stream, a); break;
        case 8: hipLaunchKernelGGL((rmsnorm_back_kernel<V, 8, 1, CODES, RES>), grid, dim3(512), 0, stream, a); break;
        case 16:
            if (a.K <= (int64_t)16 * 64 * V) {
                hipLaunchKernelGGL((rmsnorm_back_kernel<V, 16, 1, CODES, RES>), grid, dim3(1024), 0, stream, a);
                break;
            }
            // two groups a lane with 16 waves fill a CU with one block; eight waves with three leave
            // room for two (8191 x 4100 from a checkpoint: 57 -> 40 us; rows of whole eights never come
            // here with three)
            if constexpr (V == 4)
                if (a.K <= (int64_t)8 * 64 * 3 * V) {
                    hipLaunchKernelGGL((rmsnorm_back_kernel<V, 8, 3, CODES, RES>), grid, dim3(512), 0, stream, a);
                    break;
                }
            hipLaunchKernelGGL((rmsnorm_back_kernel<V, 16, 2, CODES, RES>), grid, dim3(1024), 0, stream, a);
            break;
        default: {
            const unsigned rows = (unsigned)(a.M < 1024 ? a.M : 1024);
            hipLaunchKernelGGL((rmsnorm_back_long_kernel<V, CODES>), dim3(rows), dim3(1024), 0, stream, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || !a.part) return e;
            hipLaunchKernelGGL((rmsnorm_cols_kernel<CODES>), dim3((unsigned)((a.K + 255) / 256), grid.x),
                               dim3(256), 0, stream, a);
        }
    }
    return hipGetLastError();
}

template <bool CODES, bool RES>
hipError_t launch_rms_back(const RmsBackArgs& a, hipStream_t stream) {
    return a.K % 8 == 0 ? launch_rms_back_v<8, CODES, RES>(a, stream)
                        : launch_rms_back_v<4, CODES, RES>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm(const uint16_t* x, const uint16_t* res, const float* w, float eps, int64_t M,
                          int64_t K, uint16_t* sum, uint16_t* y, int8_t* xq, float* a_scale, int pow2,
                          float* rstd, hipStream_t stream) {
    const RmsArgs a = {x, res, w, eps, M, K, sum, y, xq, a_scale, pow2, rstd};
    if (K % 8 == 0)
        return res ? launch_rmsnorm_v<8, true>(a, stream) : launch_rmsnorm_v<8, false>(a, stream);
    return res ? launch_rmsnorm_v<4, true>(a, stream) : launch_rmsnorm_v<4, false>(a, stream);
}

size_t rmsnorm_back_workspace_size(int64_t M, int64_t K) {
    const int64_t blocks = rms_back_blocks(M, K);
    return blocks > 1 ? (size_t)blocks * K * 4 : 0;
}

hipError_t launch_rmsnorm_back(const uint16_t* dy, const void* x, const float* x_scale, const float* w,
                               const float* rstd, const uint16_t* dres, int64_t M, int64_t K, uint16_t* dx,
                               float* dweight, void* workspace, hipStream_t stream) {
    const int64_t blocks = M > 0 ? rms_back_blocks(M, K) : 0;
    if (M > 0) {
        // a single block writes the column sums as they are
        float* const part = blocks == 1 ? dweight : static_cast<float*>(workspace);
        const RmsBackArgs a = {dy, x, x_scale, w, rstd, dres, M, K, dx, dweight ? part : nullptr};
        hipError_t e;
        if (x_scale)
            e = dres ? launch_rms_back<true, true>(a, stream) : launch_rms_back<true, false>(a, stream);
        else
            e = dres ? launch_rms_back<false, true>(a, stream) : launch_rms_back<false, false>(a, stream);
        if (e != hipSuccess) return e;
    }
    if (!dweight || blocks == 1) return hipSuccess;
    hipLaunchKernelGGL(rmsnorm_join_kernel, dim3((unsigned)((K + 63) / 64)), dim3(1024), 0, stream,
                       static_cast<const float*>(workspace), (int)blocks, K, dweight);
    return hipGetLastError();
}

}  // namespace bitnet
