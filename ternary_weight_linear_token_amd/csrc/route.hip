// route.hip -- what stands before and behind the products of a mixture-of-experts layer on gfx950:
// the order of the tokens by expert, and the sum of a token's expert outputs with its backward.
//
//   order     the P = T J pairs (t, j), sorted by ids[t, j], pairs of one expert in their own
//             order: slots[t, j] = row of the pair, rows[row] = t, offsets[e] = first row of
//             expert e.  A pair whose id is not in 0 .. E - 1 is dropped: slot -1; the rows behind
//             offsets[E] belong to no pair and get token -1.
//   combine   out[t] = sum_j w[t, j] y[slots[t, j]], fp32, rounded once; dropped pairs add nothing
//   backward  dy[slots[t, j]] = w[t, j] dout[t],  dw[t, j] = sum_d dout[t, d] y[slots[t, j], d]
//
// Order: a counting sort without atomics between waves, so the order is the stable one.  Every wave
// owns a run of pairs and a histogram in LDS; lanes of a wave with the same expert find each
// other by one ballot per bit of the expert's number, and their first lane counts for all.  Then
// the prefix over experts, earlier blocks and earlier waves gives each wave the row where its first
// pair of an expert goes, and a second walk over the pairs hands out the rows.  Few pairs take one
// block; more take a launch that counts per block first.
// Combine and backward: bound by HBM, one pass.
// Measured: order of 256 pairs 4.0 us, of 16384 in two launches 4.7 and 5.8 (latency: loads, the
// ballots of a wave's pairs and the prefix follow one another); combine 8192 x 2 x 4096 39 us (201 MB,
// 5.2 TB/s), its backward 53 to 56 (336 MB, 6.0 to 6.3 TB/s, dout from a cache the second time).
#include "device_common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace bitnet {

namespace {

constexpr int kOrderWaves = 8;
constexpr int64_t kOrderChunk = 1024;  // fewest pairs of a block where there are several
constexpr int64_t kOrderBlocks = 256;
constexpr int kBins = BITNET_MAX_EXPERTS + 1;  // the last bin in use is that of the dropped pairs

struct OrderArgs {
    const void* ids;
    int wide;  // 64-bit ids
    int P, J, E, chunk;
    int* counts;  // (blocks, E + 1) with several blocks
    int *rows, *offsets, *slots;
};

// Bin of pair i.
__device__ __forceinline__ int bin_of(const OrderArgs& a, int i) {
    const int64_t id = a.wide ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int*>(a.ids)[i];
    return id >= 0 && id < a.E ? (int)id : a.E;
}

// Lanes of the wave that hold this lane's bin (`live` lanes only).
__device__ __forceinline__ uint64_t same_bin(int bin, bool live, int bits) {
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(bin >> b & 1);
        m &= bin >> b & 1 ? set : ~set;
    }
    return m;
}

// f(pair, bin, first lane of the bin, lanes before this one in it, lanes in it) for every pair of
// this wave's run.
template <class F>
__device__ __forceinline__ void walk(const OrderArgs& a, int bits, const F& f) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c0 = blockIdx.x * a.chunk;
    const int c1 = a.P - c0 < a.chunk ? a.P : c0 + a.chunk;
    const int run = ((c1 - c0 + kOrderWaves * 64 - 1) / (kOrderWaves * 64)) * 64;
    const int from = c0 + wave * run, to = c1 - from < run ? c1 : from + run;
    int next = from + lane < to ? bin_of(a, from + lane) : 0;
    for (int i = from; i < to; i += 64) {
        const int bin = next;
        next = i + 64 + lane < to ? bin_of(a, i + 64 + lane) : 0;  // ahead of its use
        const bool live = i + lane < to;
        const uint64_t m = same_bin(bin, live, bits);
        if (live)
            f(i + lane, bin, (int)__builtin_ctzll(m), (int)__popcll(m & (((uint64_t)1 << lane) - 1)),
              (int)__popcll(m));
    }
}

// Counts of this block's waves, hist[wave][bin].
__device__ __forceinline__ void count(const OrderArgs& a, int bits, int (&hist)[kOrderWaves][kBins]) {
    for (int i = threadIdx.x; i < kOrderWaves * kBins; i += 64 * kOrderWaves) (&hist[0][0])[i] = 0;
    __syncthreads();
    walk(a, bits, [&](int, int bin, int first, int, int lanes) {
        if ((int)(threadIdx.x & 63) == first) atomicAdd(&hist[threadIdx.x >> 6][bin], lanes);
    });
    __syncthreads();
}

__device__ __forceinline__ int bits_of(int E) { return 32 - __builtin_clz(E); }  // bins 0 .. E

__global__ __launch_bounds__(64 * kOrderWaves) void order_count_kernel(OrderArgs a) {
    __shared__ int hist[kOrderWaves][kBins];
    count(a, bits_of(a.E), hist);
    for (int e = threadIdx.x; e <= a.E; e += 64 * kOrderWaves) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kOrderWaves; ++w) sum += hist[w][e];
        a.counts[(int64_t)blockIdx.x * (a.E + 1) + e] = sum;
    }
}

__global__ __launch_bounds__(64 * kOrderWaves) void order_kernel(OrderArgs a) {
    __shared__ int hist[kOrderWaves][kBins];  // then the next row of each wave and bin
    __shared__ int s_total[kBins], s_before[kBins];  // of all blocks, of the earlier ones
    __shared__ int s_wave[kOrderWaves];
    constexpr int kThreads = 64 * kOrderWaves;
    const int bits = bits_of(a.E), tid = threadIdx.x;
    const bool alone = gridDim.x == 1;
    if (!alone)
        for (int e = tid; e <= a.E; e += kThreads) s_total[e] = s_before[e] = 0;
    count(a, bits, hist);
    if (!alone) {
        // the counts of all blocks in one run of loads (integers: any order of the additions)
        const int bins = a.E + 1, n = (int)gridDim.x * bins, mine = (int)blockIdx.x * bins;
#pragma unroll 8
        for (int i = tid; i < n; i += kThreads) {
            const int c = a.counts[i], e = i % bins;
            if (c == 0) continue;
            atomicAdd(&s_total[e], c);
            if (i < mine) atomicAdd(&s_before[e], c);
        }
        __syncthreads();
    }
    // a thread takes bins per * tid ..: their totals, and how many of them lie in earlier blocks
    constexpr int per = (kBins + kThreads - 1) / kThreads;
    int total[per], before[per], sum = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int e = per * tid + i;
        total[i] = before[i] = 0;
        if (e <= a.E) {
            if (alone) {
#pragma unroll
                for (int w = 0; w < kOrderWaves; ++w) total[i] += hist[w][e];
            } else {
                total[i] = s_total[e];
                before[i] = s_before[e];
            }
        }
        sum += total[i];
    }
    // rows before the thread's bins
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(scan, d);
        if ((tid & 63) >= d) scan += v;
    }
    if ((tid & 63) == 63) s_wave[tid >> 6] = scan;
    __syncthreads();
    int row = scan - sum;
    for (int w = 0; w < (tid >> 6); ++w) row += s_wave[w];
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int e = per * tid + i;
        if (e <= a.E) {
            if (blockIdx.x == 0) a.offsets[e] = row;  // offsets[E]: the first dropped row
            int at = row + before[i];
#pragma unroll
            for (int w = 0; w < kOrderWaves; ++w) {
                const int c = hist[w][e];
                hist[w][e] = at;
                at += c;
            }
        }
        row += total[i];
    }
    __syncthreads();
    walk(a, bits, [&](int i, int bin, int first, int earlier, int lanes) {
        int r = 0;
        if ((int)(tid & 63) == first) r = atomicAdd(&hist[tid >> 6][bin], lanes);
        r = __shfl(r, first) + earlier;
        a.rows[r] = bin < a.E ? i / a.J : -1;
        a.slots[i] = bin < a.E ? r : -1;
    });
}

// ------------------------------------------------------------------------- combine
struct CombineArgs {
    const uint16_t* y;
    const int* slots;
    const float* w;  // NULL: 1
    int P, J;
    int64_t T, groups;  // groups of V columns
    int64_t blocks_per_row;
    uint16_t* out;
};

// V columns of one token per thread; the loads of four pairs are on their way together.
template <int V>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs p) {
    const int64_t t = blockIdx.x / p.blocks_per_row;
    const int64_t g = (blockIdx.x - t * p.blocks_per_row) * blockDim.x + threadIdx.x;
    if (g >= p.groups) return;
    const int* const slots = p.slots + t * p.J;
    const float* const w = p.w ? p.w + t * p.J : nullptr;
    const int64_t D = p.groups * V;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    for (int j0 = 0; j0 < p.J; j0 += 4) {
        RowVec<V> v[4];
        float c[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int s = j0 + u < p.J ? slots[j0 + u] : -1;
            const bool in = (unsigned)s < (unsigned)p.P;
            v[u] = zero_row_vec<V>();
            c[u] = 0.0f;
            if (in) {
                v[u] = load_row_vec<V>(p.y + (int64_t)s * D, g);
                c[u] = w ? w[j0 + u] : 1.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float f[V];
            to_f32<V>(v[u], f);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] = __builtin_fmaf(c[u], f[j], sum[j]);
        }
    }
    RowVec<V> o;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) o.w[j] = f32x2_to_bf16x2_rne(sum[2 * j], sum[2 * j + 1]);
    store_row_vec<V>(p.out + t * D, g, o);
}

struct CombineBackArgs {
    const uint16_t *dout, *y;
    const int* slots;
    const float* w;  // NULL: 1
    int P, J;
    int64_t pairs, groups;
    uint16_t* dy;
    float* dw;  // NULL: not wanted
};

// One wave per pair; the pairs of a token are neighbours, so that dout comes from the CU's cache
// after the first.
template <int V>
__global__ __launch_bounds__(256) void combine_back_kernel(CombineBackArgs p) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (i >= p.pairs) return;
    const int s = p.slots[i];
    const bool in = (unsigned)s < (unsigned)p.P;
    float dot = 0.0f;
    if (in) {
        const int64_t D = p.groups * V;
        const uint16_t* const dout = p.dout + i / p.J * D;
        const float w = p.w ? p.w[i] : 1.0f;
        for (int64_t g0 = 0; g0 < p.groups; g0 += 256) {
            RowVec<V> d[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t g = g0 + 64 * u + lane;
                d[u] = y[u] = zero_row_vec<V>();
                if (g < p.groups) {
                    d[u] = load_row_vec<V>(dout, g);
                    if (p.dw) y[u] = load_row_vec<V>(p.y + s * D, g);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t g = g0 + 64 * u + lane;
                float f[V], h[V];
                to_f32<V>(d[u], f);
                to_f32<V>(y[u], h);
                RowVec<V> o;
#pragma unroll
                for (int j = 0; j < V; ++j) dot = __builtin_fmaf(f[j], h[j], dot);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) o.w[j] = f32x2_to_bf16x2_rne(w * f[2 * j], w * f[2 * j + 1]);
                if (g < p.groups) store_row_vec<V>(p.dy + s * D, g, o);
            }
        }
    }
    if (p.dw) {
        dot = wave_sum_f32(dot);
        if (lane == 0) p.dw[i] = dot;
    }
}

int64_t order_blocks(int64_t P) {
    if (P <= 2 * kOrderChunk) return 1;
    const int64_t b = (P + kOrderChunk - 1) / kOrderChunk;
    return b < kOrderBlocks ? b : kOrderBlocks;
}

}  // namespace

size_t expert_order_workspace_size(int64_t P, int64_t E) {
    const int64_t b = order_blocks(P);
    return b > 1 ? (size_t)b * (E + 1) * sizeof(int) : 0;
}

hipError_t launch_expert_order(const void* ids, int wide, int64_t T, int64_t J, int64_t E, int* rows,
                               int* offsets, int* slots, void* workspace, hipStream_t stream) {
    const int64_t P = T * J, blocks = order_blocks(P);
    OrderArgs a = {ids, wide, (int)P, (int)(J > 0 ? J : 1), (int)E, (int)((P + blocks - 1) / blocks),
                   static_cast<int*>(workspace), rows, offsets, slots};
    if (blocks > 1) {
        hipLaunchKernelGGL(order_count_kernel, dim3((unsigned)blocks), dim3(64 * kOrderWaves), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(order_kernel, dim3((unsigned)blocks), dim3(64 * kOrderWaves), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* y, const int* slots, const float* w, int64_t T, int64_t J,
                          int64_t P, int64_t D, uint16_t* out, hipStream_t stream) {
    const int V = D % 8 == 0 ? 8 : 4;
    const int64_t groups = D / V;
    const unsigned threads = groups < 256 ? (unsigned)((groups + 63) / 64 * 64) : 256;
    const int64_t bpr = (groups + threads - 1) / threads;
    const int64_t step = max_blocks(256) / bpr;  // tokens of a launch
    for (int64_t t = 0; t < T; t += step) {
        const int64_t n = T - t < step ? T - t : step;
        const CombineArgs a = {y, slots + t * J, w ? w + t * J : nullptr, (int)P, (int)J, n, groups, bpr,
                               out + t * D};
        if (V == 8)
            hipLaunchKernelGGL(combine_kernel<8>, dim3((unsigned)(n * bpr)), dim3(threads), 0, stream, a);
        else
            hipLaunchKernelGGL(combine_kernel<4>, dim3((unsigned)(n * bpr)), dim3(threads), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_combine_back(const uint16_t* dout, const uint16_t* y, const int* slots, const float* w,
                               int64_t T, int64_t J, int64_t P, int64_t D, uint16_t* dy, float* dw,
                               hipStream_t stream) {
    const int V = D % 8 == 0 ? 8 : 4;
    const int64_t step = max_blocks(256) / J * 4;  // tokens of a launch, four pairs a block
    for (int64_t t = 0; t < T; t += step) {
        const int64_t n = T - t < step ? T - t : step;
        const CombineBackArgs a = {dout + t * D, y, slots + t * J, w ? w + t * J : nullptr, (int)P, (int)J,
                                   n * J, D / V, dy, dw ? dw + t * J : nullptr};
        const dim3 grid((unsigned)((n * J + 3) / 4));
        if (V == 8)
            hipLaunchKernelGGL(combine_back_kernel<8>, grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL(combine_back_kernel<4>, grid, dim3(256), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bitnet
