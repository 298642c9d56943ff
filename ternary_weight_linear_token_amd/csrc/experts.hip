// experts.hip -- the W2A8 product grouped by expert (mixture of experts) on gfx950.
//
//   out[p,n] = acc[p,n] w_scale[e,n] / a_scale[t],  acc[p,n] = sum_k xq[t,k] w[e,n,k]  (exact, int32)
//   for the rows p of expert e, offsets[e] <= p < offsets[e + 1], and their tokens t = rows[p]
//
// Two kernels.  What bounds the product is the bytes of the weights of the experts that have rows,
// while an expert has few, and the int8 matrix cores after that.
//  * expert_stream_kernel (a few rows for each expert): a block takes 16 rows of one expert times
//    16 NB rows of its weights and all of K, its waves interleaved 256-weight chunks of it; both
//    operands go straight from memory into registers.
//  * expert_tile_kernel: BM x BN tiles on v_mfma_i32_32x32x32_i8.  Activations pass through LDS
//    (two stages, transposed in groups of 4 x 4 bytes, 16-byte chunks XOR-swizzled by row so that
//    a fragment's rows fall in different banks); packed weights go straight into the registers of
//    the waves that use them and are expanded there.  Every matrix instruction is a slot that
//    also carries its share of the other work (an LDS read, a field of the next weights, a part
//    of the next stage's transposition), and nothing moves across slots, so that the waves of a
//    SIMD do not stand behind the matrix unit and then all behind the vector unit.
// In both the weights are the first operand, so a lane's accumulators are consecutive outputs of
// one row.  The gather of the tokens costs nothing in the loop: a thread reads the same rows of xq
// at every step, so it fetches their numbers once.
// A K that ends inside a step reads zeros of xq behind its end (whole chunks through the buffer
// descriptor's bounds, else by a mask); the weights behind the end are whatever lies there, times
// zero.  Rows behind an expert's last are computed from zeros and never stored.
#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"
#include "kernels.hpp"

namespace bitnet {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOut = 0x80000000u;  // offset behind every descriptor: reads zeros
constexpr int kXcds = 8;

struct ExpertArgs {
    const int8_t* xq;
    const float* a_scale;
    const int* rows;  // NULL: row p is token p
    const int* offsets;
    int T, P, E, K;
    int groups;
    int N[BITNET_MAX_GROUPS];
    int tile[BITNET_MAX_GROUPS + 1];  // first column tile of each matrix
    const uint8_t* packed[BITNET_MAX_GROUPS];
    const float* w_scale[BITNET_MAX_GROUPS];
    void* out[BITNET_MAX_GROUPS];
    int tiles_n;  // of all matrices
    int panel;    // row tiles of a panel
    int out_dtype;
    uint32_t first;  // first block of this launch
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}

// What a block works on; all uniform.
struct Unit {
    int e, m0, rows;  // expert, first row, number of rows
    int g, n0, N;     // matrix, first weight row, weight rows of an expert
};

// The block's unit.  Consecutive blocks go to different XCDs, so each XCD gets a contiguous run of
// units; runs walk panels of p.panel row tiles column by column, so that an XCD's L2 holds the
// panel's activations and the weights of few columns.
template <int BM, int BN>
__device__ __forceinline__ bool unit_of(const ExpertArgs& p, Unit& u) {
    const ExpertTiles<BM> tiles(p.offsets, p.E, p.P);
    const uint32_t units = (uint32_t)tiles.total * (uint32_t)p.tiles_n;
    const uint32_t b = p.first + blockIdx.x, xcd = b % kXcds, q = units / kXcds, r = units % kXcds;
    if (b / kXcds >= q + (xcd < r ? 1 : 0)) return false;
    const uint32_t t = xcd * q + min(xcd, r) + b / kXcds;
    const uint32_t per = (uint32_t)p.panel * (uint32_t)p.tiles_n, panel = t / per;
    const uint32_t high = min((uint32_t)p.panel, (uint32_t)tiles.total - panel * p.panel);
    const uint32_t in = t - panel * per;
    int col = (int)(in / high);
    tiles.find((int)(panel * p.panel + in % high), u.e, u.m0, u.rows);
    u.g = 0;
    u.N = p.N[0];
#pragma unroll
    for (int g = 1; g < BITNET_MAX_GROUPS; ++g)
        if (g < p.groups && col >= p.tile[g]) {
            u.g = g;
            u.N = p.N[g];
        }
#pragma unroll
    for (int g = 1; g < BITNET_MAX_GROUPS; ++g)
        if (u.g == g) col -= p.tile[g];
    u.n0 = col * BN;
    return true;
}

template <typename T>
__device__ __forceinline__ T pick(const T (&a)[BITNET_MAX_GROUPS], int g) {
    T r = a[0];
#pragma unroll
    for (int i = 1; i < BITNET_MAX_GROUPS; ++i) r = g == i ? a[i] : r;
    return r;
}

// Token of row i of the unit: -1 for a row behind the last or a token that is not there.
__device__ __forceinline__ int token_of(const ExpertArgs& p, const Unit& u, int i) {
    if (i >= u.rows) return -1;
    const int t = p.rows ? p.rows[u.m0 + i] : u.m0 + i;
    return (unsigned)t < (unsigned)p.T ? t : -1;
}

// ------------------------------------------------------------------------------ tiles
template <int BM, int BN, int WM, int WN, int W, bool ALIGNED>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), W) void expert_tile_kernel(ExpertArgs p) {
    constexpr int TH = 64 * (BM / WM) * (BN / WN);
    constexpr int MB = WM / 32, NB = WN / 32;
    constexpr int BK = 128, KS = BK / 32;  // a stage, and 32-k products of it
    constexpr int NA = BM * (BK / 16) / TH;  // 16-byte chunks of activations per thread and stage
    static_assert(NA >= 1 && NA * TH == BM * (BK / 16), "chunks");
    static_assert(TH % (BK / 16) == 0, "a thread keeps its chunk column");
    __shared__ __align__(1024) uint8_t lds[2][BM * BK];
    __shared__ float s_inva[BM];

    Unit u;
    if (!unit_of<BM, BN>(p, u)) return;
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, q = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / (BN / WN), wn = wave % (BN / WN);
    const int K = p.K, N = u.N, row_bytes = K / 4;
    const int nsteps = (K + BK - 1) / BK;

    // ---- loads ----
    // Activations: thread tid takes chunk tid % 8 of rows tid / 8 + j TH / 8.  Gathered rows are
    // addressed from the start of xq (the host has checked that 31 bits reach over it), sorted
    // ones from the tile's first.
    const int cc = tid % (BK / 16);
    const __amdgpu_buffer_rsrc_t ra =
        p.rows ? rsrc(p.xq, (uint32_t)(p.T * K)) : rsrc(p.xq + (int64_t)u.m0 * K, (uint32_t)(u.rows * K));
    uint32_t voff_a[NA];
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int t = token_of(p, u, tid / (BK / 16) + j * (TH / (BK / 16)));
        voff_a[j] = t < 0 ? kOut : (uint32_t)((p.rows ? t : t - u.m0) * K + 16 * cc);
    }
    for (int i = tid; i < BM; i += TH) {
        const int t = token_of(p, u, i);
        s_inva[i] = t < 0 ? 0.0f : 1.0f / p.a_scale[t];
    }
    // Weights: lane (l32, q) takes 16 packed bytes k / 4 = 16 q .. of row 32 i + l32 of the wave.
    const int rows_b = min(BN, N - u.n0);
    const uint8_t* wbase = pick(p.packed, u.g) + ((int64_t)u.e * N + u.n0) * row_bytes;
    const uint32_t skew = ALIGNED ? 0u : (uint32_t)((uintptr_t)wbase & 3);  // rows at any byte
    const __amdgpu_buffer_rsrc_t rb = rsrc(wbase - skew, (uint32_t)((rows_b * row_bytes + skew + 3) & ~3u));
    uint32_t voff_b[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int row = wn * WN + 32 * i + l32;
        // rows behind the last one read zeros (beside the descriptor's end in the last dword)
        voff_b[i] = row < rows_b ? (uint32_t)(row * row_bytes) + skew + 16 * q : kOut;
    }

    u32x4 ar[NA], br[2][NB];
    auto load_a = [&](int j, int step) {
        const int k0 = step * BK;
        // a chunk behind the row's end reads zeros; soff 0 keeps kOut from wrapping
        const bool in = k0 + 16 * cc < K && voff_a[j] != kOut;
        ar[j] = load16(ra, in ? voff_a[j] + k0 : kOut, 0);
    };
    // the part of a chunk behind the row's end (K % 16 != 0)
    auto mask_a = [&](int j, int step) {
        if (!ALIGNED) {
            const int left = K - step * BK - 16 * cc;  // bytes, a multiple of 4
#pragma unroll
            for (int d = 0; d < 4; ++d) ar[j][d] = left > 4 * d ? ar[j][d] : 0u;
        }
    };
    auto load_b = [&](int set, int i, int step) {
        const bool in = step < nsteps && voff_b[i] != kOut;
        const uint32_t off = in ? voff_b[i] + step * (BK / 4) : kOut;
        if (ALIGNED) {
            br[set][i] = load16(rb, off, 0);
        } else {
            const u32x4 v = load16(rb, off & ~3u, 0);
            const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(rb, (off & ~3u) + 16, 0, 0);
            const uint32_t sh = 8 * (off & 3);
            u32x4 o;
            o[0] = __builtin_amdgcn_alignbit(v[1], v[0], sh);
            o[1] = __builtin_amdgcn_alignbit(v[2], v[1], sh);
            o[2] = __builtin_amdgcn_alignbit(v[3], v[2], sh);
            o[3] = __builtin_amdgcn_alignbit(x, v[3], sh);
            br[set][i] = o;
        }
    };

    // Byte offset of chunk c of row r in a stage.
    auto at = [](int r, int c) { return r * BK + ((c ^ (r & 7)) << 4); };
    auto store_a = [&](int j, uint8_t* s) {
        const uint32_t d[4] = {ar[j][0], ar[j][1], ar[j][2], ar[j][3]};
        uint32_t e[4];
        transpose4x4_bytes(d, e);
        *reinterpret_cast<uint4*>(s + at(tid / (BK / 16) + j * (TH / (BK / 16)), cc)) =
            make_uint4(e[0], e[1], e[2], e[3]);
    };

    // ---- operands of 32 k: weights w (expanded), activations x (from LDS) ----
    struct Operands {
        v4i w[NB], x[MB];
    };
    Operands op[2];
    // lane group q owns the 16-weight groups 4 q + s of a stage
    auto expand = [&](Operands& o, const u32x4 (&b)[NB], int s, int part) {
        const int i = part >> 2;
        const uint32_t d = b[i][s];
        switch (part & 3) {
            case 0: o.w[i][0] = (int)ternary_field_i8<0>(d); break;
            case 1: o.w[i][1] = (int)ternary_field_i8<1>(d); break;
            case 2: o.w[i][2] = (int)ternary_field_i8<2>(d); break;
            default: o.w[i][3] = (int)ternary_field_i8<3>(d);
        }
    };
    int row_x[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j) row_x[j] = wm * WM + 32 * j + l32;
    auto read = [&](Operands& o, const uint8_t* stage, int s, int j) {
        o.x[j] = *reinterpret_cast<const v4i*>(stage + at(row_x[j], 4 * q + s));
    };

    v16i acc[MB][NB];
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0;

    // Step it multiplies stage it % 2 and weight set it % 2, while the activations of step it + 1, in
    // registers, go into the other stage and are loaded for step it + 2, and the other weight set
    // is loaded for it + 1.  One barrier a step, before its last 32 k, whose operands are already
    // in registers; the first operands of the next step are read behind it.
    constexpr int NM = MB * NB, S = (KS - 1) * NM;  // slots; those before the barrier
#pragma unroll
    for (int j = 0; j < NA; ++j) load_a(j, 0);
#pragma unroll
    for (int i = 0; i < NB; ++i) load_b(0, i, 0);
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        mask_a(j, 0);
        store_a(j, lds[0]);
        load_a(j, 1);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < MB; ++j) read(op[0], lds[0], 0, j);
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) expand(op[0], br[0], 0, e);
    auto step = [&](int it, auto set_c) {
        constexpr int set = decltype(set_c)::value;
        const uint8_t* const cur = lds[set];
        uint8_t* const nxt = lds[set ^ 1];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const bool last = s == KS - 1;
            if (last) __syncthreads();
            const Operands& o = op[s & 1];
            Operands& n = op[(s + 1) & 1];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                acc[m % MB][m / MB] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.w[m / MB], o.x[m % MB],
                                                                            acc[m % MB][m / MB], 0, 0, 0);
                const int slot = s * NM + m;
                if (slot < NB) load_b(set ^ 1, slot, it + 1);
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    if (j * ((NM + 1) / 2) / MB == m) read(n, last ? nxt : cur, last ? 0 : s + 1, j);
#pragma unroll
                for (int e = 0; e < 4 * NB; ++e)
                    if (NM / 2 + e * (NM - NM / 2) / (4 * NB) == m) expand(n, br[last ? set ^ 1 : set], last ? 0 : s + 1, e);
#pragma unroll
                for (int j = 0; j < NA; ++j)
                    if (j * S / NA + S / NA / 2 == slot) {
                        mask_a(j, it + 1);
                        store_a(j, nxt);
                        load_a(j, it + 2);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    int it = 0;
    for (; it + 2 <= nsteps; it += 2) {
        step(it, std::integral_constant<int, 0>());
        step(it + 1, std::integral_constant<int, 1>());
    }
    if (it < nsteps) step(it, std::integral_constant<int, 0>());

    // ---- outputs: lane (l32, q) of block (j, i) has row 32 j + l32, columns 32 i + 8 g + 4 q + 0 .. 3 ----
    const float* const ws = pick(p.w_scale, u.g) + (int64_t)u.e * N;
    void* const out = pick(p.out, u.g);
    const int dt = p.out_dtype;
    const bool wide = N % (dt == BITNET_OUT_BF16 ? 8 : 4) == 0;  // 16-byte aligned rows
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int nb = u.n0 + wn * WN + 32 * i;
        float sc[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int n = nb + 8 * (r >> 2) + 4 * q + (r & 3);
            sc[r] = n < N ? ws[n] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int ml = wm * WM + 32 * j + l32;
            const bool live = ml < u.rows;
            const float inv = s_inva[ml];
            const int64_t o = (int64_t)(u.m0 + ml) * N + nb;
            if (dt == BITNET_OUT_BF16 && wide && nb + 32 <= N) {
                uint32_t h[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    h[r] = f32x2_to_bf16x2_rne(((float)acc[j][i][2 * r] * sc[2 * r]) * inv,
                                               ((float)acc[j][i][2 * r + 1] * sc[2 * r + 1]) * inv);
                // lanes l and l + 32 hold the halves of 8 columns: exchange, so that each has 8
#pragma unroll
                for (int g = 0; g < 4; g += 2) {
                    const auto a = __builtin_amdgcn_permlane32_swap(h[2 * g], h[2 * g + 2], false, false);
                    const auto b = __builtin_amdgcn_permlane32_swap(h[2 * g + 1], h[2 * g + 3], false, false);
                    if (live)
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o + 8 * (g + q)) =
                            make_uint4(a[0], b[0], a[1], b[1]);
                }
            } else if (live) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = 8 * g + 4 * q;
                    if (dt != BITNET_OUT_BF16 && wide && nb + n + 4 <= N) {
                        uint4 v;
                        if (dt == BITNET_OUT_I32)
                            v = make_uint4((uint32_t)acc[j][i][4 * g], (uint32_t)acc[j][i][4 * g + 1],
                                           (uint32_t)acc[j][i][4 * g + 2], (uint32_t)acc[j][i][4 * g + 3]);
                        else
                            v = make_uint4(__float_as_uint(((float)acc[j][i][4 * g] * sc[4 * g]) * inv),
                                           __float_as_uint(((float)acc[j][i][4 * g + 1] * sc[4 * g + 1]) * inv),
                                           __float_as_uint(((float)acc[j][i][4 * g + 2] * sc[4 * g + 2]) * inv),
                                           __float_as_uint(((float)acc[j][i][4 * g + 3] * sc[4 * g + 3]) * inv));
                        *reinterpret_cast<uint4*>(static_cast<uint32_t*>(out) + o + n) = v;
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (nb + n + r < N)
                                store_out(out, o + n + r, dt, acc[j][i][4 * g + r], sc[4 * g + r], inv);
                    }
                }
            }
        }
    }
}

// ----------------------------------------------------------------------- few rows
constexpr int kStreamWaves = 4;

// 16 rows of one expert times 16 NB weight rows and all of K (K % 16 == 0).  Wave w takes the
// 256-weight chunks w, w + 4, ..; two batches of U chunks are in flight.
template <int NB, int U>
__global__ __launch_bounds__(64 * kStreamWaves) void expert_stream_kernel(ExpertArgs p) {
    constexpr int BN = 16 * NB;
    __shared__ int red[kStreamWaves][NB * 4 * 64];
    Unit u;
    if (!unit_of<16, BN>(p, u)) return;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.K, N = u.N, row_bytes = K / 4;
    const int nch = (K + 255) / 256;
    const int rows_b = min(BN, N - u.n0);
    const __amdgpu_buffer_rsrc_t rb = rsrc(
        pick(p.packed, u.g) + ((int64_t)u.e * N + u.n0) * row_bytes, (uint32_t)(rows_b * row_bytes));
    uint32_t voff_b[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)  // rows behind the last one read zeros
        voff_b[i] = 16 * i + l16 < rows_b ? (uint32_t)((16 * i + l16) * row_bytes + 16 * q) : kOut;
    const int token = token_of(p, u, l16);
    const __amdgpu_buffer_rsrc_t ra =
        p.rows ? rsrc(p.xq, (uint32_t)(p.T * K)) : rsrc(p.xq + (int64_t)u.m0 * K, (uint32_t)(u.rows * K));
    const uint32_t voff_a = token < 0 ? kOut : (uint32_t)((p.rows ? token : token - u.m0) * K + 64 * q);
    // the output pairs of this thread: scales asked for before the loop
    const int nj = (nch - wave + kStreamWaves - 1) / kStreamWaves;

    struct Chunk {
        u32x4 w[NB], x[4];
    };
    auto load_w = [&](int j, Chunk& c) {
        const int ch = wave + kStreamWaves * j;
#pragma unroll
        for (int i = 0; i < NB; ++i)
            c.w[i] = load16(rb, ch < nch && voff_b[i] != kOut ? voff_b[i] + 64 * ch : kOut, 0);
    };
    auto load_x = [&](int j, Chunk& c) {
        const int ch = wave + kStreamWaves * j;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = voff_a != kOut && 256 * ch + 64 * q + 16 * s < K;
            c.x[s] = load16(ra, in ? voff_a + 256 * ch + 16 * s : kOut, 0);
        }
    };
    v4i acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = v4i{0, 0, 0, 0};
    auto compute = [&](const Chunk& c) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t d[4] = {c.x[s][0], c.x[s][1], c.x[s][2], c.x[s][3]};
            uint32_t e[4];
            transpose4x4_bytes(d, e);
            const v4i x = {(int)e[0], (int)e[1], (int)e[2], (int)e[3]};
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const uint32_t b = c.w[i][s];
                const v4i w = {(int)ternary_field_i8<0>(b), (int)ternary_field_i8<1>(b),
                               (int)ternary_field_i8<2>(b), (int)ternary_field_i8<3>(b)};
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc[i], 0, 0, 0);
            }
        }
    };
    Chunk a[U], b[U];
#pragma unroll
    for (int k = 0; k < U; ++k) load_w(k, a[k]);
#pragma unroll
    for (int k = 0; k < U; ++k) load_x(k, a[k]);
    for (int j0 = 0; j0 < nj; j0 += 2 * U) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            load_w(j0 + U + k, b[k]);
            load_x(j0 + U + k, b[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (j0 + k < nj) compute(a[k]);
        if (j0 + U >= nj) break;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            load_w(j0 + 2 * U + k, a[k]);
            load_x(j0 + 2 * U + k, a[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (j0 + U + k < nj) compute(b[k]);
    }
    // 16x16 accumulator: lane l, register r -> weight row 4 (l / 16) + r, token l % 16
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][(16 * i + 4 * q + r) * 16 + l16] = acc[i][r];
    __syncthreads();
    const float* const ws = pick(p.w_scale, u.g) + (int64_t)u.e * N;
    void* const out = pick(p.out, u.g);
    for (int idx = tid; idx < BN * u.rows; idx += 64 * kStreamWaves) {
        const int m = idx / BN, n = idx % BN;
        if (n >= rows_b) continue;
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kStreamWaves; ++w) sum += red[w][n * 16 + m];
        const int t = token_of(p, u, m);
        store_out(out, (int64_t)(u.m0 + m) * N + u.n0 + n, p.out_dtype, sum, ws[u.n0 + n],
                  t < 0 ? 0.0f : 1.0f / p.a_scale[t]);
    }
}

// Codes and scales of the tokens rows[p], one group of a row per thread.
template <typename V>
__global__ __launch_bounds__(256) void gather_codes_kernel(const int8_t* __restrict__ xq,
                                                           const float* __restrict__ a_scale, int T,
                                                           const int* __restrict__ rows, int64_t groups,
                                                           int64_t blocks_per_row, int8_t* __restrict__ out,
                                                           float* __restrict__ out_scale) {
    const int64_t p = blockIdx.x / blocks_per_row;
    const int64_t g = (blockIdx.x - p * blocks_per_row) * blockDim.x + threadIdx.x;
    if (g >= groups) return;
    const int t = rows[p];
    const bool in = (unsigned)t < (unsigned)T;
    V v = {};
    if (in) v = reinterpret_cast<const V*>(xq)[t * groups + g];
    reinterpret_cast<V*>(out)[p * groups + g] = v;
    if (g == 0) out_scale[p] = in ? a_scale[t] : 1.0f;
}

template <class KERNEL>
hipError_t launch_units(KERNEL kernel, ExpertArgs a, int bm, int bn, int threads, int panel,
                        hipStream_t stream) {
    int64_t tn = 0;
    for (int g = 0; g < BITNET_MAX_GROUPS; ++g) {
        a.tile[g] = (int)tn;
        if (g < a.groups) tn += (a.N[g] + bn - 1) / bn;
    }
    a.tile[BITNET_MAX_GROUPS] = (int)tn;
    a.tiles_n = (int)tn;
    a.panel = panel;
    const int64_t units = expert_tiles(a.P, a.E, bm) * tn;
    // (units of 16 x 16 outputs at least: more than the card holds)
    if (units > INT32_MAX) return hipErrorInvalidValue;
    const int64_t most = max_blocks(threads) / kXcds * kXcds;
    const int64_t blocks = (units + kXcds - 1) / kXcds * kXcds;
    for (int64_t b = 0; b < blocks; b += most) {
        a.first = (uint32_t)b;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(threads), 0,
                           stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_gemm_experts(const int8_t* xq, const float* a_scale, int64_t T, const int* rows,
                               const int* offsets, int64_t P, int64_t E, int64_t K, int groups,
                               const uint8_t* const* packed, const float* const* w_scale,
                               const int64_t* N, void* const* out, int out_dtype, hipStream_t stream) {
    ExpertArgs a = {};
    a.xq = xq;
    a.a_scale = a_scale;
    a.rows = rows;
    a.offsets = offsets;
    a.T = (int)T;
    a.P = (int)P;
    a.E = (int)E;
    a.K = (int)K;
    a.out_dtype = out_dtype;
    for (int g = 0; g < groups; ++g) {
        if (N[g] == 0) continue;
        a.N[a.groups] = (int)N[g];
        a.packed[a.groups] = packed[g];
        a.w_scale[a.groups] = w_scale[g];
        a.out[a.groups++] = out[g];
    }
    const int64_t per = P / (E < P ? E : P);  // rows of an expert, if they are spread evenly
    const bool aligned = K % 16 == 0;
    if (aligned && per <= 16) return launch_units(expert_stream_kernel<2, 2>, a, 16, 32, 64 * kStreamWaves, 1, stream);
    if (per <= 64)
        return aligned ? launch_units(expert_tile_kernel<64, 128, 64, 32, 2, true>, a, 64, 128, 256, 2, stream)
                       : launch_units(expert_tile_kernel<64, 128, 64, 32, 2, false>, a, 64, 128, 256, 2, stream);
    if (per <= 192)
        return aligned ? launch_units(expert_tile_kernel<128, 128, 64, 64, 2, true>, a, 128, 128, 256, 4, stream)
                       : launch_units(expert_tile_kernel<128, 128, 64, 64, 2, false>, a, 128, 128, 256, 4, stream);
    return aligned ? launch_units(expert_tile_kernel<256, 256, 128, 64, 2, true>, a, 256, 256, 512, 4, stream)
                   : launch_units(expert_tile_kernel<256, 256, 128, 64, 2, false>, a, 256, 256, 512, 4, stream);
}

hipError_t launch_gather_codes(const int8_t* xq, const float* a_scale, int64_t T, const int* rows, int64_t P,
                               int64_t K, int8_t* out, float* out_scale, hipStream_t stream) {
    const int64_t groups = K / (K % 16 == 0 ? 16 : 4);
    const unsigned threads = groups < 256 ? (unsigned)((groups + 63) / 64 * 64) : 256;
    const int64_t bpr = (groups + threads - 1) / threads, step = max_blocks(256) / bpr;
    for (int64_t p = 0; p < P; p += step) {
        const int64_t n = P - p < step ? P - p : step;
        if (K % 16 == 0)
            hipLaunchKernelGGL(gather_codes_kernel<uint4>, dim3((unsigned)(n * bpr)), dim3(threads), 0, stream, xq,
                               a_scale, (int)T, rows + p, groups, bpr, out + p * K, out_scale + p);
        else
            hipLaunchKernelGGL(gather_codes_kernel<uint32_t>, dim3((unsigned)(n * bpr)), dim3(threads), 0, stream,
                               xq, a_scale, (int)T, rows + p, groups, bpr, out + p * K, out_scale + p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bitnet
