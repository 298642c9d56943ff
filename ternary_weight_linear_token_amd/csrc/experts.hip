// experts.hip -- the W2A8 product grouped by expert (mixture of experts) on gfx950.
//
//   out[p,n] = acc[p,n] w_scale[e,n] / a_scale[t],  acc[p,n] = sum_k xq[t,k] w[e,n,k]  (exact, int32)
//   for the rows p of expert e, offsets[e] <= p < offsets[e + 1], and their tokens t = rows[p]
//
// Two kernels.  What bounds the product is the bytes of the weights of the experts that have rows,
// while an expert has few, and the int8 matrix cores after that.
//  * expert_stream_kernel (a few rows for each expert): a block takes 16 rows of one expert times
//    64 rows of its weights and all of K, its waves interleaved 256-weight chunks of it; both
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
// Measured: one token, two of 8 experts of 14336 x 4096, gate and up 15.7 us (59 MB, 3.8 TB/s: the launch
// and one chain of loads, products and the join of four waves); 32 tokens, 8 of 64 experts of 640 x 2560
// 15.4 us (53 MB); 4096 rows of 8 experts of 14336 x 4096, gate and up 458 to 490 us (1.96 to 2.1 POP/s, the
// matrix cores busy 61% of the cycles of a chip that holds about 1.8 GHz under such a load; a library's
// int8 product of one large matrix 2.07).
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

// Descriptor of a uniform range, in scalar registers wherever it was computed: in vector registers it
// would put a loop over the lanes around every load.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)b) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)u, (short)0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}

// What a block works on; all uniform.
struct Unit {
    int e, m0, rows;  // expert, first row, number of rows
    int g, n0, N;     // matrix, first weight row, weight rows of an expert
};

// Matrix and first weight row of column tile col of all matrices.
template <int BN>
__device__ __forceinline__ void column_of(const ExpertArgs& p, int col, Unit& u) {
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
}

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
    const int col = (int)(in / high);
    tiles.find((int)(panel * p.panel + in % high), u.e, u.m0, u.rows);
    column_of<BN>(p, col, u);
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
template <int BM, int BN, int WM, int WN, int G, int D, int W, bool ALIGNED>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN) * G, W) void expert_tile_kernel(ExpertArgs p) {
    constexpr int WPG = (BM / WM) * (BN / WN), TH = 64 * WPG;  // waves, threads of a group
    constexpr int MB = WM / 32, NB = WN / 32;
    constexpr int BK = 128, KS = BK / 32;  // a stage, and 32-k products of it
    constexpr int NA = BM * (BK / 16) / TH;  // 16-byte chunks of activations per thread and stage
    static_assert(NA >= 1 && NA * TH == BM * (BK / 16), "chunks");
    static_assert(TH % (BK / 16) == 0, "a thread keeps its chunk column");
    constexpr int kStage = BM * BK, kSums = WPG * MB * NB * 16 * 64 * 4;  // bytes of a stage; of a group's sums
    constexpr int kLds = G * (2 * kStage > kSums && G > 1 ? 2 * kStage : (G > 1 ? kSums : 2 * kStage));
    __shared__ __align__(1024) uint8_t smem[kLds];
    __shared__ float s_inva[BM];

    Unit u;
    if (!unit_of<BM, BN>(p, u)) return;
    // G groups of waves share a tile: group g takes the stages g, g + G, ..; all run as many
    const int g = G > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / TH) : 0;
    const int tid = threadIdx.x - g * TH, lane = tid & 63, l32 = lane & 31, q = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / (BN / WN), wn = wave % (BN / WN);
    const int K = p.K, N = u.N, row_bytes = K / 4;
    const int nsteps = ((K + BK - 1) / BK + G - 1) / G;
    uint8_t* const lds = smem + g * 2 * kStage;

    // ---- loads ----
    // Activations: thread tid takes chunk tid % 8 of rows tid / 8 + j TH / 8.  Gathered rows are
    // addressed from the start of xq (the host has checked that 31 bits reach over it), sorted
    // ones from the tile's first.
    const int cc = tid % (BK / 16);
    const __amdgpu_buffer_rsrc_t ra =
        rsrc(p.xq + (p.rows ? 0 : (int64_t)u.m0 * K), (uint32_t)((p.rows ? p.T : u.rows) * K));
    uint32_t voff_a[NA];
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int t = token_of(p, u, tid / (BK / 16) + j * (TH / (BK / 16)));
        voff_a[j] = t < 0 ? kOut : (uint32_t)((p.rows ? t : t - u.m0) * K + 16 * cc);
    }
    for (int i = threadIdx.x; i < BM; i += TH * G) {
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

    // Activations are loaded D steps before they go to LDS, weights one step before their use.
    static_assert(D == 1 || D == 2, "sets go round with the stages");
    u32x4 ar[D][NA], br[2][NB];
    auto load_a = [&](int set, int j, int step) {
        const int k0 = (step * G + g) * BK;
        // a chunk behind the row's end reads zeros; soff 0 keeps kOut from wrapping
        const bool in = k0 + 16 * cc < K && voff_a[j] != kOut;
        ar[set][j] = load16(ra, in ? voff_a[j] + k0 : kOut, 0);
    };
    // the part of a chunk behind the row's end (K % 16 != 0)
    auto mask_a = [&](int set, int j, int step) {
        if (!ALIGNED) {
            const int left = K - (step * G + g) * BK - 16 * cc;  // bytes, a multiple of 4
#pragma unroll
            for (int d = 0; d < 4; ++d) ar[set][j][d] = left > 4 * d ? ar[set][j][d] : 0u;
        }
    };
    auto load_b = [&](int set, int i, int step) {
        const bool in = step < nsteps && voff_b[i] != kOut;
        const uint32_t off = in ? voff_b[i] + (step * G + g) * (BK / 4) : kOut;
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
    auto store_a = [&](int set, int j, uint8_t* s) {
        const uint32_t d[4] = {ar[set][j][0], ar[set][j][1], ar[set][j][2], ar[set][j][3]};
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

    // Step it multiplies stage and weight set it % 2, while the activations of step it + 1, in
    // registers, go into the other stage and their registers are loaded for step it + 1 + D, and
    // the other weight set for step it + 1.  One barrier a step, before its last 32 k, whose
    // operands are already in registers; the first operands of the next step are read behind it.
    constexpr int NM = MB * NB, S = (KS - 1) * NM;  // slots; those before the barrier
#pragma unroll
    for (int i = 0; i < NB; ++i) load_b(0, i, 0);
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int j = 0; j < NA; ++j) load_a(d, j, d);
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        mask_a(0, j, 0);
        store_a(0, j, lds);
        load_a(0, j, D);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < MB; ++j) read(op[0], lds, 0, j);
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) expand(op[0], br[0], 0, e);
    auto step = [&](int it, auto at_c) {
        constexpr int at = decltype(at_c)::value;  // it % 2
        constexpr int a_set = (at + 1) % D;
        const uint8_t* const cur = lds + at * kStage;
        uint8_t* const nxt = lds + (at ^ 1) * kStage;
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
                if (slot < NB) load_b(at ^ 1, slot, it + 1);
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    if (j * ((NM + 1) / 2) / MB == m) read(n, last ? nxt : cur, last ? 0 : s + 1, j);
#pragma unroll
                for (int e = 0; e < 4 * NB; ++e)
                    if (NM / 2 + e * (NM - NM / 2) / (4 * NB) == m)
                        expand(n, br[last ? at ^ 1 : at], last ? 0 : s + 1, e);
#pragma unroll
                for (int j = 0; j < NA; ++j)
                    if (j * S / NA + S / NA / 2 == slot) {
                        mask_a(a_set, j, it + 1);
                        store_a(a_set, j, nxt);
                        load_a(a_set, j, it + 1 + D);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // pairs of steps, then the odd one (an exit inside the loop would give the accumulators a
    // second live range)
    int it = 0;
    for (; it + 2 <= nsteps; it += 2) {
        step(it, std::integral_constant<int, 0>());
        step(it + 1, std::integral_constant<int, 1>());
    }
    if (it < nsteps) step(it, std::integral_constant<int, 0>());

    // ---- outputs: lane (l32, q) of block (j, i) has row 32 j + l32, columns 32 i + 8 c + 4 q + 0 .. 3 in
    // registers 4 c ..; eight registers at a time (h: c = 2 h and 2 h + 1) ----
    const float* const ws = pick(p.w_scale, u.g) + (int64_t)u.e * N;
    void* const out = pick(p.out, u.g);
    const int dt = p.out_dtype;
    const bool wide = N % (dt == BITNET_OUT_BF16 ? 8 : 4) == 0;  // 16-byte aligned rows
    auto scales = [&](int i, int h, float (&sc)[8]) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int n = u.n0 + wn * WN + 32 * i + 16 * h + 8 * (r >> 2) + 4 * q + (r & 3);
            sc[r] = n < N ? ws[n] : 0.0f;
        }
    };
    auto emit = [&](int j, int i, int h, const int (&v)[8], const float (&sc)[8]) {
        const int nb = u.n0 + wn * WN + 32 * i + 16 * h;
        const int ml = wm * WM + 32 * j + l32;
        const bool live = ml < u.rows;
        const float inv = s_inva[ml];
        const int64_t o = (int64_t)(u.m0 + ml) * N + nb;
        if (dt == BITNET_OUT_BF16 && wide && nb + 16 <= N) {
            uint32_t b[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                b[r] = f32x2_to_bf16x2_rne(((float)v[2 * r] * sc[2 * r]) * inv,
                                           ((float)v[2 * r + 1] * sc[2 * r + 1]) * inv);
            // lanes l and l + 32 hold the halves of 8 columns: exchange, so that each has 8
            const auto x = __builtin_amdgcn_permlane32_swap(b[0], b[2], false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(b[1], b[3], false, false);
            if (live)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o + 8 * q) =
                    make_uint4(x[0], y[0], x[1], y[1]);
        } else if (live) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int n = 8 * c + 4 * q;
                if (dt != BITNET_OUT_BF16 && wide && nb + n + 4 <= N) {
                    uint32_t x[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x[r] = dt == BITNET_OUT_I32
                                   ? (uint32_t)v[4 * c + r]
                                   : __float_as_uint(((float)v[4 * c + r] * sc[4 * c + r]) * inv);
                    *reinterpret_cast<uint4*>(static_cast<uint32_t*>(out) + o + n) =
                        make_uint4(x[0], x[1], x[2], x[3]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (nb + n + r < N) store_out(out, o + n + r, dt, v[4 * c + r], sc[4 * c + r], inv);
                }
            }
        }
    };
    if constexpr (G == 1) {
        // the columns of a row one behind another, so that their stores meet in a cache line (512 rows each
        // of 8 experts, 14336 x 4096, twice: 230 MB written instead of 407, 492 -> 470 us)
        float sc[NB][2][8];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) scales(i, h, sc[i][h]);
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int v[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] = acc[j][i][8 * h + r];
                    emit(j, i, h, v, sc[i][h]);
                }
    } else {
        // every group leaves its sums in LDS and adds up, over the groups, the part it writes
        constexpr int EV = MB * NB * 2;  // eighths of 16 registers
        static_assert(EV % G == 0, "parts");
        int* const sums = reinterpret_cast<int*>(smem);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sums[((g * WPG + wave) * EV * 8 + (j * NB + i) * 16 + r) * 64 + lane] = acc[j][i][r];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < EV / G; ++e) {
            const int ev = g * (EV / G) + e;  // uniform
            int v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                v[r] = 0;
#pragma unroll
                for (int k = 0; k < G; ++k) v[r] += sums[((k * WPG + wave) * EV * 8 + ev * 8 + r) * 64 + lane];
            }
            float sc[8];
            scales(ev / 2 % NB, ev & 1, sc);
            emit(ev / 2 / NB, ev / 2 % NB, ev & 1, v, sc);
        }
    }
}

// ----------------------------------------------------------------------- few rows
constexpr int kStreamWaves = 4;

// 16 rows of one expert times 64 rows of its weights and all of K.  Wave w takes the
// 256-weight chunks w, w + 4, ..; it has the weights of one chunk in flight, which come from memory,
// and the activations of two halves of a chunk, which come from a cache: with few registers for
// each, a CU holds the five blocks that hide both.  Rows of weights at any byte (K % 16 != 0): a weight
// dword is put together from the aligned ones around it when it is used (4100 columns of 8 rows each of
// another expert, 14336 twice: 42 us, in 64 x 128 tiles 73; of 4096 columns 35).
template <bool ALIGNED>
__global__ __launch_bounds__(64 * kStreamWaves, 5) void expert_stream_kernel(ExpertArgs p) {
    constexpr int NB = 4, BM = 16, BN = 16 * NB, TH = 64 * kStreamWaves;
    constexpr int MO = BM * BN / TH;  // outputs of a thread
    __shared__ int red[kStreamWaves][NB * 256];
    // column tile x of row tile y: no block shares its weights, so which XCD takes it does not matter
    Unit u;
    const ExpertTiles<BM> tiles(p.offsets, p.E, p.P);
    if ((int)blockIdx.y >= tiles.total) return;
    column_of<BN>(p, (int)blockIdx.x, u);
    tiles.find((int)blockIdx.y, u.e, u.m0, u.rows);
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.K, N = u.N, row_bytes = K / 4;
    const int nch = (K + 255) / 256;
    const int rows_b = min(BN, N - u.n0);
    const uint8_t* const wbase = pick(p.packed, u.g) + ((int64_t)u.e * N + u.n0) * row_bytes;
    const uint32_t skew = ALIGNED ? 0u : (uint32_t)((uintptr_t)wbase & 3);
    const __amdgpu_buffer_rsrc_t rb = rsrc(wbase - skew, ALIGNED ? (uint32_t)(rows_b * row_bytes)
                                                                 : (uint32_t)((rows_b * row_bytes + skew + 3) & ~3u));
    uint32_t voff_b[NB], shift[NB];  // of the dword that holds the first weight; bits in front of it
#pragma unroll
    for (int i = 0; i < NB; ++i) {  // rows behind the last one read zeros
        const uint32_t off = (uint32_t)((16 * i + l16) * row_bytes + 16 * q) + skew;
        voff_b[i] = 16 * i + l16 < rows_b ? off & ~3u : kOut;
        shift[i] = 8 * (off & 3);
    }
    u32x4 w[NB];
    uint32_t w4[ALIGNED ? 1 : NB];  // the fifth dword
    auto load_w = [&](int j) {
        const int ch = wave + kStreamWaves * j;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const uint32_t off = ch < nch && voff_b[i] != kOut ? voff_b[i] + 64 * ch : kOut;
            w[i] = load16(rb, off, 0);
            if constexpr (!ALIGNED) w4[i] = __builtin_amdgcn_raw_buffer_load_b32(rb, off + 16, 0, 0);
        }
    };
    load_w(0);
    const __amdgpu_buffer_rsrc_t ra =
        rsrc(p.xq + (p.rows ? 0 : (int64_t)u.m0 * K), (uint32_t)((p.rows ? p.T : u.rows) * K));
    const int token = token_of(p, u, l16);
    const uint32_t voff_a = token < 0 ? kOut : (uint32_t)((p.rows ? token : token - u.m0) * K + 64 * q);
    u32x4 x[2][2];
    auto load_x = [&](int j, int h) {  // half h of chunk j
        const int ch = wave + kStreamWaves * j;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = 256 * ch + 32 * h + 16 * s;
            x[h][s] = load16(ra, voff_a != kOut && k + 64 * q < K ? voff_a + k : kOut, 0);
        }
    };
    load_x(0, 0);
    load_x(0, 1);
    // scales of this thread's outputs, column tid % BN of rows tid / BN + i TH / BN
    const int n = u.n0 + tid % BN;
    const float ws = n < N ? pick(p.w_scale, u.g)[(int64_t)u.e * N + n] : 0.0f;
    float scale[MO];
#pragma unroll
    for (int i = 0; i < MO; ++i) {
        const int t = token_of(p, u, tid / BN + i * (TH / BN));
        scale[i] = t < 0 ? 1.0f : p.a_scale[t];  // a row of zeros stays zero
    }
    v4i acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = v4i{0, 0, 0, 0};
    const int nj = (nch - wave + kStreamWaves - 1) / kStreamWaves;
    for (int j = 0; j < nj; ++j) {
        if (!ALIGNED && 256 * (wave + kStreamWaves * j) + 256 > K) {
            // what lies behind the row's end
            const int left = K - 256 * (wave + kStreamWaves * j) - 64 * q;  // bytes, a multiple of 4
#pragma unroll
            for (int d = 0; d < 16; ++d)
                x[d >> 3][(d >> 2) & 1][d & 3] = left > 4 * d ? x[d >> 3][(d >> 2) & 1][d & 3] : 0u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t d[4] = {x[h][s][0], x[h][s][1], x[h][s][2], x[h][s][3]};
                uint32_t e[4];
                transpose4x4_bytes(d, e);
                const v4i a = {(int)e[0], (int)e[1], (int)e[2], (int)e[3]};
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    uint32_t b = w[i][2 * h + s];
                    if constexpr (!ALIGNED)
                        b = __builtin_amdgcn_alignbit(2 * h + s < 3 ? w[i][(2 * h + s + 1) & 3] : w4[i], b, shift[i]);
                    const v4i c = {(int)ternary_field_i8<0>(b), (int)ternary_field_i8<1>(b),
                                   (int)ternary_field_i8<2>(b), (int)ternary_field_i8<3>(b)};
                    acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(c, a, acc[i], 0, 0, 0);
                }
            }
            load_x(j + 1, h);
        }
        load_w(j + 1);
    }
    // 16x16 accumulator: lane l, register r -> weight row 4 (l / 16) + r, token l % 16
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][(16 * i + 4 * q + r) * BM + l16] = acc[i][r];
    __syncthreads();
    void* const out = pick(p.out, u.g);
#pragma unroll
    for (int i = 0; i < MO; ++i) {
        const int m = tid / BN + i * (TH / BN);
        if (m >= u.rows || n >= N) continue;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < kStreamWaves; ++v) sum += red[v][(tid % BN) * BM + m];
        store_out(out, (int64_t)(u.m0 + m) * N + n, p.out_dtype, sum, ws, 1.0f / scale[i]);
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

// Column tiles of all matrices; their number goes to tile[].
int64_t column_tiles(ExpertArgs& a, int bn) {
    int64_t tn = 0;
    for (int g = 0; g < BITNET_MAX_GROUPS; ++g) {
        a.tile[g] = (int)tn;
        if (g < a.groups) tn += (a.N[g] + bn - 1) / bn;
    }
    a.tile[BITNET_MAX_GROUPS] = (int)tn;
    return tn;
}

template <class KERNEL>
hipError_t launch_units(KERNEL kernel, ExpertArgs a, int bm, int bn, int threads, int panel,
                        hipStream_t stream) {
    const int64_t tn = column_tiles(a, bn);
    a.tiles_n = (int)tn;
    a.panel = panel;
    const int64_t units = expert_tiles(a.P, a.E, bm) * tn;
    // (at most 2^15 column tiles, of four matrices of 2^20 rows: more outputs than the card holds)
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
    // Rows of an expert and row tiles, if the rows are spread evenly; and the columns' tiles.
    const int64_t active = E < P ? E : P, per = P / active;
    int64_t cols = 0;
    for (int g = 0; g < a.groups; ++g) cols += (a.N[g] + 127) / 128;
    const int64_t units = active * ((per + 63) / 64) * cols;  // of 64 x 128
    const bool aligned = K % 16 == 0;
    // Few rows: the stream re-reads the activations for every 64 weight rows, 64 x 128 tiles keep
    // them in LDS but need two blocks on a CU to hide their steps' latency.  Two rows each of 64 experts
    // (640 x 2560, twice) 13.0 us against 16.9, eight 21.2 against 21.5, 16 29.0 against 22.4; four rows
    // each of 8 experts (4096 x 14336) 33 against 44, 16 49 against 44; with few tiles 16 rows of 4
    // (1408 x 8192, 44 tiles) 14.4 against 21.7, of 16 (768 x 2048, 96) 9.2 against 9.3.  Columns off 16 cost
    // the tiles more: 16 rows of 8 (14336 x 4100) 64 against 74, but 12 of 64 (640 x 644, twice) 14.9 against 13.3.
    const bool few = per <= 8 || (per <= 16 && (units <= 192 || (!aligned && K >= 2048)));
    const int64_t tn = few ? column_tiles(a, 64) : 0, tm = few ? expert_tiles(P, E, 16) : 0;  // at most 2048 row tiles
    if (few && tn * tm <= max_blocks(64 * kStreamWaves)) {  // (the tiles are launched in parts)
        if (aligned)
            hipLaunchKernelGGL(expert_stream_kernel<true>, dim3((unsigned)tn, (unsigned)tm), dim3(64 * kStreamWaves),
                               0, stream, a);
        else
            hipLaunchKernelGGL(expert_stream_kernel<false>, dim3((unsigned)tn, (unsigned)tm),
                               dim3(64 * kStreamWaves), 0, stream, a);
        return hipGetLastError();
    }
    // 128 x 256 where there are a hundred rows, one tile for every CU, and 32 steps or a thousand rows: 512
    // rows each of 8 experts (14336 x 4096, twice) 470 us against 631 in 64 x 128 tiles and 559 in 256 x 256 ones, of
    // which a quarter is padding and one block fills a CU; 256 rows (4096 x 14336) 167 against 182.  Fewer
    // tiles: 434 rows of 3 experts (342 x 2432, twice) 38 against 14; fewer steps: 128 rows of 64
    // (2560 x 640) 44 against 37, but 4096 rows of 4 (4096 x 1280) 115 against 135; columns off 16 (rows of 4-byte loads): 884 rows of 8 (2490 x 3592)
    // 151 against 141.
    int64_t wide = 0;
    for (int g = 0; g < a.groups; ++g) wide += (a.N[g] + 255) / 256;
    wide *= active * ((per + 127) / 128);
    if (aligned && per >= 96 && wide >= 256 && (K >= 2048 || per >= 1024))
        return launch_units(expert_tile_kernel<128, 256, 128, 64, 1, 1, 2, true>, a, 128, 256, 256, 4, stream);
    // Too few tiles for two blocks on a CU: two groups of waves share the steps of each.  32 rows each of
    // 8 experts (4096 x 14336) 71 us against 81, 21 rows of 21 (997 x 6104) 31 against 44; 64 rows of 30
    // (4320 x 684) 51 against 42.
    if (units < 512)
        return aligned ? launch_units(expert_tile_kernel<64, 128, 64, 32, 2, 1, 4, true>, a, 64, 128, 512, 2, stream)
                       : launch_units(expert_tile_kernel<64, 128, 64, 32, 2, 1, 4, false>, a, 64, 128, 512, 2, stream);
    // Columns off 16: two steps of activations in flight, three blocks on a CU (77 rows of 17, 967 x 2068,
    // twice 28.0 us against 28.9; 1708 of 18, 1071 x 1464 143 against 153; 55 of 30, 4320 x 684 41 against 43).
    return aligned ? launch_units(expert_tile_kernel<64, 128, 64, 32, 1, 1, 4, true>, a, 64, 128, 256, 2, stream)
                   : launch_units(expert_tile_kernel<64, 128, 64, 32, 1, 2, 3, false>, a, 64, 128, 256, 2, stream);
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
