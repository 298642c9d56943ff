// experts.hpp -- how the blocks of a product grouped by expert find their rows: shared by the
// forward product (experts.hip) and the gradients (grad.hip).
//
// The rows of a call are sorted by expert and offsets[e] .. offsets[e + 1] are those of expert e; the
// offsets lie in device memory, so the host knows neither the counts nor the number of tiles.
// It launches as many blocks as any counts could need (min(E, P) experts may each end in a
// partial tile), and every wave of a block counts the tiles itself: lane l takes the experts
// per * l .., a scan over the wave gives the tiles before each, and a ballot the expert of a tile.
#pragma once

#include "device_common.hpp"

namespace bitnet {

// Most tiles of `bm` rows that P rows of E experts can make (P up to 2^30, so 31 bits hold the sum).
template <class T>
__host__ __device__ __forceinline__ T expert_tiles(T P, T E, int bm) {
    const T e = E < P ? E : P;
    return (P + e * (bm - 1)) / bm;
}

// Inclusive sum over the wave (every lane active).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31
    return v;
}

// Rows of expert e, whatever the offsets hold: inside 0 .. P, none where they run backwards.
struct ExpertRows {
    int first, count;
};
__host__ __device__ __forceinline__ ExpertRows expert_rows(const int* offsets, int e, int P) {
    auto inside = [P](int v) { return v < 0 ? 0 : (v < P ? v : P); };
    const int a = inside(offsets[e]), b = inside(offsets[e + 1]);
    return {a, b > a ? b - a : 0};
}

// Tiles of BM rows of the experts per * lane .. of one lane; `last`: the rows of the last of them.
// Offsets that go up and down may give every second expert all P rows.  The bound, which sorted rows
// do not pass, keeps the sum over the 64 lanes within 31 bits even then (tiles of fewer than 64 rows are
// taken for few rows only).
template <int BM>
__host__ __device__ __forceinline__ int lane_tiles(const int* offsets, int E, int P, int per, int lane,
                                                   ExpertRows& last) {
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e < E) {
            last = expert_rows(offsets, e, P);
            sum += (last.count + BM - 1) / BM;
        }
    }
    const int bound = P / BM + per;
    return sum < bound ? sum : bound;
}

// The tiles of BM rows of all experts, in the experts' order.
template <int BM>
struct ExpertTiles {
    const int* offsets;
    int E, P, per, sum, scan;
    ExpertRows mine;  // of the lane's expert, with one expert a lane
    int total;        // uniform

    __device__ __forceinline__ ExpertTiles(const int* off, int experts, int rows)
        : offsets(off), E(experts), P(rows), per((experts + 63) >> 6), sum(0), mine{0, 0} {
        const int lane = threadIdx.x & 63;
        sum = per == 1 ? lane_tiles<BM>(offsets, E, P, 1, lane, mine)
                       : lane_tiles<BM>(offsets, E, P, per, lane, mine);
        scan = wave_scan(sum);
        // no more than the host counted on
        total = min(__builtin_amdgcn_readlane(scan, 63), expert_tiles(P, E, BM));
    }

    // Expert, first row and number of rows (at most BM) of tile t < total; all uniform.
    __device__ __forceinline__ void find(int t, int& e, int& first, int& rows) const {
        const uint64_t past = __ballot(scan > t);
        const int l = (int)__builtin_ctzll(past);
        int left = t - (__builtin_amdgcn_readlane(scan, l) - __builtin_amdgcn_readlane(sum, l));
        ExpertRows r = {__builtin_amdgcn_readlane(mine.first, l), __builtin_amdgcn_readlane(mine.count, l)};
        e = l * per;
        if (per > 1) {
            for (;; ++e) {
                r = expert_rows(offsets, e, P);
                const int n = (r.count + BM - 1) / BM;
                if (left < n || e == E - 1) break;
                left -= n;
            }
        }
        // the same in every lane, and here in scalar registers
        e = __builtin_amdgcn_readfirstlane(e);
        first = __builtin_amdgcn_readfirstlane(r.first + left * BM);
        rows = __builtin_amdgcn_readfirstlane(min(BM, r.count - left * BM));
    }
};

}  // namespace bitnet
