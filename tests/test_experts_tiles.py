"""How the blocks of a product grouped by expert count their tiles, on the CPU: the lanes' part of it
compiled for the host."""
import os
import subprocess

import numpy as np
import pytest

from ternary_weight_linear_token_amd import build as bw_build

# the lanes' sums and the bound of their total for tiles of 64 and of 128 rows
PROGRAM = r"""
#include <cstdio>
#include "experts.hpp"
using namespace bitnet;
template <int BM> void count(const int* offsets, int E, int P) {
    const int per = (E + 63) / 64;
    for (int lane = 0; lane < 64; ++lane) {
        ExpertRows last = {0, 0};
        std::printf("%d ", lane_tiles<BM>(offsets, E, P, per, lane, last));
    }
    std::printf("%d\n", expert_tiles(P, E, BM));
}
int main() {
    int P, E;
    while (std::scanf("%d %d", &P, &E) == 2) {
        int offsets[BITNET_MAX_EXPERTS + 1];
        for (int e = 0; e <= E; ++e)
            if (std::scanf("%d", &offsets[e]) != 1) return 1;
        count<64>(offsets, E, P);
        count<128>(offsets, E, P);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def lanes(tmp_path_factory):
    if not os.path.exists(bw_build.HIPCC):
        pytest.skip("hipcc is not installed")
    d = tmp_path_factory.mktemp("tiles")
    src, exe = str(d / "tiles.hip"), str(d / "tiles")
    with open(src, "w") as f:
        f.write('#include "bitnet_w2a8.h"\n' + PROGRAM)
    subprocess.run([bw_build.HIPCC] + bw_build.FLAGS + ["--offload-host-only", src, "-o", exe], check=True,
                   capture_output=True)

    def run(P, offsets):
        text = f"{P} {len(offsets) - 1} " + " ".join(map(str, offsets))
        out = subprocess.run([exe], input=text, text=True, check=True, capture_output=True).stdout
        rows = [list(map(int, line.split())) for line in out.splitlines()]
        return {bm: (r[:64], r[64]) for bm, r in zip((64, 128), rows)}
    return run


@pytest.mark.parametrize("P,E", [(1, 1), (63, 5), (64, 64), (1000, 65), (5000, 1024), (1 << 30, 3), (1 << 30, 1024)])
def test_tiles_of_sorted_rows(lanes, P, E):
    rng = np.random.RandomState(P % 1000 + E)
    for kind in ("even", "skewed", "one"):
        p = {"even": np.ones(E) / E, "skewed": rng.dirichlet(np.full(E, 0.3)), "one": np.eye(E)[E // 2]}[kind]
        counts = rng.multinomial(P, p).astype(np.int64)
        offsets = np.concatenate([[0], np.cumsum(counts)])
        for bm, (sums, most) in lanes(P, offsets).items():
            per = (E + 63) // 64
            want = np.zeros(64 * per, dtype=np.int64)
            want[:E] = (counts + bm - 1) // bm
            assert sums == want.reshape(64, per).sum(1).tolist(), (kind, bm)
            assert sum(sums) <= most == (P + min(E, P) * (bm - 1)) // bm


@pytest.mark.parametrize("P", [40, 1 << 20, (1 << 28) + 5, 1 << 30])
@pytest.mark.parametrize("E", [5, 64, 1000, 1024])
def test_tiles_of_offsets_that_make_no_sense(lanes, P, E):
    # up and down, beyond the rows, at random: the sum over the lanes stays within 31 bits, and a lane
    # counts no more than its experts have
    rng = np.random.RandomState(E)
    far = 2 ** 31 - 1
    for offsets in ([0, P] * (E // 2 + 1), [-far - 1, far] * (E // 2 + 1), [far] * (E + 1),
                    rng.randint(-far, far, E + 1).tolist()):
        offsets = offsets[:E + 1]
        cut = np.clip(np.array(offsets, dtype=np.int64), 0, P)
        counts = np.maximum(cut[1:] - cut[:-1], 0)
        for bm, (sums, _) in lanes(P, offsets).items():
            per = (E + 63) // 64
            have = np.zeros(64 * per, dtype=np.int64)
            have[:E] = (counts + bm - 1) // bm
            assert sum(sums) < 2 ** 31
            assert all(0 <= s <= h for s, h in zip(sums, have.reshape(64, per).sum(1)))
