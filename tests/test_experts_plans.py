"""Which gradient kernel a product grouped by expert takes, on the CPU: the rule of grad.hip, compiled
for the host with launches that report their tile, and the sizes that the GPU tests run."""
import os
import re
import subprocess

import pytest

from ternary_weight_linear_token_amd import build as bw_build
from test_gpu_experts import GRADS, test_large_gradients as large
from test_gpu_experts_limits import SEVERAL, test_weight_gradient_against_the_codes_values as operands

LARGE_GRADS = next(m.args[1] for m in large.pytestmark if m.args[:1] == ("P,E,N,K",))

STUBS = r"""
#include <cstdint>
#include <cstdio>
#include "bitnet_w2a8.h"
typedef int hipError_t;
typedef void* hipStream_t;
enum Rows { kWhole, kOdd, kOddEnd };
struct GradArgs {
    const uint16_t* dy[BITNET_MAX_GROUPS];
    const uint8_t* b[BITNET_MAX_GROUPS];
    const float* scale[BITNET_MAX_GROUPS];
    int L[BITNET_MAX_GROUPS], groups, I, J, out_dtype;
    void* out;
    const int* offsets;
    int E, P;
};
template <int C, Rows R> int launch_experts(GradArgs, hipStream_t) { return 10 * C + R; }
"""
MAIN = r"""
int main() {
    long long weight, P, E, K, groups, n;
    while (std::scanf("%lld %lld %lld %lld %lld", &weight, &P, &E, &K, &groups) == 5) {
        int64_t N[BITNET_MAX_GROUPS];
        const uint16_t* dy[BITNET_MAX_GROUPS] = {};
        const uint8_t* packed[BITNET_MAX_GROUPS] = {};
        const float* scale[BITNET_MAX_GROUPS] = {};
        for (int g = 0; g < groups; ++g) {
            if (std::scanf("%lld", &n) != 1) return 1;
            N[g] = n;
        }
        // weight: 0, or 1 for fp32 and 2 for bf16
        std::printf("%d\n", weight ? launch_grad_weight_experts(nullptr, nullptr, nullptr, nullptr, P, E, N[0], K, nullptr,
                                         weight == 1 ? BITNET_OUT_F32 : BITNET_OUT_BF16, nullptr)
                                   : launch_grad_input_experts(dy, nullptr, P, E, packed, scale, N, (int)groups, K,
                                                               nullptr, nullptr));
    }
    return 0;
}
"""


def source():
    with open(os.path.join(bw_build.CSRC, "grad.hip")) as f:
        return f.read()


@pytest.fixture(scope="module")
def taken(tmp_path_factory):
    """(table entry, kind of rows) of a call: taken(weight, P, E, K, Ns)."""
    text = source()
    cus = re.search(r"^constexpr \w+ kCUs = \d+;", text, re.M).group(0)
    rules = [re.search(r"^hipError_t launch_grad_%s_experts\(.*?^}" % kind, text, re.M | re.S).group(0)
             for kind in ("input", "weight")]
    d = tmp_path_factory.mktemp("plans")
    src, exe = str(d / "plans.cpp"), str(d / "plans")
    with open(src, "w") as f:
        f.write("\n".join([STUBS, cus] + rules + [MAIN]))
    subprocess.run(["g++", "-std=c++17", "-I", bw_build.INCLUDE, src, "-o", exe],
                   check=True, capture_output=True)

    def run(weight, P, E, K, Ns):
        line = " ".join(map(str, [weight, P, E, K, len(Ns)] + list(Ns)))
        out = int(subprocess.run([exe], input=line, text=True, check=True, capture_output=True).stdout)
        return out // 10, ("whole", "odd", "odd end")[out % 10]
    return run


def compiled():
    """Every (entry, kind of rows) that a rule of the experts' gradients launches, and the entries'
    modes and steps."""
    text = source()
    lines = text[text.index("constexpr GradCfg kExpertCfg[] = {"):].split("};")[0]
    rows = re.findall(r"^    \{(\d), \d+, \d+, \d+, \d+, \d, (\d+),", lines, re.M)
    assert len(rows) == lines.count("    {")
    calls = set(re.findall(r"launch_experts<(\d+), k(\w+)>", text))
    names = {"Whole": "whole", "Odd": "odd", "OddEnd": "odd end"}
    return {(int(c), names[r]) for c, r in calls}, [(m == "0", int(bl)) for m, bl in rows]


def test_gpu_sizes_reach_every_kernel(taken):
    want, cfgs = compiled()
    assert {c for c, _ in want} == set(range(len(cfgs)))
    one = {taken(0, P, E, K, [N]) for P, E, N, K in GRADS + LARGE_GRADS}
    one |= {taken(w, P, E, K, [N]) for P, E, N, K in GRADS + LARGE_GRADS for w in (1, 2)}
    assert one == want


def test_gpu_sizes_check_the_weight_gradients_operands_in_every_kernel(taken):
    want, cfgs = compiled()
    sizes = next(m.args[1] for m in operands.pytestmark if m.args[:1] == ("P,E,N,K",))
    for w in (1, 2):
        assert {taken(w, P, E, K, [N]) for P, E, N, K in sizes} == {(c, r) for c, r in want if cfgs[c][0]}


def test_gpu_sizes_cross_between_stacks_in_every_kernel(taken):
    # sums of several steps over each of two stacks at least
    want, cfgs = compiled()
    seen = set()
    for P, E, Ns, K in SEVERAL:
        entry, rows = taken(0, P, E, K, Ns)
        assert sum(n > cfgs[entry][1] for n in Ns) >= 2
        seen.add((entry, rows))
    assert seen == {(c, r) for c, r in want if not cfgs[c][0]}
