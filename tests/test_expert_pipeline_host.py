"""The stages of the expert products' inputs (not gpu): whatever the order in which loads
arrive and warps go on, a warp multiplies the inputs of its own step.

The kernels' own header says how many stages and barriers each form has and which step uses
which; the protocol around them (arm a barrier, copy, wait for a parity, count, ask for the next
inputs) is played through in random orders, some warps and some loads far behind the others."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exl3_trellis_weight_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "expert_form.cuh"
using namespace exl3;

static int forms = 0;

template <class F> const char *play(int n, unsigned seed) {
    constexpr int G = F::kGroups, S = F::kStages, L = F::kArrivals, W = kExpertWarps / G;
    std::mt19937 rng(seed);
    auto some = [&](int m) { return (int)(rng() % (unsigned)m); };
    struct Load {
        int step, weight;
    };
    struct Warp {
        int step, weight;
        bool reads;
    };
    std::vector<Load> way;                         // armed and not yet arrived
    std::vector<int> phase(L, 0), armed(L, 0), holds(S, -1), used(S, 0);
    std::vector<Warp> warps(kExpertWarps);
    // what is far behind: a warp, a step's load
    auto pace = [&] { return some(8) == 0 ? 1 : 1 + some(300); };
    for (int w = 0; w < kExpertWarps; w++)
        warps[w] = {w / W, pace(), false};
    const char *wrong = nullptr;
    auto issue = [&](int i) {
        if (armed[F::arrival(i)]++)
            wrong = "a barrier armed twice in a phase";
        holds[F::stage(i)] = -1;                   // being written
        way.push_back({i, pace()});
    };
    for (int i = 0; i < S && i < n; i++)
        issue(i);
    auto passes = [&](const Warp &w) { return (unsigned)(phase[F::arrival(w.step)] & 1) != F::parity(w.step); };
    for (;;) {
        // one of what can happen now
        long all = 0;
        for (auto &l : way)
            all += l.weight;
        bool left = false;
        for (auto &w : warps)
            if (w.step < n) {
                left = true;
                if (w.reads || passes(w))
                    all += w.weight;
            }
        if (!left)
            return way.empty() ? nullptr : "a load that nobody waited for";
        if (all == 0)
            return "nobody goes on";
        long pick = (long)(((unsigned long)rng() << 16 ^ rng()) % (unsigned long)all);
        bool done = false;
        for (size_t k = 0; k < way.size() && !done; k++)
            if ((pick -= way[k].weight) < 0) {
                const int i = way[k].step;
                way.erase(way.begin() + k);
                holds[F::stage(i)] = i;
                phase[F::arrival(i)]++;
                armed[F::arrival(i)]--;
                done = true;
            }
        for (int k = 0; k < kExpertWarps && !done; k++) {
            Warp &w = warps[k];
            if (w.step >= n || !(w.reads || passes(w)) || (pick -= w.weight) >= 0)
                continue;
            done = true;
            const int i = w.step, s = F::stage(i);
            if (holds[s] != i)
                return w.reads ? "inputs replaced under a reader" : "inputs of another step";
            if (!w.reads) {
                w.reads = true;
                continue;
            }
            w.reads = false;
            w.step += G;
            w.weight = pace();
            if (i + S < n && ++used[s] == W) {
                used[s] = 0;
                issue(i + S);
            }
        }
        if (wrong)
            return wrong;
    }
}

template <int K, int RB, bool LO, bool TWO> int form() {
    using F = ExpertForm<K, RB, LO, TWO>;
    forms++;
    for (unsigned seed = 0; seed < 60; seed++)
        if (const char *e = play<F>(1 + (int)(seed * 7 % (5 * F::kStages + 3)), seed)) {
            std::printf("K %d, %d rows, parts %d, matrices %d: %d stages, %d barriers, %d groups, order %u: %s\n", K, F::kRows, LO ? 2 : 1,
                        F::kMatrices, F::kStages, F::kArrivals, F::kGroups, seed, e);
            return 1;
        }
    return 0;
}
template <int K> int forms_of() {
    return form<K, 1, false, false>() + form<K, 2, false, false>() + form<K, 4, false, false>() + form<K, 1, true, false>() + form<K, 2, true, false>() +
           form<K, 1, false, true>() + form<K, 2, false, true>() + form<K, 4, false, true>() + form<K, 1, true, true>() + form<K, 2, true, true>();
}

int main() {
    const int failed = forms_of<1>() + forms_of<2>() + forms_of<3>() + forms_of<4>();
    std::printf("%d forms, %d failed\n", forms, failed);
    return failed ? 1 : 0;
}
"""


def test_every_warp_has_the_inputs_of_its_step(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "steps.cpp", tmp_path / "steps"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-O1", "-I", CSRC, "-x", "c++", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("40 forms")


def test_the_order_of_inputs_stands_in_one_place():
    """Which of 16 inputs a lane takes goes by K and the transposition: whoever stores inputs for the
    fragments asks the same function."""
    rule, places = re.compile(r"K\s*==\s*3\s*\?\s*0\s*:\s*(?:\w+\.)?K\s*==\s*1\s*\?\s*2\s*:\s*1"), []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            places += [name] * len(rule.findall(f.read()))
    assert places == ["linear.cuh"]
