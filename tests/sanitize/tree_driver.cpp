// tree_driver.cpp -- drives the C ABI's host-side validation of tree
// speculative decoding (kda_tree_api.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer: every integer argument of every call, two at a
// time, over extreme values.  The size arithmetic must neither overflow a
// signed type nor read out of bounds, and no status but the documented ones
// may come back.  Pointers are fake device addresses; a call that passes
// validation reaches a launcher here, which checks that the launch's grid is
// one that can be launched and reports failure (KDA_ERR_DEVICE).  Exit status
// 0 when every check passes.  Test infrastructure only.
#include <stdint.h>
#include <stdio.h>

#include <climits>
#include <functional>
#include <vector>

#include "../../gated_delta_rule_27_amd/csrc/kda_tree.h"
#include "kda.h"

namespace {

int failures = 0, launches = 0;

void* P(int i, uintptr_t off = 0) {
    return reinterpret_cast<void*>((uintptr_t(1) << 40) + uintptr_t(i) * (uintptr_t(1) << 56) / 32 + off);
}
float* F(int i) { return static_cast<float*>(P(i)); }
int32_t* I(int i) { return static_cast<int32_t*>(P(i)); }

// a launch of this many workgroups
hipError_t grid(const char* what, int64_t wgs, int64_t threads) {
    ++launches;
    if (wgs < 1 || wgs > INT32_MAX || wgs * threads >= (int64_t(1) << 32)) {
        fprintf(stderr, "FAIL: %s would launch %lld workgroups of %lld\n", what, (long long)wgs, (long long)threads);
        ++failures;
    }
    return hipErrorInvalidValue;
}

}  // namespace

namespace kda {
hipError_t launch_tree_prologue(const TreePrologueArgs& a, int, hipStream_t) {
    const int64_t per = tree_prologue_sequences(a.B, a.H);
    return grid("prologue", tree_prologue_tasks(a.H) * ((a.B + per - 1) / per), 256);
}
hipError_t launch_tree_decode(const TreeDecodeArgs& a, int, hipStream_t) {
    return grid("decode", (int64_t)a.B * a.H, 256);
}
hipError_t launch_tree_accept(const TreeAcceptArgs& a, int, hipStream_t) { return grid("accept", a.B, 1024); }
hipError_t launch_tree_commit(const TreeCommitArgs& a, int, hipStream_t) {
    return grid("commit", (int64_t)a.B * a.H * 2, 256);   // (the history's are at most as many)
}
}  // namespace kda

namespace {

typedef std::vector<int32_t> Ints;

struct Call {
    const char* name;
    Ints base;
    std::function<int(const Ints&)> run;
};

void expect(const char* what, int got, int want) {
    if (got != want) {
        fprintf(stderr, "FAIL: %s returned %d, expected %d\n", what, got, want);
        ++failures;
    }
}

}  // namespace

int main() {
    const kda_dtype dt = KDA_BF16;
    const std::vector<Call> calls = {
        {"prologue", {4, 8, 2, 128},
         [&](const Ints& x) {
             return kda_tree_prologue(P(0), P(1), P(2), P(3), P(4), F(5), F(6), I(7), I(8), x[0], x[1], x[2], x[3],
                                      dt, P(9), 1e-6f, P(10), P(11), P(12), P(13), P(14), nullptr);
         }},
        {"decode", {4, 8, 2, 128, 128},
         [&](const Ints& x) {
             return kda_tree_decode(P(0), P(1), P(2), P(3), P(4), F(5), I(6), I(7), x[0], x[1], x[2], x[3], x[4], dt,
                                    P(8), nullptr);
         }},
        {"accept", {4, 8, 1000},
         [&](const Ints& x) {
             return kda_tree_accept(P(0), P(1), I(2), I(3), I(4), F(5), x[0], x[1], x[2], dt, I(6), I(7), I(8),
                                    nullptr);
         }},
        {"commit", {4, 8, 6, 2, 128, 128},
         [&](const Ints& x) {
             return kda_tree_commit(P(0), P(1), P(2), P(3), F(4), I(5), I(6), x[0], x[1], x[2], x[3], x[4], x[5], dt,
                                    P(7), P(8), P(9), P(10), nullptr);
         }},
    };
    const int32_t extreme[] = {INT32_MIN, -1, 0, 1, 2, 63, 64, 65, 127, 128, 129, 1 << 16, (1 << 16) + 1, 1 << 22,
                               (1 << 22) - 1, (1 << 22) + 1, 1 << 23, (1 << 23) - 1, 1 << 24, (1 << 24) + 1,
                               1 << 30, INT32_MAX - 1, INT32_MAX};
    for (const Call& c : calls) {
        expect(c.name, c.run(c.base), KDA_ERR_DEVICE);
        for (size_t i = 0; i < c.base.size(); ++i)
            for (size_t j = i; j < c.base.size(); ++j)
                for (int32_t x : extreme)
                    for (int32_t y : extreme) {
                        Ints a = c.base;
                        a[i] = x;
                        a[j] = y;
                        const int got = c.run(a);
                        if (got < KDA_OK || got > KDA_ERR_DEVICE) {
                            fprintf(stderr, "FAIL: %s: status %d\n", c.name, got);
                            ++failures;
                        }
                    }
    }
    if (failures) return 1;
    printf("all checks passed (%d launches)\n", launches);
    return 0;
}
