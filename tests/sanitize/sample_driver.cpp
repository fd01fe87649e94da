// sample_driver.cpp -- drives the C ABI's host-side validation of
// sampling (kda_sample_api.cpp) under AddressSanitizer and
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

#include "../../gated_delta_rule_27_amd/csrc/kda_sample.h"
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
hipError_t launch_sample(const SampleArgs& a, int, hipStream_t) {
    grid("rows", a.R, 1024);
    return grid("tiles", sample_groups(a.R, a.V), 256);
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
        {"sample", {4, 1000},
         [&](const Ints& x) {
             const size_t n = kda_sample_workspace_size(x[0], x[1]);
             return kda_sample(P(0), F(1), F(2), I(3), F(4), F(5), x[0], x[1], dt, I(6), P(7), P(8), n, nullptr);
         }},
        {"sample, probabilities alone", {4, 1000},
         [&](const Ints& x) {
             const size_t n = kda_sample_workspace_size(x[0], x[1]);
             return kda_sample(P(0), nullptr, F(2), I(3), F(4), F(5), x[0], x[1], KDA_F32, nullptr, P(7), P(8), n,
                               nullptr);
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
