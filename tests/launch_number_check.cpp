// launch_number_check.cpp -- the launch numbers that chained-carry words are
// tagged with (scratch_state.hpp), run on the host.  Exits 0 if, between two
// clears of all that a call reads, no number comes twice and none reaches the
// bit that the tags add.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "scratch_state.hpp"

using namespace libscan;

#define CHECK(x)                                              \
    do {                                                      \
        if (!(x)) {                                           \
            std::printf("line %d: %s\n", __LINE__, #x);       \
            std::exit(1);                                     \
        }                                                     \
    } while (0)

int main()
{
    StateTable table;
    const uintptr_t key = 4096;
    uint64_t n = 0, before = 0;
    // An unknown buffer is cleared, and its numbers start anew.
    ClearPlan p = table.prepare(key, kKindDesc, 0, 1000, 1, false, &n);
    CHECK(p.header && p.bytes == 1000 && n == 1);
    std::set<uint64_t> seen = {n};
    // Calls of several launches count each; other kinds leave nothing valid.
    const struct { int kind; uint64_t sig, launches; } calls[] = {
        {kKindDesc, 0, 1}, {kKindDesc, 0, 3}, {kKindData, 0, 0}, {kKindDesc, 0, 1}, {kKindRadix, 12, 8},
        {kKindDesc, 0, 1}, {kKindDesc, 0, 2}, {kKindDesc, 0, 1}};
    for (int round = 0; round < 3; ++round) {
        for (const auto &c : calls) {
            p = table.prepare(key, c.kind, c.sig, 1000, c.launches, false, &n);
            if (c.kind != kKindDesc)
                continue;
            if (p.header)
                seen.clear();
            for (uint64_t i = 0; i < c.launches; ++i)
                CHECK(seen.insert(n - i).second);
            CHECK(n < kMaxLaunchesBetweenClears);
        }
    }
    // Recorded once, a buffer is cleared by every call, recorded or not.
    for (bool capturing : {true, false, true, false}) {
        p = table.prepare(key, kKindDesc, 0, 1000, 1, capturing, &n);
        CHECK(p.header && p.bytes == 1000 && n == 1);
    }
    // The numbers end below the bit: the state is cleared and they start anew.
    const uintptr_t other = 8192;
    table.prepare(other, kKindDesc, 0, 64, kMaxLaunchesBetweenClears - 3, false, &before);
    p = table.prepare(other, kKindDesc, 0, 64, 1, false, &n);
    CHECK(!p.header && n == before + 1 && n < kMaxLaunchesBetweenClears);
    table.prepare(other, kKindDesc, 0, 64, 1, false, &before);
    p = table.prepare(other, kKindDesc, 0, 64, 1, false, &n);
    CHECK(before < kMaxLaunchesBetweenClears && n < kMaxLaunchesBetweenClears);
    std::printf("ok\n");
    return 0;
}
