// The division of attn_decode's work among its workgroups (attn_plan), run on the host with 64 lanes:
// every worker has to come to the sequence that holds its first unit, and know how many units lie before.
#include <cstdio>
#include <random>
#include <vector>

#include "../../weight_streaming_linear_amd/csrc/attn.h"

using namespace wsl;

namespace {

int fails = 0;

AttnArgs args_of(const std::vector<int32_t> &lens, int n_kv, int workers, int capacity, int q_len, int64_t window) {
    AttnArgs a = {};
    a.lens = lens.data();
    a.n_seq = static_cast<int32_t>(lens.size()), a.n_kv = n_kv, a.workers = workers, a.capacity = capacity;
    a.q_len = q_len, a.window = window;
    a.over_heads = attn_div(static_cast<uint32_t>(n_kv));
    return a;
}

AttnPlan plan_of(const AttnArgs &a, uint32_t w) {
    AttnPlan got[64];
    wave::run([&] { const AttnPlan p = attn_plan(a, w); got[wave::at] = p; });
    for (int l = 1; l < 64; ++l)
        if (got[l].seq != got[0].seq || got[l].total != got[0].total || got[l].each != got[0].each ||
            got[l].before != got[0].before || got[l].cost != got[0].cost)
            ++fails, std::printf("FAILED: lane %d of worker %u differs\n", l, w);
    return got[0];
}

void check_shares(const std::vector<int32_t> &lens, int n_kv, int workers, int capacity, int q_len, int64_t window) {
    const AttnArgs a = args_of(lens, n_kv, workers, capacity, q_len, window);
    const int step = workers > 64 ? 7 : 1;      // (not every worker of the large cases)
    for (int w = 0; w < workers; w += step) {
        const AttnPlan p = plan_of(a, static_cast<uint32_t>(w));
        int64_t total = 0, before = 0;
        int32_t seq = 0;
        bool found = false;
        const int64_t x = static_cast<int64_t>(w) * p.each;
        for (size_t b = 0; b < lens.size(); ++b) {
            const int64_t units = attn_span(a, lens[b]).tiles + p.cost;
            if (!found && x < total + units * n_kv) found = true, seq = static_cast<int32_t>(b), before = total / n_kv;
            total += units * n_kv;
        }
        const bool ok = p.total == total && p.each >= 1 && static_cast<int64_t>(p.each) * workers >= total &&
                        (!found || (p.seq == seq && p.before == before));
        if (!ok)
            ++fails, std::printf("FAILED: worker %d of %d, %zu sequences, %d heads: sequence %d, %d units before of %d; "
                                 "expected %d, %lld of %lld\n", w, workers, lens.size(), n_kv, p.seq, p.before, p.total,
                                 seq, static_cast<long long>(before), static_cast<long long>(total));
    }
}

}  // namespace

int main() {
    std::mt19937 rng(5);
    int cases = 0;
    for (const int n : {1, 2, 5, 63, 64, 65, 200, 4100})
        for (const int n_kv : {1, 3, 8})
            for (const int workers : {8, 40, 256})
                for (const int64_t window : {int64_t(0), int64_t(300)}) {
                    std::vector<int32_t> lens(static_cast<size_t>(n));
                    for (auto &x : lens) {
                        x = static_cast<int32_t>(rng() % (n < 100 ? 6000 : 900));
                        if (rng() % 5 == 0) x = static_cast<int32_t>(rng() % 3) - 1;     // empty, one, out of range
                    }
                    check_shares(lens, n_kv, workers, 5000, 5, window);
                    ++cases;
                }
    // the lowest position that is seen, for windows up to the largest number there is
    for (const int64_t window : {int64_t(1), int64_t(5), int64_t(1) << 31, int64_t(1) << 40, INT64_MAX - 300, INT64_MAX - 1, INT64_MAX})
        for (int32_t len = 0; len < 600; ++len)
            for (const int q_len : {1, 2, 5, 256}) {
                AttnArgs a = args_of({}, 1, 8, 5000, q_len, attn_window(window, 5000));
                int32_t want = 0;       // the first row that stands at a token at all is at 0 or at len - q_len
                const int32_t at = len > q_len ? len - q_len : 0;
                if (window <= at) want = at - static_cast<int32_t>(window) + 1;
                if (attn_lowest(a, len) != want)
                    ++fails, std::printf("FAILED: lowest of %d with %d queries, window %lld: %d\n", len, q_len,
                                         static_cast<long long>(window), attn_lowest(a, len));
            }
    // whole items: nothing is shared out, but what a worker is told is still defined
    for (const int n : {1, 7, 300})
        for (const int n_kv : {1, 8}) {
            const std::vector<int32_t> lens(static_cast<size_t>(n), 200);
            AttnArgs a = args_of(lens, n_kv, n * n_kv, 512, 1, 0);
            a.whole = 1;
            for (int w = 0; w < n * n_kv; ++w) {
                const AttnPlan p = plan_of(a, static_cast<uint32_t>(w));
                if (p.seq != w / n_kv || p.cost != 0 || p.before != 0 || p.each != 1 || p.total != n * n_kv)
                    ++fails, std::printf("FAILED: whole item %d: sequence %d, each %d of %d\n", w, p.seq, p.each, p.total);
            }
            ++cases;
        }
    std::printf("%s: %d cases\n", fails ? "FAILED" : "ok", cases);
    return fails ? 1 : 0;
}
