// The argument checks of the pages, rotary, sampling and adapter entry points over extreme numbers:
// every combination has to come back (no overflow, no fault), and the plain ones pass.
#include <cstdio>

#include "../../include/wsl.h"
#include "../../weight_streaming_linear_amd/csrc/validate.h"

int main() {
    const int64_t big[] = {INT64_MIN, -1, 0, 1, 8, 16, 64, 128, 4096, int64_t(1) << 22, int64_t(1) << 30,
                           int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, INT64_MAX};
    alignas(16) static char mem[64];
    int fails = 0, seen = 0, fine = 0;
    int32_t *w = reinterpret_cast<int32_t *>(mem);
    const wsl_kv_pages p = {w, w, w, w, 4, 8, 8, 32, 16};
    if (wsl::check_kv_pages(&p) != WSL_OK || wsl::check_trim(&p, mem) != WSL_OK) ++fails;
    if (wsl::check_grow(&p, nullptr, 3, 12, mem, mem, mem) != WSL_OK) ++fails;
    if (wsl::check_rotary(mem, 8, 1024, mem, 2, 1024, 0, 3, 128, 64, mem, mem, 1.0, 1, mem, 1024, mem, 256, 1) != WSL_OK) ++fails;
    if (wsl::check_sample(mem, 1, 3, 100, 101, nullptr, mem, mem, mem, 100) != WSL_OK) ++fails;
    if (wsl::check_lora(mem, mem, 3, 16, 100, 64, mem, nullptr, mem, 5, 64, mem, 100, mem, 101, 0) != WSL_OK) ++fails;
    for (int64_t a : big)
        for (int64_t b : big)
            for (int64_t c : big) {
                for (int field = 0; field < 5; ++field) {
                    wsl_kv_pages d = p;
                    int64_t *f[] = {&d.n_seq, &d.pages_per_seq, &d.ld_table, &d.n_pages, &d.page_size};
                    *f[field] = a;
                    *f[(field + 2) % 5] = b;
                    fine += wsl::check_grow(&d, nullptr, c, b, mem, nullptr, nullptr) == WSL_OK;
                    fine += wsl::check_trim(&d, mem) == WSL_OK;
                }
                fine += wsl::check_rotary(mem, a, b, mem, c, a, 0, b, 128, 64, mem, mem, 1.0, 0, mem, b, mem, c, 1) == WSL_OK;
                fine += wsl::check_rotary(mem, 8, 1024, nullptr, a, b, 1, 3, b, c, mem, mem, 1.0, 0, mem, 1024, nullptr, 0, 1) == WSL_OK;
                fine += wsl::check_rotary(mem, a, b, mem, a, b, 1, c, 256, 2, mem, mem, 1.0, 0, mem, b, mem, b, 1) == WSL_OK;
                fine += wsl::check_sample(mem, 0, a, b, c, nullptr, mem, mem, mem, c) == WSL_OK;
                fine += wsl::check_lora(mem, mem, a, b, c, 64, mem, mem, mem, a, b, mem, c, mem, c, 0) == WSL_OK;
                fine += wsl::check_lora(mem, mem, 3, 16, a, b, mem, mem, mem, c, b, mem, a, mem, a, 1) == WSL_OK;
                fine += wsl::lora_shape_ok(a, b, c);
                ++seen;
            }
    std::printf("%s: %d combinations, %d accepted\n", fails ? "FAILED" : "ok", seen, fine);
    return fails ? 1 : 0;
}
