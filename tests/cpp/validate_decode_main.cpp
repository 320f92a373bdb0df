// The argument checks of the cache, attention and verification entry points over extreme
// numbers: every combination has to come back (no overflow, no fault), and the plain ones pass.
#include <cstdio>

#include "../../include/wsl.h"
#include "../../weight_streaming_linear_amd/csrc/validate.h"

int main() {
    const int64_t big[] = {INT64_MIN, -1, 0, 1, 16, 64, 127, 128, 256, 4096, int64_t(1) << 26, int64_t(1) << 30,
                           int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, INT64_MAX};
    alignas(16) static char mem[64];
    int fails = 0, seen = 0, fine = 0;
    wsl_kv_cache c = {mem, mem, nullptr, nullptr, WSL_KV_BF16, 4, 2, 16, 64, 2048, 1024, 64};
    if (wsl::check_kv_cache(&c) != WSL_OK) ++fails;
    for (int field = 0; field < 7; ++field)
        for (int64_t a : big)
            for (int64_t b : big) {
                wsl_kv_cache d = c;
                int64_t *f[] = {&d.n_pages, &d.n_kv, &d.page_size, &d.head_dim, &d.page_stride, &d.head_stride,
                                &d.token_stride};
                *f[field] = a;
                *f[(field + 3) % 7] = b;
                fine += wsl::check_kv_cache(&d) == WSL_OK;
                fine += wsl::check_kv_rows(&d, mem, mem, WSL_OUT_F32, a, b, 4096, mem) == WSL_OK;
                fine += wsl::check_attn(&d, mem, WSL_OUT_BF16, a, 1, 8, b, mem, a, b, mem, 1.f, b, mem, 0, a, nullptr) == WSL_OK;
                ++seen;
            }
    for (int64_t a : big)
        for (int64_t b : big)
            for (int64_t e : big) {
                fine += wsl::check_attn_shape(WSL_OUT_F32, a, b, e, 8, 128, a, b) == WSL_OK;
                fine += wsl::check_verify(mem, mem, WSL_OUT_BF16, a, b, e, e, a, mem, nullptr, mem, mem, mem) == WSL_OK;
                ++seen;
            }
    if (wsl::check_kv_rows(&c, mem, mem, WSL_OUT_F32, 3, 128, 128, mem) != WSL_OK) ++fails;
    if (wsl::check_attn(&c, mem, WSL_OUT_BF16, 2, 4, 8, 512, mem, 8, 8, mem, 1.f, 0, mem, WSL_OUT_F32, 512, mem) != WSL_OK) ++fails;
    if (wsl::check_verify(mem, nullptr, WSL_OUT_F32, 2, 4, 100, 101, 0, mem, mem, mem, mem, mem) != WSL_OK) ++fails;
    if (wsl::check_workspace(nullptr, 0, 0, 16) != WSL_OK || wsl::check_workspace(mem, 64, 65, 16) != WSL_E_RANGE) ++fails;
    std::printf("%s: %d combinations, %d accepted\n", fails ? "FAILED" : "ok", seen, fine);
    return fails ? 1 : 0;
}
