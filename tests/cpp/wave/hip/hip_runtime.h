// Enough of the device language for a host compiler to run integer wave code: 64 lanes take turns as
// contexts of one thread, and wait for each other wherever lanes exchange something.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <ucontext.h>

#define __device__
#define __host__
#define __forceinline__ inline

struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
struct double2 { double x, y; };
struct uint2 { unsigned x, y; };
struct uint4 { unsigned x, y, z, w; };
inline float2 make_float2(float x, float y) { return {x, y}; }
inline uint2 make_uint2(unsigned x, unsigned y) { return {x, y}; }
inline uint4 make_uint4(unsigned x, unsigned y, unsigned z, unsigned w) { return {x, y, z, w}; }
struct dim3 { unsigned x, y, z; };
typedef void *hipStream_t;

namespace wave {
constexpr int kLanes = 64;
inline ucontext_t host, lanes[kLanes];
inline int at;                      // the lane that runs
inline int32_t slots[2][kLanes];
inline int turn[kLanes];            // which of the two slots a lane writes next

// Every lane's value, once all have come here.  (Two sets in turn: a lane may come to the next
// exchange while others still read this one.)
inline const int32_t *exchange(int32_t v) {
    const int t = turn[at];
    turn[at] ^= 1;
    slots[t][at] = v;
    swapcontext(&lanes[at], &host);
    return slots[t];
}

struct Index {
    struct X {
        operator unsigned() const { return static_cast<unsigned>(at); }
    } x;
};

// Runs f on 64 lanes; f comes to the same exchanges in all of them.
template <typename F>
void run(F f) {
    static char stacks[kLanes][1 << 15];
    static F *fn;
    static int left;
    fn = &f, left = kLanes;
    for (int l = 0; l < kLanes; ++l) {
        turn[l] = 0;
        getcontext(&lanes[l]);
        lanes[l].uc_stack.ss_sp = stacks[l];
        lanes[l].uc_stack.ss_size = sizeof stacks[l];
        lanes[l].uc_link = &host;
        makecontext(&lanes[l], +[] { (*fn)(); --left; }, 0);
    }
    while (left > 0)
        for (at = 0; at < kLanes; ++at) swapcontext(&host, &lanes[at]);
}
}  // namespace wave

static const wave::Index threadIdx = {};
static const dim3 blockDim = {wave::kLanes, 1, 1}, blockIdx = {0, 0, 0};

inline unsigned __umulhi(unsigned a, unsigned b) { return static_cast<unsigned>(static_cast<uint64_t>(a) * b >> 32); }
inline uint64_t __ballot(bool on) {
    const int32_t *v = wave::exchange(on);
    uint64_t m = 0;
    for (int l = 0; l < wave::kLanes; ++l) m |= static_cast<uint64_t>(v[l] != 0) << l;
    return m;
}
inline bool __any(bool on) { return __ballot(on) != 0; }

inline int wave_readlane(int v, int l) { return wave::exchange(v)[l & 63]; }
// Moves among lanes: CTRL 0x111 .. 0x11f from that many lanes before in the row of 16, 0x142 the row
// before's last lane, 0x143 lane 31; `old` where there is none or the row (a bit of ROWS) is left out.
inline int wave_update_dpp(int old, int v, int ctrl, int rows) {
    const int32_t *all = wave::exchange(v);
    const int l = wave::at, row = l >> 4;
    if (!((rows >> row) & 1)) return old;
    if (ctrl == 0x142) return row > 0 ? all[16 * row - 1] : old;
    if (ctrl == 0x143) return l >= 32 ? all[31] : old;
    const int n = ctrl - 0x110;
    return (l & 15) >= n ? all[l - n] : old;
}
inline float __shfl_xor(float v, int mask, int) {
    const int32_t *all = wave::exchange(__builtin_bit_cast(int32_t, v));
    return __builtin_bit_cast(float, all[wave::at ^ mask]);
}
#define __builtin_amdgcn_readlane(v, l) wave_readlane(v, l)
#define __builtin_amdgcn_readfirstlane(v) wave_readlane(v, 0)
#define __builtin_amdgcn_update_dpp(old, v, ctrl, rows, banks, bound) wave_update_dpp(old, v, ctrl, rows)
#define __builtin_amdgcn_logf(x) __builtin_log2f(x)
#define __builtin_amdgcn_exp2f(x) __builtin_exp2f(x)
