// Paged key-value cache: kv_cache_write and kv_cache_read for gfx950.
//
// The cache is the decode step's other stream beside the weights: a step reads every cached
// key and value once (deep-fold README, "Метод": a step reads only the valid prefix of the
// cache), so it is kept in bf16 or in 8 bits.  The 8-bit form of one head's row x of one
// token is
//     a = max|x|,  e = least integer >= -110 with a <= 448 * 2^e,
//     code = e4m3 nearest to x * 2^-e (ties to even),  value = code * 2^e,
// with the byte e + 127 beside the codes.  The scale is a power of two because the codes
// are floating point already: x * 2^-e, code * 2^e and the value's bf16 form are then exact,
// so the code's rounding (at most 2^-4 of a normal value) is the only one in the whole path,
// and a reader needs no multiplication that rounds.  A scale a / 448 would keep the same
// relative step.  e >= -110 keeps the smallest nonzero value, 2^(e - 9), a normal bf16
// number.
#include "device_common.h"

namespace wsl {
namespace {

constexpr int kExpMin = -110;

struct KvArgs {
    const void *k, *v;            // cache
    const uint8_t *ke, *ve;       // scale bytes (e4m3)
    int64_t page_stride, head_stride, token_stride;   // elements
    int64_t n_slots;
    int64_t ld_k, ld_v;           // rows outside the cache: elements from token to token
    uint32_t rows, n_kv, head_dim, page_size;
    int lane_shift;               // log2 of the lanes that share one row
};

// Index of the page and of the token in it: 32-bit division where every slot fits.
__device__ __forceinline__ void split_slot(const KvArgs &a, int64_t slot, int64_t &page, uint32_t &at) {
    if (a.n_slots <= 0xffffffffll) {
        const uint32_t s = static_cast<uint32_t>(slot), p = s / a.page_size;
        page = p;
        at = s - p * a.page_size;
    } else {
        page = slot / a.page_size;
        at = static_cast<uint32_t>(slot - page * a.page_size);
    }
}

// One lane holds 8 consecutive elements of a row; 1 << lane_shift lanes share the row (head_dim
// / 8 rounded up to a power of two, lanes beyond head_dim idle), so a row's maximum is a few
// lane exchanges and every access is 8 to 32 bytes of consecutive memory per lane.  (For 64000 tokens
// of 8 heads of 128, bf16 to fp32: 149 us; lanes of 4 elements, 16 bytes of fp32, 192; two and four
// rows a lane at once 161 and 171.)
template <int FMT, int XFMT>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a, const void *__restrict__ k_new,
                                                       const void *__restrict__ v_new,
                                                       const int64_t *__restrict__ slots,
                                                       uint32_t *__restrict__ status) {
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    const uint32_t row = id >> a.lane_shift, d = (id & ((1u << a.lane_shift) - 1u)) * 8u;
    const bool is_v = blockIdx.y != 0;
    const bool in = row < a.rows && d < a.head_dim;
    const uint32_t tok = in ? row / a.n_kv : 0, head = in ? row - tok * a.n_kv : 0;
    float x[8];
    uint4 raw = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (in) {
        const int64_t src = static_cast<int64_t>(tok) * (is_v ? a.ld_v : a.ld_k) +
                            static_cast<int64_t>(head) * a.head_dim + d;
        const void *from = is_v ? v_new : k_new;
        if constexpr (XFMT == WSL_OUT_F32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(from) + src);
            const float4 lo = p[0], hi = p[1];
            x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w;
            x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
        } else {
            raw = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(from) + src);
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    const int64_t slot = in ? slots[tok] : -1;
    const bool put = slot >= 0 && slot < a.n_slots;
    int64_t page = 0;
    uint32_t at = 0;
    if (put) split_slot(a, slot, page, at);
    if (in && !put && slot != -1 && status != nullptr && d == 0 && head == 0) atomicOr(status, WSL_STATUS_INDEX);
    const int64_t dst = page * a.page_stride + static_cast<int64_t>(head) * a.head_stride +
                        static_cast<int64_t>(at) * a.token_stride + d;
    void *cache = const_cast<void *>(is_v ? a.v : a.k);
    if constexpr (FMT == WSL_KV_BF16) {
        if constexpr (XFMT == WSL_OUT_F32)
            raw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                             pack_bf16x2(x[6], x[7]));
        if (put) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(cache) + dst) = raw;
    } else {
        // max over the bit patterns of |x|: ordered like the values, infinities and NaN above
        // every finite value
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu;
            top = b > top ? b : top;
        }
        for (int off = (1 << a.lane_shift) >> 1; off >= 1; off >>= 1) {
            const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), off, 64));
            top = o > top ? o : top;
        }
        uint2 codes;
        int e = 0;
        if (top >= 0x7f800000u) {      // a NaN or an infinity: the row reads back as NaN
            codes = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
            if (put && d == 0 && status != nullptr) atomicOr(status, WSL_STATUS_NONFINITE);
        } else {
            // a = (1 + f / 2^23) * 2^n, 448 = 1.75 * 2^8 (a subnormal a is below every e >= -110)
            e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
            e = e < kExpMin ? kExpMin : e;
            const float inv = __builtin_bit_cast(float, static_cast<uint32_t>(127 - e) << 23);
            int lo = 0, hi = 0;
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, lo, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, lo, true);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * inv, x[5] * inv, hi, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * inv, x[7] * inv, hi, true);
            codes = make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
        }
        if (put) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + dst) = codes;
            if (d == 0)
                const_cast<uint8_t *>(is_v ? a.ve : a.ke)[(page * a.n_kv + head) * a.page_size + at] =
                    static_cast<uint8_t>(e + 127);
        }
    }
}

// The same lane assignment, the other way.  code * 2^e is exact in fp32 and, e4m3 having four
// significant bits and e >= -110, in bf16.  Cache and outputs are streamed (the 64000 tokens 149 -> 142
// us, 5.5 TB/s read and written; streaming the cache alone 140, but 8192 tokens written and read 22.6
// us against 21.4).
template <int FMT, int OFMT>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a, const int64_t *__restrict__ slots,
                                                      void *__restrict__ k_out, void *__restrict__ v_out,
                                                      uint32_t *__restrict__ status) {
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    const uint32_t row = id >> a.lane_shift, d = (id & ((1u << a.lane_shift) - 1u)) * 8u;
    const bool is_v = blockIdx.y != 0;
    if (row >= a.rows || d >= a.head_dim) return;
    const uint32_t tok = row / a.n_kv, head = row - tok * a.n_kv;
    const int64_t slot = slots[tok];
    const bool get = slot >= 0 && slot < a.n_slots;
    if (!get && slot != -1 && status != nullptr && d == 0 && head == 0) atomicOr(status, WSL_STATUS_INDEX);
    u32x4 raw = {0, 0, 0, 0};               // bf16 pairs
    if (get) {
        int64_t page;
        uint32_t at;
        split_slot(a, slot, page, at);
        const int64_t src = page * a.page_stride + static_cast<int64_t>(head) * a.head_stride +
                            static_cast<int64_t>(at) * a.token_stride + d;
        const void *cache = is_v ? a.v : a.k;
        if constexpr (FMT == WSL_KV_BF16) {
            raw = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(cache) + src));
        } else {
            const u32x2 c = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(cache) + src));
            const uint8_t eb = (is_v ? a.ve : a.ke)[(page * a.n_kv + head) * a.page_size + at];
            const float s = __builtin_bit_cast(float, static_cast<uint32_t>(eb) << 23);
            raw.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, false));
            raw.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, true));
            raw.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, false));
            raw.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, true));
        }
    }
    const int64_t dst = static_cast<int64_t>(tok) * (is_v ? a.ld_v : a.ld_k) +
                        static_cast<int64_t>(head) * a.head_dim + d;
    void *out = is_v ? v_out : k_out;
    if constexpr (OFMT == WSL_OUT_BF16) {
        __builtin_nontemporal_store(raw, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(out) + dst));
    } else {
        f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(out) + dst);
        __builtin_nontemporal_store(f32x4{bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)}, o);
        __builtin_nontemporal_store(f32x4{bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)}, o + 1);
    }
}

KvArgs make_args(const wsl_kv_cache *c, int64_t count, int64_t ld_k, int64_t ld_v) {
    KvArgs a;
    a.k = c->k, a.v = c->v, a.ke = c->k_exp, a.ve = c->v_exp;
    a.page_stride = c->page_stride, a.head_stride = c->head_stride, a.token_stride = c->token_stride;
    a.n_slots = c->n_pages * c->page_size;
    a.ld_k = ld_k, a.ld_v = ld_v;
    a.rows = static_cast<uint32_t>(count * c->n_kv);
    a.n_kv = static_cast<uint32_t>(c->n_kv);
    a.head_dim = static_cast<uint32_t>(c->head_dim);
    a.page_size = static_cast<uint32_t>(c->page_size);
    a.lane_shift = 1;
    while ((8 << a.lane_shift) < c->head_dim) ++a.lane_shift;
    return a;
}

dim3 grid_of(const KvArgs &a) {
    return dim3(static_cast<unsigned>(((static_cast<int64_t>(a.rows) << a.lane_shift) + 255) / 256), 2);
}

}  // namespace

int launch_kv_write(const wsl_kv_cache *c, const void *k, const void *v, int xfmt, int64_t count, int64_t ld_k,
                    int64_t ld_v, const int64_t *slots, uint32_t *status, hipStream_t s) {
    const KvArgs a = make_args(c, count, ld_k, ld_v);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid_of(a), dim3(256), 0, s, a, k, v, slots, status); };
    if (c->fmt == WSL_KV_BF16)
        xfmt == WSL_OUT_F32 ? go(kv_write_kernel<WSL_KV_BF16, WSL_OUT_F32>)
                            : go(kv_write_kernel<WSL_KV_BF16, WSL_OUT_BF16>);
    else
        xfmt == WSL_OUT_F32 ? go(kv_write_kernel<WSL_KV_E4M3, WSL_OUT_F32>)
                            : go(kv_write_kernel<WSL_KV_E4M3, WSL_OUT_BF16>);
    return WSL_OK;
}

int launch_kv_read(const wsl_kv_cache *c, const int64_t *slots, int64_t count, void *k, void *v, int ofmt,
                   int64_t ld_k, int64_t ld_v, uint32_t *status, hipStream_t s) {
    const KvArgs a = make_args(c, count, ld_k, ld_v);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid_of(a), dim3(256), 0, s, a, slots, k, v, status); };
    if (c->fmt == WSL_KV_BF16)
        ofmt == WSL_OUT_F32 ? go(kv_read_kernel<WSL_KV_BF16, WSL_OUT_F32>)
                            : go(kv_read_kernel<WSL_KV_BF16, WSL_OUT_BF16>);
    else
        ofmt == WSL_OUT_F32 ? go(kv_read_kernel<WSL_KV_E4M3, WSL_OUT_F32>)
                            : go(kv_read_kernel<WSL_KV_E4M3, WSL_OUT_BF16>);
    return WSL_OK;
}

}  // namespace wsl
