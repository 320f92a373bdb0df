// Pages of a key-value cache kept on the device: kv_pages_grow and kv_pages_trim for gfx950.
//
// IPE page, "What is built": a decode step reads no device value back.  Lengths, block table and the
// stack of free pages stay on the device, so a captured step can take in its tokens, and give the
// pages of fallen drafts back, by itself.  With held_b = ceil(len_b / page), need_b the pages that
// sequence b lacks and off_b the sum of need over those before it, page i of b is
// free[n_free - 1 - off_b - i]: one running sum over the sequences, after which every token finds its
// own slot without looking at another.
//
// Bound: latency, of one workgroup's loads one after the other; the bytes (16 to 20 a token) are nothing.
// Measured: grow 3.2 us for one sequence, 6.8 for 256 of 5 tokens; 4.6 and 4.5 in two launches for
// 64 prompts of 166,500 tokens together; trim of the same 4.7, 5.3 and 11.7.
#include "device_common.h"

namespace wsl {
namespace {

constexpr int kMost = 1024;            // threads of the workgroup that goes over the sequences
// Tokens that it sees to itself.  That and a second launch for them, grow and trim together, in us: 64 sequences, 64 tokens
// 10.3 and 11.6, 1024 12.5 and 12.9, 4096 15.2 and 13.2, 16384 25 and 13; 1024 sequences, 1024 tokens 15.4 and 18.9, 4096 18.5 and
// 19.1, 8192 22.8 and 18.9.  (Outside of graphs, a launch costs the host 2.7 us besides.)
constexpr int64_t kOneLaunch = 4096;

// What the tokens of a sequence need to know.
struct Row {
    int32_t start, count;              // its tokens in the call's
    int32_t len;                       // before the call; -1: the tokens are not taken in
    int32_t top;                       // place in the stack of the first page taken
};

struct PagesArgs {
    int32_t *table, *lens, *free_pages, *n_free;
    const int32_t *want;               // new tokens of each sequence, or the lengths to trim to
    int64_t each, n_tokens;
    int64_t *slots, *positions;
    int32_t *starts;
    Row *rows;
    uint32_t *status;
    int64_t ld_table;
    uint32_t n_seq, n_pages, page_size, capacity;      // capacity: tokens of a row
};

__device__ __forceinline__ uint32_t pages_of(uint32_t tokens, uint32_t page_size) {
    return (tokens + page_size - 1) / page_size;       // tokens < 2^31, page_size <= 2^30
}

__device__ __forceinline__ int32_t clamped(int32_t n_free, uint32_t n_pages, bool &bad) {
    const int32_t most = static_cast<int32_t>(n_pages);
    if (n_free < 0 || n_free > most) bad = true;
    return n_free < 0 ? 0 : (n_free > most ? most : n_free);
}

// Sums over the threads before this one, and over all.  `sums` holds one entry a wave.
__device__ __forceinline__ int64_t before(int64_t v, int64_t &all, int64_t *sums) {
    const int lane = static_cast<int>(threadIdx.x & 63), wave = static_cast<int>(threadIdx.x >> 6);
    const int waves = static_cast<int>(blockDim.x >> 6);
    int64_t up = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(static_cast<long long>(up), off, 64);
        if (lane >= off) up += o;
    }
    __syncthreads();                                   // the sums of the call before have been read
    if (lane == 63) sums[wave] = up;
    __syncthreads();
    int64_t at = up - v;
    all = 0;
    for (int w = 0; w < waves; ++w) {
        if (w < wave) at += sums[w];
        all += sums[w];
    }
    return at;
}

// The slot and position of token t, which lies in sequence b.
__device__ __forceinline__ void place_token(const PagesArgs &a, uint32_t t, uint32_t b, const Row &r, bool &bad) {
    int64_t slot = -1, position = -1;
    const uint32_t i = t - static_cast<uint32_t>(r.start);
    if (r.len >= 0 && i < static_cast<uint32_t>(r.count)) {
        const uint32_t at = static_cast<uint32_t>(r.len) + i, place = at / a.page_size, in = at - place * a.page_size;
        const uint32_t held = pages_of(static_cast<uint32_t>(r.len), a.page_size);
        int32_t *entry = a.table + b * a.ld_table + place;
        int32_t page;
        if (place < held) {
            page = *entry;
        } else {
            page = a.free_pages[r.top - static_cast<int32_t>(place - held)];
            if (in == 0) *entry = page;                // every new page's first token is in this call
        }
        position = at;
        if (static_cast<uint32_t>(page) < a.n_pages) slot = static_cast<int64_t>(page) * a.page_size + in;
        else bad = true;
    }
    a.slots[t] = slot;
    if (a.positions != nullptr) a.positions[t] = position;
}

// The sequence whose tokens hold t: the last that starts at or before it.
template <typename Starts>
__device__ __forceinline__ uint32_t sequence_of(uint32_t t, uint32_t n_seq, Starts start) {
    uint32_t lo = 0, n = n_seq;                        // n_seq >= 1
    while (n > 1) {
        const uint32_t half = n / 2;
        if (static_cast<uint32_t>(start(lo + half)) <= t) lo += half;
        n -= half;
    }
    return lo;
}

// One workgroup: the running sums over all sequences.  ALL: their tokens too.
template <bool ALL>
__global__ __launch_bounds__(kMost) void grow_kernel(PagesArgs a) {
    __shared__ int64_t sums[kMost / 64];
    __shared__ Row rows[ALL ? kMost : 1];
    __shared__ int32_t taken;
    const uint32_t tid = threadIdx.x;
    bool bad = false, out_of_pages = false;
    const int32_t had = a.n_seq ? clamped(*a.n_free, a.n_pages, bad) : 0;
    if (tid == 0) taken = 0;
    int64_t tokens = 0, needs = 0;
    for (uint32_t b0 = 0; b0 < a.n_seq; b0 += blockDim.x) {
        const uint32_t b = b0 + tid;
        const bool in = b < a.n_seq;
        const int64_t len = in ? a.lens[b] : 0, grow = !in ? 0 : (a.want != nullptr ? a.want[b] : a.each);
        const int64_t count = grow > 0 ? grow : 0;
        int64_t all;
        const int64_t start = tokens + before(count, all, sums);
        tokens += all;
        const bool ok = in && len >= 0 && len <= a.capacity && grow >= 0 && grow <= a.capacity - len &&
                        (count == 0 || start + count <= a.n_tokens);
        bad |= in && !ok;
        const int64_t need = ok ? pages_of(static_cast<uint32_t>(len + grow), a.page_size) -
                                      static_cast<int64_t>(pages_of(static_cast<uint32_t>(len), a.page_size)) : 0;
        const int64_t off = needs + before(need, all, sums);
        needs += all;
        const bool served = ok && (need == 0 || off + need <= had);
        out_of_pages |= ok && !served;
        if (in) {
            Row r;
            r.start = static_cast<int32_t>(start < a.n_tokens ? start : a.n_tokens);
            r.count = static_cast<int32_t>(count < a.n_tokens ? count : a.n_tokens);
            r.len = served ? static_cast<int32_t>(len) : -1;
            r.top = served && need ? had - 1 - static_cast<int32_t>(off) : 0;
            if constexpr (ALL) rows[b] = r;
            else a.rows[b] = r;
            if (served && grow) a.lens[b] = static_cast<int32_t>(len + grow);
            if (served && need) atomicMax(&taken, static_cast<int32_t>(off + need));
            if (a.starts != nullptr) a.starts[b] = r.start;
        }
    }
    __syncthreads();
    if (tid == 0) {
        if (a.n_seq) *a.n_free = had - taken;
        if (a.starts != nullptr) a.starts[a.n_seq] = static_cast<int32_t>(tokens < a.n_tokens ? tokens : a.n_tokens);
    }
    if constexpr (ALL) {
        for (uint32_t t = tid; t < a.n_tokens; t += blockDim.x) {
            Row none = {0, 0, -1, 0};
            uint32_t b = 0;
            if (a.n_seq) {
                b = sequence_of(t, a.n_seq, [&](uint32_t i) { return rows[i].start; });
                none = rows[b];
            }
            place_token(a, t, b, none, bad);
        }
    }
    const uint32_t st = (bad ? WSL_STATUS_INDEX : 0u) | (out_of_pages ? WSL_STATUS_PAGES : 0u);
    if (st && a.status != nullptr) atomicOr(a.status, st);
}

__global__ __launch_bounds__(256) void slots_kernel(PagesArgs a) {
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    if (t >= a.n_tokens) return;
    bool bad = false;
    Row r = {0, 0, -1, 0};
    uint32_t b = 0;
    if (a.n_seq) {
        b = sequence_of(t, a.n_seq, [&](uint32_t i) { return a.rows[i].start; });
        r = a.rows[b];
    }
    place_token(a, t, b, r, bad);
    if (bad && a.status != nullptr) atomicOr(a.status, WSL_STATUS_INDEX);
}

// One workgroup.  The total first: the last page given back lies lowest.
__global__ __launch_bounds__(kMost) void trim_kernel(PagesArgs a) {
    __shared__ int64_t sums[kMost / 64];
    __shared__ uint32_t offs[kMost], first[kMost];
    const uint32_t tid = threadIdx.x;
    bool bad = false;
    const int32_t had = clamped(*a.n_free, a.n_pages, bad);
    // pages that sequence b gives back, and the first of them
    const auto gives = [&](uint32_t b, uint32_t &at, int32_t &len) -> uint32_t {
        at = 0, len = -1;
        if (b >= a.n_seq) return 0;
        const int32_t is = a.lens[b], to = a.want[b];
        if (is < 0 || static_cast<uint32_t>(is) > a.capacity || to < 0) {
            bad = true;
            return 0;
        }
        if (to >= is) return 0;
        len = to;
        at = pages_of(static_cast<uint32_t>(to), a.page_size);
        return pages_of(static_cast<uint32_t>(is), a.page_size) - at;
    };
    int64_t total = 0, all, given = 0;
    uint32_t at;
    int32_t len;
    for (uint32_t b0 = 0; b0 < a.n_seq; b0 += blockDim.x) {
        before(gives(b0 + tid, at, len), all, sums);
        total += all;
    }
    for (uint32_t b0 = 0; b0 < a.n_seq; b0 += blockDim.x) {
        const uint32_t back = gives(b0 + tid, at, len);
        const int64_t off = before(back, all, sums);   // pages of 2^31 - 1 tokens: a chunk's fit 42 bits
        // a chunk's pages that the stack can hold at all fit 31 bits; beyond, they are dropped
        offs[tid] = static_cast<uint32_t>(off < 0x7fffffff ? off : 0x7fffffff);
        first[tid] = at;
        if (len >= 0) a.lens[b0 + tid] = len;
        __syncthreads();
        const uint32_t here = static_cast<uint32_t>(all < 0x7fffffff ? all : 0x7fffffff);
        const uint32_t seqs = a.n_seq - b0 < blockDim.x ? a.n_seq - b0 : blockDim.x;
        for (uint32_t i = tid; i < here; i += blockDim.x) {
            const uint32_t s = sequence_of(i, seqs, [&](uint32_t j) { return offs[j]; });
            const int64_t dest = had + total - 1 - given - i;
            if (dest < a.n_pages) a.free_pages[dest] = a.table[(b0 + s) * a.ld_table + first[s] + (i - offs[s])];
            else bad = true;
        }
        given += all;
        __syncthreads();
    }
    if (tid == 0 && total) *a.n_free = static_cast<int32_t>(had + total < a.n_pages ? had + total : a.n_pages);
    if (bad && a.status != nullptr) atomicOr(a.status, WSL_STATUS_INDEX);
}

PagesArgs args_of(const wsl_kv_pages *p, const int32_t *want, uint32_t *status) {
    PagesArgs a = {};
    a.table = p->table, a.lens = p->lens, a.free_pages = p->free_pages, a.n_free = p->n_free;
    a.want = want, a.status = status;
    a.ld_table = p->ld_table;
    a.n_seq = static_cast<uint32_t>(p->n_seq);
    a.n_pages = static_cast<uint32_t>(p->n_pages);
    a.page_size = static_cast<uint32_t>(p->page_size);
    const int64_t room = p->pages_per_seq * p->page_size;      // < 2^61
    a.capacity = static_cast<uint32_t>(room < 0x7fffffff ? room : 0x7fffffff);
    return a;
}

unsigned threads_for(int64_t n) {
    const int64_t t = (n + 63) / 64 * 64;
    return static_cast<unsigned>(t < 64 ? 64 : (t > kMost ? kMost : t));
}

}  // namespace

size_t grow_ws_bytes(int64_t n_seq, int64_t n_tokens) {
    return n_seq <= kMost && n_tokens <= kOneLaunch ? 0 : static_cast<size_t>(n_seq) * sizeof(Row);
}

int launch_grow(const wsl_kv_pages *p, const int32_t *d_new, int64_t each, int64_t n_tokens, int64_t *slots,
                int64_t *positions, int32_t *starts, void *ws, uint32_t *status, hipStream_t s) {
    PagesArgs a = args_of(p, d_new, status);
    a.each = each, a.n_tokens = n_tokens, a.slots = slots, a.positions = positions, a.starts = starts;
    a.rows = static_cast<Row *>(ws);
    if (p->n_seq <= kMost && n_tokens <= kOneLaunch) {
        hipLaunchKernelGGL(grow_kernel<true>, dim3(1), dim3(threads_for(p->n_seq > n_tokens ? p->n_seq : n_tokens)), 0, s, a);
        return WSL_OK;
    }
    hipLaunchKernelGGL(grow_kernel<false>, dim3(1), dim3(threads_for(p->n_seq)), 0, s, a);
    if (n_tokens)
        hipLaunchKernelGGL(slots_kernel, dim3(static_cast<unsigned>((n_tokens + 255) / 256)), dim3(256), 0, s, a);
    return WSL_OK;
}

int launch_trim(const wsl_kv_pages *p, const int32_t *lens, uint32_t *status, hipStream_t s) {
    hipLaunchKernelGGL(trim_kernel, dim3(1), dim3(kMost), 0, s, args_of(p, lens, status));
    return WSL_OK;
}

}  // namespace wsl
