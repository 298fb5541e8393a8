// KV cache in q4_0 pages: the plan of a step (offsets, pages, slots) and the
// append of new keys and values.
//
// kq_kv_plan is two scans over the requests (new tokens, fresh pages) and one
// map over the tokens:
//   cu[b] = min(sum of new before b, cap),  seq = cached + new,
//   first[b] = taken + sum over earlier requests of their fresh pages,
//   slot(t) = page(pos / page_size) * page_size + pos % page_size.
// A fresh page always begins with one of the step's own tokens, so the thread
// of that token writes the table entry, and every other thread of the page
// computes the same page from free_pages without reading the table.
//
// Both are bound by latency (one launch for up to 4096 tokens, else two):
// 48 requests of one token 4.0 us, 1021 prompts of 460,000 tokens 8.8 us.
//
// kq_kv_append writes each 32-value block as d = -m / 8 (m the value of
// largest magnitude, the first of equals) and codes trunc(x * (1/d) + 8.5) in
// 0..15, every step a separately rounded fp32 operation.
// Bound by instruction issue for prompts (72 % of the slots, the ALU pipe 68 %),
// by latency for a step: 8192 tokens of 8 heads of 128 in fp32 19.1 us (77 MB,
// 4.0 TB/s; packed fp32 multiplies and adds: 2 % less), 2777 tokens of 5 heads of 64 in bf16
// 8 us, 48 tokens of 8 heads of 128 in bf16 5.7 us.
#include "kq_kv.cuh"

namespace kq {
namespace {

constexpr int kPlanThreads = 1024;

struct PlanParams {
    const int32_t* cached;
    const int32_t* fresh;       // new tokens per request
    int n_seqs;
    int page;
    Divisor by_page;
    int32_t* table;
    int max_blocks;
    const int32_t* free_pages;
    int n_free;
    const int32_t* taken;
    int32_t* taken_out;
    int32_t* seq_lens;
    int32_t* cu;
    int32_t* first;
    int32_t* slots;
    int32_t* positions;
    int cap;
    int32_t* err;
};

// Inclusive scan of one value per thread over the CTA (kPlanThreads threads);
// the total is left in *total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();   // part is free again
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int64_t w = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        part[lane] = w;
    }
    __syncthreads();
    *total = part[31];
    return v + (warp ? part[warp - 1] : 0);
}

// Token t of the step: its request (the last b with cu[b] <= t, found in the
// n_seqs + 1 ascending offsets), position and slot; the page's first token
// writes a fresh page's table entry.
__device__ __forceinline__ int plan_find(const int32_t* cu, int lo, int hi, int t) {
    while (lo < hi) {   // first b with cu[b + 1] > t
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
__device__ __forceinline__ void plan_token(const PlanParams& p, const int32_t* cu, int total, int t, int lo, int hi, int& bad) {
    int slot = -1, pos = -1;
    if (t < total) {
        lo = plan_find(cu, lo, hi, t);
        const int c0 = cu[lo], c1 = cu[lo + 1];
        const int old = p.seq_lens[lo] - (c1 - c0);
        pos = old + (t - c0);
        const int j = divide(pos, p.by_page), off = pos - j * p.page;
        const int held = divide(old + p.page - 1, p.by_page);
        int page = -1;
        if (j >= p.max_blocks) {
            bad |= KQ_DEV_TOO_MANY;
        } else if (j >= held) {
            const int64_t at = static_cast<int64_t>(p.first[lo]) + (j - held);
            if (at < p.n_free) page = p.free_pages[at];
            else bad |= KQ_DEV_TOO_MANY;
            if (off == 0) p.table[static_cast<int64_t>(lo) * p.max_blocks + j] = page;
            if (at < p.n_free && page < 0) bad |= KQ_DEV_BAD_RANGE;
        } else {
            page = p.table[static_cast<int64_t>(lo) * p.max_blocks + j];
            if (page < 0) bad |= KQ_DEV_BAD_RANGE;
        }
        const int64_t at = static_cast<int64_t>(page) * p.page + off;
        if (page >= 0) {
            if (at <= 0x7fffffff) slot = static_cast<int>(at);
            else bad |= KQ_DEV_BAD_RANGE;
        }
    }
    p.slots[t] = slot;
    if (p.positions) p.positions[t] = pos;
}

// One CTA: both scans; with `map` also the tokens (a step's few tokens need
// no second launch).
__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(const PlanParams p, int map) {
    __shared__ int64_t part[32];
    pdl_launch();
    pdl_wait();
    const int tid = threadIdx.x;
    int64_t tokens = 0, pages = 0;   // running totals
    int bad = 0;
    int64_t taken = *p.taken;
    if (taken < 0) {
        taken = 0;
        bad |= KQ_DEV_BAD_RANGE;
    }
    const int most = p.max_blocks * p.page;
    for (int b0 = 0; b0 < p.n_seqs; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int old = 0, add = 0;
        if (b < p.n_seqs) {
            old = p.cached[b];
            add = p.fresh[b];
            if (old < 0 || old > most || add < 0) bad |= KQ_DEV_BAD_RANGE;
            old = old < 0 ? 0 : (old > most ? most : old);
            add = add < 0 ? 0 : add;
        }
        int64_t sum;
        int64_t end = tokens + block_scan(add, part, &sum);
        int64_t begin = end - add;
        if (end > p.cap) bad |= KQ_DEV_TOO_MANY;
        begin = begin < p.cap ? begin : p.cap;
        end = end < p.cap ? end : p.cap;
        tokens += sum;
        const int put = static_cast<int>(end - begin);
        const int seq = old + put;
        int need = 0;
        if (b < p.n_seqs) {
            int blocks = divide(seq + p.page - 1, p.by_page), held = divide(old + p.page - 1, p.by_page);
            blocks = blocks < p.max_blocks ? blocks : p.max_blocks;
            need = blocks > held ? blocks - held : 0;
        }
        const int64_t pend = pages + block_scan(need, part, &sum);
        pages += sum;
        if (b < p.n_seqs) {
            p.seq_lens[b] = seq;
            p.cu[b] = static_cast<int>(begin);
            const int64_t at = taken + pend - need;
            p.first[b] = at < p.n_free ? static_cast<int>(at) : p.n_free;
        }
    }
    const int total = static_cast<int>(tokens < p.cap ? tokens : p.cap);
    if (tid == 0) {
        p.cu[p.n_seqs] = total;
        const int64_t at = taken + pages;
        *p.taken_out = static_cast<int>(at < p.n_free ? at : (taken > p.n_free ? taken : p.n_free));
    }
    if (map) {
        __syncthreads();   // the offsets written above
        for (int t = tid; t < p.cap; t += kPlanThreads) plan_token(p, p.cu, total, t, 0, p.n_seqs - 1, bad);
    }
    if (bad && p.err) atomicOr(p.err, bad);
}

// plan_find by a whole warp: 32 offsets a step instead of one.
__device__ __forceinline__ int plan_find_warp(const int32_t* cu, int lo, int hi, int t) {
    const int lane = threadIdx.x & 31;
    while (hi - lo >= 32) {
        const int step = (hi - lo + 32) / 32, at = lo + step * lane;   // the last lane's is at most hi
        const unsigned past = __ballot_sync(0xffffffffu, at >= hi || cu[at + 1] > t);
        const int l = __ffs(past) - 1;
        if (past == 0) {
            lo = lo + step * 31 + 1;
        } else {
            hi = lo + step * l < hi ? lo + step * l : hi;
            lo = l ? lo + step * (l - 1) + 1 : lo;
        }
    }
    const unsigned past = __ballot_sync(0xffffffffu, lo + lane >= hi || cu[lo + lane + 1] > t);
    return lo + __ffs(past) - 1;
}

// 1024 tokens a block; the requests of its first and last token bound the
// others' search.  Bound by latency: two dependent searches and a store.
__global__ void __launch_bounds__(256) plan_map_kernel(const PlanParams p) {
    pdl_launch();
    pdl_wait();
    __shared__ int ends[2];
    const int t0 = blockIdx.x * 1024, total = p.cu[p.n_seqs], warp = threadIdx.x >> 5;
    if (warp < 2 && t0 < total) {
        const int last = total - 1 < t0 + 1023 ? total - 1 : t0 + 1023;
        const int b = plan_find_warp(p.cu, 0, p.n_seqs - 1, warp ? last : t0);
        if ((threadIdx.x & 31) == 0) ends[warp] = b;
    }
    __syncthreads();
    int bad = 0;
    for (int k = 0; k < 4; ++k) {
        const int t = t0 + 256 * k + threadIdx.x;
        if (t < p.cap) plan_token(p, p.cu, total, t, ends[0], ends[1], bad);
    }
    if (bad && p.err) atomicOr(p.err, bad);
}

// ------------------------------------------------------------------ append
struct AppendParams {
    const void* src[2];        // k, v
    uint8_t* pool[2];
    int64_t stride[2];         // elements between tokens
    const int32_t* slots;
    int n_blocks;              // tokens * heads * blocks of a row
    int n_slots;
    int n_heads;
    int page;
    Divisor by_heads, by_page;
    int32_t* err;
};

// Four lanes a block of 32 values, eight consecutive values a lane, for the key
// and the value of the same place: 4 or 8 bytes read and 1.125 written for a
// key and value.  An even block and the odd one after it
// are 9 words:
//   d0 c0 c1 | c2..c5 | c6..c9 | c10..c13 | c14 c15 d1 | c0..c3 | ... | c12..c15
// (c: code bytes), so the lanes of an even block store their four bytes shifted
// by two, with the last two bytes of the lane before; those of an odd block as
// they are.  Nothing orders the words of two tokens with one slot: each word is
// one token's.
template <bool F32>
struct Eight {
    uint4 a, b;
};
template <>
struct Eight<false> {
    uint4 a;
};
template <bool F32>
__device__ __forceinline__ Eight<F32> load_eight(const void* src, int64_t at) {
    Eight<F32> r;
    if constexpr (F32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(src) + at);
        r.a = ldg_nc_v4(s);
        r.b = ldg_nc_v4(s + 1);
    } else {
        r.a = ldg_nc_v4(static_cast<const uint16_t*>(src) + at);
    }
    return r;
}
template <bool F32>
__device__ __forceinline__ void widen(const Eight<F32>& r, float (&x)[8]) {
    if constexpr (F32) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
    } else {
        const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = bf16lo_to_f32(w[k]);
            x[2 * k + 1] = bf16hi_to_f32(w[k]);
        }
    }
}

// Encodes the quad's 32 values and stores them into the row pair at `dst` (the
// even block's first byte).  All lanes of the warp take part.
__device__ __forceinline__ int encode_store(const float (&x)[8], bool put, bool odd, uint8_t* dst) {
    const int lane = threadIdx.x & 31, part = lane & 3;
    // largest magnitude, the first of equals (magnitudes order as their bits)
    float m = x[0];
    uint32_t mb = __float_as_uint(x[0]) & 0x7fffffffu;
#pragma unroll
    for (int k = 1; k < 8; ++k) {
        const uint32_t b = __float_as_uint(x[k]) & 0x7fffffffu;
        if (b > mb) {
            mb = b;
            m = x[k];
        }
    }
    uint32_t top = mb;
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const unsigned who = (__ballot_sync(0xffffffffu, mb == top) >> (lane & 28)) & 15u;
    m = __shfl_sync(0xffffffffu, m, (lane & 28) + __ffs(who) - 1);
    const float d = m * -0.125f;
    const uint32_t hb = __half_as_ushort(__float2half_rn(d));
    const float inv = (hb & 0x7fffu) == 0 ? 0.f : __frcp_rn(d);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // 0.49 .. 16.5; adding 2^23 towards zero leaves the integer part
        const float f = fminf(__fadd_rn(__fmul_rn(x[k], inv), 8.5f), 15.f);
        const uint32_t q = __float_as_uint(__fadd_rz(f, 8388608.f));
        c[k >> 2] |= (q & 15u) << (8 * (k & 3));
    }
    // values 0..15 are the low nibbles, 16..31 the high ones: bytes 8 part .. of
    // the lower lanes meet those of the lane two on
    const bool upper = part >= 2;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? c[0] : c[1], 2);
    const uint32_t bytes = upper ? (got | (c[1] << 4)) : (c[0] | (got << 4));
    // word q of the block: lanes 0, 2, 1, 3 hold bytes 0.., 4.., 8.., 12..
    const int q = 2 * (part & 1) + (part >> 1);
    const int before = (lane & 28) + (part == 0 ? 0 : part == 2 ? 0 : part == 1 ? 2 : 1);   // lane of word q - 1
    const uint32_t prev = __shfl_sync(0xffffffffu, bytes, before);
    const uint32_t next_d = __shfl_down_sync(0xffffffffu, hb, 4);   // the odd block's scale
    if (put) {
        uint32_t* w = reinterpret_cast<uint32_t*>(dst);
        if (odd) {
            w[5 + q] = bytes;
        } else {
            w[q] = __byte_perm(q ? prev >> 16 : hb, bytes, 0x5410);
            if (q == 3) w[4] = (bytes >> 16) | (next_d << 16);
        }
    }
    return put && (hb & 0x7fffu) > 0x6fffu ? KQ_DEV_X_RANGE : 0;   // past 8188: a value past 65504
}

template <bool F32, int NB>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    pdl_launch();
    pdl_wait();
    const int part = threadIdx.x & 3;
    const int i = static_cast<int>(blockIdx.x * 64u + (threadIdx.x >> 2));   // block
    const bool in = i < p.n_blocks;
    const int row = (in ? i : 0) / NB, blk = (in ? i : 0) - row * NB;
    const int tok = divide(row, p.by_heads), head = row - tok * p.n_heads;
    const int slot = p.slots[tok];
    const bool put = in && slot >= 0 && slot < p.n_slots;
    int bad = in && !put && slot != -1 ? KQ_DEV_BAD_RANGE : 0;
    const int at = (head * NB + blk) * 32 + 8 * part;
    const Eight<F32> rk = load_eight<F32>(p.src[0], tok * p.stride[0] + at);
    const Eight<F32> rv = load_eight<F32>(p.src[1], tok * p.stride[1] + at);
    const int pg = divide(put ? slot : 0, p.by_page);
    const int off = (put ? slot : 0) - pg * p.page;
    // the row pair of an even block and the odd one after it (NB is even)
    const int64_t to = ((static_cast<int64_t>(pg) * p.n_heads + head) * p.page + off) * (NB * 18) + (blk >> 1) * 36;
    float x[8];
    widen<F32>(rk, x);
    bad |= encode_store(x, put, blk & 1, p.pool[0] + to);
    widen<F32>(rv, x);
    bad |= encode_store(x, put, blk & 1, p.pool[1] + to);
    if (bad && p.err) atomicOr(p.err, bad);
}

template <bool F32>
int append_of(const AppendParams& p, int nb, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.n_blocks) + 63) / 64));
    switch (nb) {
    case 2: return launch_pdl(append_kernel<F32, 2>, grid, 256, 0, s, p);
    case 4: return launch_pdl(append_kernel<F32, 4>, grid, 256, 0, s, p);
    case 6: return launch_pdl(append_kernel<F32, 6>, grid, 256, 0, s, p);
    case 8: return launch_pdl(append_kernel<F32, 8>, grid, 256, 0, s, p);
    default: return KQ_ERR_UNSUPPORTED;
    }
}

}  // namespace

int launch_kv_plan(const int32_t* cached_lens, const int32_t* new_lens, int64_t n_seqs, int page_size,
                   int32_t* block_table, int64_t max_blocks, const int32_t* free_pages, int64_t n_free,
                   const int32_t* taken, int32_t* taken_out, int32_t* seq_lens, int32_t* cu_new, int32_t* first_page,
                   int32_t* slot_map, int32_t* positions, int64_t cap, int32_t* err_flag, cudaStream_t s) {
    PlanParams p{cached_lens, new_lens, static_cast<int>(n_seqs), page_size, divisor_of(static_cast<uint64_t>(page_size)), block_table, static_cast<int>(max_blocks),
                 free_pages, static_cast<int>(n_free), taken, taken_out, seq_lens, cu_new, first_page, slot_map,
                 positions, static_cast<int>(cap), err_flag};
    const int map = cap <= 4 * kPlanThreads;
    const int rc = launch_pdl(plan_scan_kernel, dim3(1), kPlanThreads, 0, s, p, map);
    if (rc || map) return rc;
    return launch_pdl(plan_map_kernel, dim3(static_cast<unsigned>((cap + 1023) / 1024)), 256, 0, s, p);
}

int launch_kv_append(const void* k, const void* v, int f32, int64_t n_tokens, int64_t k_stride, int64_t v_stride,
                     int n_heads, int head_dim, const int32_t* slot_map, void* k_pool, void* v_pool, int64_t n_pages,
                     int page_size, int32_t* err_flag, cudaStream_t s) {
    AppendParams p{{k, v}, {static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool)}, {k_stride, v_stride},
                   slot_map, static_cast<int>(n_tokens * n_heads * (head_dim / 32)), static_cast<int>(n_pages * page_size), n_heads,
                   page_size, divisor_of(static_cast<uint64_t>(n_heads)), divisor_of(static_cast<uint64_t>(page_size)), err_flag};
    return f32 ? append_of<true>(p, head_dim / 32, s) : append_of<false>(p, head_dim / 32, s);
}

}  // namespace kq
