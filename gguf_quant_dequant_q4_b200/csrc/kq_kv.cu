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
// kq_kv_append writes each 32-value block as d = -m / 8 (m the value of
// largest magnitude, the first of equals) and codes trunc(x * (1/d) + 8.5) in
// 0..15, every step a separately rounded fp32 operation.
#include "kq_kv.cuh"

namespace kq {
namespace {

constexpr int kPlanThreads = 1024;

struct PlanParams {
    const int32_t* cached;
    const int32_t* fresh;       // new tokens per request
    int n_seqs;
    int page;
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
__device__ __forceinline__ void plan_token(const PlanParams& p, const int32_t* cu, int total, int t, int& bad) {
    int slot = -1, pos = -1;
    if (t < total) {
        int lo = 0, hi = p.n_seqs - 1;
        while (lo < hi) {   // first b with cu[b + 1] > t
            const int mid = (lo + hi) >> 1;
            if (cu[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        const int c0 = cu[lo], c1 = cu[lo + 1];
        const int old = p.seq_lens[lo] - (c1 - c0);
        pos = old + (t - c0);
        const int j = pos / p.page, off = pos - j * p.page;
        const int held = (old + p.page - 1) / p.page;
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
            int blocks = (seq + p.page - 1) / p.page, held = (old + p.page - 1) / p.page;
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
        for (int t = tid; t < p.cap; t += kPlanThreads) plan_token(p, p.cu, total, t, bad);
    }
    if (bad && p.err) atomicOr(p.err, bad);
}

__global__ void __launch_bounds__(256) plan_map_kernel(const PlanParams p) {
    pdl_launch();
    pdl_wait();
    const int t = blockIdx.x * 256 + threadIdx.x;
    int bad = 0;
    if (t < p.cap) plan_token(p, p.cu, p.cu[p.n_seqs], t, bad);
    if (bad && p.err) atomicOr(p.err, bad);
}

// ------------------------------------------------------------------ append
struct AppendParams {
    const void* src[2];        // k, v
    uint8_t* pool[2];
    int64_t stride[2];         // elements between tokens
    const int32_t* slots;
    int64_t n_blocks;          // tokens * heads * blocks of a row
    int64_t n_slots;
    int n_heads;
    int page;
    int32_t* err;
};

// Four lanes a block of 32 values, eight consecutive values a lane; the
// values' codes meet their partner 16 values on through one exchange with the
// lane two away, after which every lane stores four of the block's 16 bytes.
template <bool F32, int NB>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    pdl_launch();
    pdl_wait();
    const bool values = blockIdx.y != 0;   // keys or values
    const void* src = values ? p.src[1] : p.src[0];
    const int64_t stride = values ? p.stride[1] : p.stride[0];
    const int lane = threadIdx.x & 31, part = lane & 3;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 2;   // block
    const bool in = i < p.n_blocks;
    const int64_t row = (in ? i : 0) / NB;
    const int blk = static_cast<int>((in ? i : 0) - row * NB);
    const int64_t tok = row / p.n_heads;
    const int head = static_cast<int>(row - tok * p.n_heads);
    const int slot = p.slots[tok];
    int bad = 0;
    const bool put = in && slot >= 0 && slot < p.n_slots;
    if (in && !put && slot != -1) bad = KQ_DEV_BAD_RANGE;
    float x[8];
    const int64_t at = tok * stride + (static_cast<int64_t>(head) * NB + blk) * 32 + 8 * part;
    if constexpr (F32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(src) + at);
        const uint4 a = ldg_nc_v4(s), b = ldg_nc_v4(s + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
    } else {
        const uint4 a = ldg_nc_v4(static_cast<const uint16_t*>(src) + at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = bf16lo_to_f32(w[k]);
            x[2 * k + 1] = bf16hi_to_f32(w[k]);
        }
    }
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
    const __half h = __float2half_rn(d);
    const uint32_t hb = __half_as_ushort(h);
    if (put && (hb & 0x7c00u) == 0x7c00u) bad |= KQ_DEV_X_RANGE;
    const float inv = (hb & 0x7fffu) == 0 ? 0.f : __frcp_rn(d);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float f = __fadd_rn(__fmul_rn(x[k], inv), 8.5f);
        const int q = static_cast<int>(fminf(fmaxf(f, 0.f), 15.f));   // truncates
        c[k >> 2] |= static_cast<uint32_t>(q) << (8 * (k & 3));
    }
    const bool upper = part >= 2;   // values 16..31: the high nibbles
    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? c[0] : c[1], 2);
    const uint32_t bytes = upper ? (got | (c[1] << 4)) : (c[0] | (got << 4));
    if (put) {
        const int64_t pg = slot / p.page;
        const int off = slot - static_cast<int>(pg) * p.page;
        uint8_t* dst = (values ? p.pool[1] : p.pool[0]) + (((pg * p.n_heads + head) * p.page + off) * NB + blk) * 18;
        // lanes 0, 1 hold bytes 0..3 and 8..11, lanes 2, 3 bytes 4..7 and 12..15
        uint16_t* o = reinterpret_cast<uint16_t*>(dst + 2 + 8 * (part & 1) + (upper ? 4 : 0));
        o[0] = static_cast<uint16_t>(bytes);
        o[1] = static_cast<uint16_t>(bytes >> 16);
        if (part == 0) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(hb);
    }
    if (bad && p.err) atomicOr(p.err, bad);
}

template <bool F32>
int append_of(const AppendParams& p, int nb, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.n_blocks + 63) / 64), 2);
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
    PlanParams p{cached_lens, new_lens, static_cast<int>(n_seqs), page_size, block_table, static_cast<int>(max_blocks),
                 free_pages, static_cast<int>(n_free), taken, taken_out, seq_lens, cu_new, first_page, slot_map,
                 positions, static_cast<int>(cap), err_flag};
    const int map = cap <= 4 * kPlanThreads;
    const int rc = launch_pdl(plan_scan_kernel, dim3(1), kPlanThreads, 0, s, p, map);
    if (rc || map) return rc;
    return launch_pdl(plan_map_kernel, dim3(static_cast<unsigned>((cap + 255) / 256)), 256, 0, s, p);
}

int launch_kv_append(const void* k, const void* v, int f32, int64_t n_tokens, int64_t k_stride, int64_t v_stride,
                     int n_heads, int head_dim, const int32_t* slot_map, void* k_pool, void* v_pool, int64_t n_pages,
                     int page_size, int32_t* err_flag, cudaStream_t s) {
    AppendParams p{{k, v}, {static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool)}, {k_stride, v_stride},
                   slot_map, n_tokens * n_heads * (head_dim / 32), n_pages * page_size, n_heads, page_size, err_flag};
    return f32 ? append_of<true>(p, head_dim / 32, s) : append_of<false>(p, head_dim / 32, s);
}

}  // namespace kq
