// kq_kv_attention over a paged q4_0 cache, for steps of few tokens a sequence
// (and every step whose head size the prompt kernel does not cover).
//
// One pass over the keys with a running maximum and sum: for the rows (token,
// query head) that share one key head,
//   o = sum_j 2^(y_j - m) v_j / sum_j 2^(y_j - m),  y_j = log2(e) scale q.k_j.
// The wire blocks are never expanded to values.  The tensor cores take the
// 4-bit codes as binary16 subnormals (mma.sync keeps subnormal operands
// exact), keys as the rows of the A operand:
//   S[key, row]  = sum over blocks of d(key, block) * ((code - 8) . q): two
//                  AND-masks turn four packed codes into two operand words, the
//                  high ones 16 times too large, against q / 16; the -8 is the
//                  accumulator's start, -8 * sum of the block's q
//   O[dim, row] += code[dim, key] * (P d)[key, row]: the low codes, and whole
//                  bytes (low + 16 high), from which the low sums come off at
//                  the end, as does 8 sum P d
// q is scaled by a power of two per row (as every decode kernel of this
// library), so only P and P * d are rounded, to binary16.  P is relative to a
// reference 5 below the row's maximum, which moves only when the maximum is more
// than 13 above it; d is in units of a power of two near the tile's largest, and
// scales 2^10 times smaller get a pass of their own.  So P is off by at most
// 2^-11 of itself or 2^-30 of the row's largest weight, and P * d by 2^-11 of
// itself or 2^-20 of the largest weight times d.  Maximum, sum and all accumulators are fp32.
//
// Work is cut by keys, not by sequences: the tiles of 32 keys of all
// (sequence, key head, 8 or 16 rows) segments form one list, and every CTA of
// a grid that fills the GPU once takes an equal run of it, whatever the
// lengths (found on the device from the lengths; the host reads nothing).  In
// a CTA one warp reads the block table and issues bulk copies of 16- or
// 32-key runs into a ring of stages; the other warps take the tiles in turn,
// each with a maximum, sum and accumulator of its own, joined in shared memory
// at the end of a segment.  A segment that spans CTAs leaves fp32 partial
// results in the work space, joined in list order by a second kernel: no
// atomics on data, the same result on every run.
//
// Bound by latency at the few warps that the registers leave (3.7 a scheduler:
// 57 % of the issue slots, 48 % of the ALU pipe, 44 % of DRAM's peak), and with
// short segments by their starts and joins.  Kernels alone: one sequence of 700
// keys, 32 heads over 8 of 128: 13.9 us; 24 of up to 4100 keys, 16 over 16 of
// 64: 33; 16 of up to 6000 with 3 to 5 tokens each and a window, 16 over 4 of
// 256: 39; 48 of up to 8192, 32 over 8 of 128: 69 (3.3 TB/s); 2 of 150,000 to
// 200,000, 64 over 8 of 128: 98 (4.1 TB/s; 103 after seconds at the power cap).
// What the steps were worth on the last of these: work split by keys 143 us;
// four producer lanes a tile, value scales through a table 117; q in shared
// memory, in-place rescaling, whole bytes 100; segments' fixed cost in the
// split 96 (and 87 -> 67 on the ragged batch); scores and value scales of any
// size 98 (and 69).  Fetching by the consumer warps
// themselves instead of a producer: 115, more warps at fewer registers: 117 to
// 133, -8 by exact subtraction from every operand: 117.
#include "kq_kv.cuh"

namespace kq {
namespace {

constexpr int kTile = 32;        // keys of a tile
// A segment counts as its tiles and kSegCost more in the list: its queries,
// first copies and join take about as long as that many tiles.  A CTA whose
// part of a segment is within these has nothing to do there.  (Ragged batch of
// 48 sequences up to 8192 keys, heads of 128: 87 us without, 70 with 12, 68 with
// 20, 70 with 28, 78 with 60; chosen on this batch, the other shapes take the
// same.)
constexpr int kSegCost = 20;
constexpr int kMinShare = kSegCost + 7;   // least units of a CTA's share: a tile a warp
// A row's reference is 5 below its maximum when it moves, which it does when the
// maximum is more than 13 above it: P, 2^(score - reference), stays within 2^13,
// P * d below 2^15.
constexpr float kPBias = 5.f, kLazy = 8.f;
// A tile's value scales are taken in units 2^ve near their largest: ve moves
// when the largest is 2^2 and more times it, or below 2^-kDrop of it.  Scales
// below 2^-kBelow of the unit get a pass of their own, so that binary16's last
// step, 2^-24, is at most 2^-19 of the largest P (2^5 at least) times the scale.
constexpr int kDrop = 3, kBelow = 10;

// A sequence's share of the work.
struct Seq {
    int tok0, qlen, pos0, len;   // first token, tokens, its position, keys
    int lo;                      // first key any row sees
    int t0, nt;                  // first tile, tiles of a segment
    int rt;                      // row tiles
};

template <int R>
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int b) {
    const Given in = given_of(p, b);
    Seq s;
    s.tok0 = in.tok0;
    s.qlen = in.qlen;
    s.pos0 = in.pos0;
    s.len = in.len;
    int lo = 0;
    if (p.window > 0) {
        lo = s.pos0 - p.window + 1;
        lo = lo < 0 ? 0 : (lo > s.len ? s.len : lo);
    }
    s.lo = lo;
    s.t0 = lo / kTile;
    const int nt = (s.len + kTile - 1) / kTile - s.t0;
    s.nt = nt < 1 ? 1 : nt;      // a segment without keys still writes its zeros
    const int rows = s.qlen * p.group;
    s.rt = rows > p.few ? 0 : (rows + R - 1) / R;   // (more rows: the prompt kernel's)
    return s;
}
__device__ __forceinline__ int64_t units_of(const AttnParams& p, const Seq& s) {
    return static_cast<int64_t>(s.nt + kSegCost) * s.rt * p.n_kv;
}

// A place in the list: sequence, key head, row tile and unit of the segment.
struct Place {
    int b, h, rt, unit;
    int64_t left;                // units of the CTA's share from here on
};
// The share's part of the segment at a place: units, and tiles [t0, t0 + n).
struct Part {
    int units, t0, n;
};
__device__ __forceinline__ Part part_of(const Place& at, const Seq& s) {
    const int seg = s.nt + kSegCost;
    Part r;
    r.units = static_cast<int>(at.left < seg - at.unit ? at.left : seg - at.unit);
    r.t0 = at.unit > kSegCost ? at.unit - kSegCost : 0;
    const int end = at.unit + r.units - kSegCost;
    r.n = end > r.t0 ? end - r.t0 : 0;
    return r;
}

// Length of the list, by all threads of the CTA.
template <int R>
__device__ __forceinline__ int64_t list_total(const AttnParams& p, unsigned long long* sum) {
    if (threadIdx.x == 0) *sum = 0;
    __syncthreads();
    int64_t mine = 0;
    for (int b = threadIdx.x; b < p.n_seqs; b += blockDim.x) mine += units_of(p, seq_of<R>(p, b));
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((threadIdx.x & 31) == 0 && mine) atomicAdd(sum, static_cast<unsigned long long>(mine));
    __syncthreads();
    return static_cast<int64_t>(*sum);
}
// One warp: the sequence that holds unit u and the units before it.
template <int R>
__device__ __forceinline__ int list_find(const AttnParams& p, int64_t u, int64_t& before) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        const int64_t n = b < p.n_seqs ? units_of(p, seq_of<R>(p, b)) : 0;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const unsigned over = __ballot_sync(0xffffffffu, base + inc > u);
        if (over) {
            const int l = __ffs(over) - 1;
            before = base + __shfl_sync(0xffffffffu, inc - n, l);
            return b0 + l;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    before = base;
    return p.n_seqs;
}
__device__ __forceinline__ int64_t share_of(int64_t total, int n_ctas) {
    const int64_t s = (total + n_ctas - 1) / n_ctas;
    return s < kMinShare ? kMinShare : s;
}

// Exponent of the value scale 2^ve that brings a binary16 magnitude (8188 at
// most) to [1, 2), below 1 from subnormals.
__device__ __forceinline__ int exponent_of(uint32_t mag) {
    const int e = static_cast<int>(mag >> 10) - 15;
    return e < -14 ? -14 : e;
}
// 2^e as binary16 bits; 0 below its smallest.
__device__ __forceinline__ uint32_t bits_of_exp2(int e) {
    return e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : (e >= -24 ? 1u << (e + 24) : 0u);
}

// x *= f in its own register (a rarely taken branch must not rename what the
// other path would have to copy).
__device__ __forceinline__ void mul_in_place(float& x, float f) { asm volatile("mul.f32 %0, %0, %1;" : "+f"(x) : "f"(f)); }
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts_u16(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(v)) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

template <int NB, int NT>
struct Shape {
    static constexpr int D = 32 * NB;
    static constexpr int R = 8 * NT;                   // rows of a segment
    static constexpr int RB = 18 * NB;                 // bytes of a row
    static constexpr int kStage = 2 * kTile * RB;      // keys, then values
    static constexpr bool two = NB * NT <= 4;          // two CTAs an SM
    static constexpr int kWarps = two ? 7 : NB * NT <= 8 ? 11 : 7;   // consumer warps (and one producer)
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int DP = D + 4;                   // joined rows, padded (bank conflicts)
    static constexpr int kJoin = 3 * R * DP * 4;       // three buffers of fp32 rows
    static constexpr int kScale = 64 * NB;             // a warp's value scales of a tile, in operand order
    static constexpr int kQ = NT * NB * 512;            // q as operand words, a 16-byte quad a lane
    static constexpr int kStart = NT * NB * 64;         // the accumulators' start, a quad for every t
    static constexpr int kRow = 3 * R * 4;              // of every row: y scale, last and first key seen
    static constexpr int kHead = 1024 + 2 * kWarps * R * 4 + kWarps * kScale + kQ + kStart + kRow;
    static constexpr int kBudget = (two ? 113 : 226) * 1024;
    static constexpr int kFit = (kBudget - kHead - kJoin) / kStage;
    // A stage belongs to one consumer warp (NST a multiple of their number):
    // were it shared, a warp could wait for a stage's next use before the use
    // before it has landed (copies land in any order), and take that phase's
    // parity for its own.
    static constexpr int NST = (kFit > 32 ? 32 : kFit) / kWarps * kWarps;
    static constexpr int kSmem = kHead + kJoin + NST * kStage;
    static constexpr int kSlot = R * D + 2 * R;        // floats of a partial result
};

template <int NB, int NT>
__global__ void __launch_bounds__(Shape<NB, NT>::kThreads, Shape<NB, NT>::two ? 2 : 1) attn_kernel(const AttnParams p) {
    using C = Shape<NB, NT>;
    constexpr int R = C::R, RB = C::RB, NST = C::NST, D = C::D, kWarps = C::kWarps;
    static_assert(NST >= kWarps && NST % kWarps == 0, "stages of its own for every consumer warp");
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + 32;
    uint32_t* vmask = reinterpret_cast<uint32_t*>(smem + 512);   // keys of the stage that are there
    volatile int* abort_ = reinterpret_cast<volatile int*>(smem + 640);
    unsigned long long* sum = reinterpret_cast<unsigned long long*>(smem + 648);
    Place* place = reinterpret_cast<Place*>(smem + 656);
    float* wm = reinterpret_cast<float*>(smem + 1024);   // [warp][R] maximum
    float* wl = wm + kWarps * R;                         // [warp][R] sum
    const uint32_t scales = smem_u32(smem) + 1024 + 2 * kWarps * R * 4 + (threadIdx.x >> 5) * C::kScale;
    uint8_t* qmem = smem + 1024 + 2 * kWarps * R * 4 + kWarps * C::kScale;
    const uint32_t qtab = smem_u32(qmem) + 16 * (threadIdx.x & 31), ctab = smem_u32(qmem) + C::kQ;
    float* yrow = reinterpret_cast<float*>(qmem + C::kQ + C::kStart);
    int* hirow = reinterpret_cast<int*>(yrow + R);
    int* lorow = hirow + R;
    float* join = reinterpret_cast<float*>(smem + C::kHead);
    const uint32_t ring = smem_u32(smem) + C::kHead + C::kJoin;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        *abort_ = 0;
        fence_barrier_init();
    }
    pdl_launch();
    pdl_wait();
    const int64_t total = list_total<R>(p, sum);
    if (blockIdx.x == 0 && p.err) {   // (for the prompt kernel's sequences too)
        int bad = 0;
        for (int b = tid; b < p.n_seqs; b += C::kThreads) bad |= given_of(p, b).bad;
        if (bad) atomicOr(p.err, bad);
    }
    const int64_t share = share_of(total, p.n_ctas);
    const int64_t u0 = share * blockIdx.x;
    if (u0 >= total) return;
    if (warp == 0) {
        int64_t before;
        const int b = list_find<R>(p, u0, before);
        const Seq s = seq_of<R>(p, b);
        const int64_t off = u0 - before, seg = off / (s.nt + kSegCost);
        if (lane == 0) {
            place->b = b;
            place->h = static_cast<int>(seg / s.rt);
            place->rt = static_cast<int>(seg % s.rt);
            place->unit = static_cast<int>(off - seg * (s.nt + kSegCost));
            place->left = total - u0 < share ? total - u0 : share;
        }
    }
    __syncthreads();
    Place at = *place;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_) return false;
        if (!mbar_wait(bar, parity, p.status)) {
            *abort_ = 1;
            return false;
        }
        return true;
    };
    // next segment of the list
    auto advance = [&](Seq& s) {
        at.unit = 0;
        if (++at.rt == s.rt) {
            at.rt = 0;
            if (++at.h == p.n_kv) {
                at.h = 0;
                do {
                    ++at.b;
                    s = seq_of<R>(p, at.b);
                } while (s.rt == 0);
            }
        }
    };

    if (warp == kWarps) {
        // ------------------------------------------------ producer
        // Four lanes a tile (keys or values, first or second 16 keys), BT tiles
        // at a time: their table entries, waits and copies overlap.
        constexpr int BT = NST >= 16 ? 8 : 4;
        uint32_t n = 0, phase = 0;   // next stage, its phase
        const int64_t page_bytes = static_cast<int64_t>(p.n_kv) * p.page * RB;
        const int q = lane >> 2, kv = lane & 1, sl = (lane >> 1) & 1;
        Seq s = seq_of<R>(p, at.b);
        while (at.left > 0) {
            const Part part = part_of(at, s);
            const int tiles = part.n, tile0 = s.t0 + part.t0;
            const uint8_t* src = (kv ? p.vp : p.kp) + static_cast<int64_t>(at.h) * p.page * RB;
            const int32_t* row = p.table + static_cast<int64_t>(at.b) * p.max_blocks;
            // page of this lane's keys of tile i; -1: no visible key, -2: no such page
            int rem = 0, page = -1;
            auto look = [&](int i) {
                const int key = (tile0 + i) * kTile + 16 * sl;
                page = -1;
                if (q < BT && i < tiles && key < s.len && key + 16 > s.lo) {
                    const int blk = page_of(p, key);
                    rem = key - blk * p.page;
                    page = row[blk];
                    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages)) page = -2;
                }
            };
            look(q);
            for (int i0 = 0; i0 < tiles; i0 += BT) {
                const int pg = page, i = i0 + q;
                const uint8_t* from = src + pg * page_bytes + rem * RB;
                const bool run = sl ? rem >= 16 : rem + 32 <= p.page;   // the tile's keys are one run
                look(i + BT);
                if (pg == -2 && kv == 0 && p.err) atomicOr(p.err, KQ_DEV_BAD_RANGE);
                const unsigned in = (__ballot_sync(0xffffffffu, pg >= 0) >> (lane & 28)) & 15u;
                uint32_t st = n + q;
                uint32_t par = phase ^ 1;
                if (st >= NST) {
                    st -= NST;
                    par ^= 1;
                }
                bool ok = q < BT && i < tiles;
                if (ok && (lane & 3) == 0) {
                    ok = wait(&empty[st], par);
                    if (ok) {
                        vmask[st] = ((in & 1u) ? 0xffffu : 0u) | ((in & 4u) ? 0xffff0000u : 0u);
                        mbar_arrive_expect_tx(&full[st], __popc(in) * 16 * RB);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, lane & 28);
                const bool both = in == 15u && run;
                if (ok && pg >= 0 && !(both && sl)) {
                    uint8_t* d = smem + C::kHead + C::kJoin + st * C::kStage + (kv * kTile + sl * 16) * RB;
                    bulk_g2s(d, from, both ? 32 * RB : 16 * RB, &full[st]);
                }
                n += tiles - i0 < BT ? tiles - i0 : BT;
                if (n >= NST) {
                    n -= NST;
                    phase ^= 1;
                }
            }
            at.left -= part.units;
            if (at.left > 0) advance(s);
        }
        if (*abort_) {
            // let copies in flight land before the CTA's shared memory goes
            const uint64_t t0 = global_ns();
            while (global_ns() - t0 < 2000000ull) __nanosleep(10000);
        }
        return;
    }

    // -------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    // key of row r of the j-th 16 of a tile: strides that keep the eight rows
    // of a load on different banks
    auto tau = [](int j, int r) {
        const int gg = r & 7, up = r >> 3;
        if (NB == 4) return 16 * j + 2 * gg + up;
        if (NB == 8) return 16 * j + r;
        return 4 * gg + 2 * j + up;
    };
    // where key `lane` has its value scale: rows 2t', 2t' + 1, 2t' + 8, 2t' + 9
    // of both 16s are the eight halves of t'
    uint32_t scale_at = scales;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (tau(j, r) == lane) scale_at += 16 * ((r & 7) >> 1) + 8 * j + 4 * (r >> 3) + 2 * (r & 1);
    int first = warp;            // this warp's first tile of the segment
    uint32_t stage = warp, phase = 0;
    Seq s = seq_of<R>(p, at.b);
    int slot = 0;                // partial slot: 0 while in the share's first segment
    Part pt{};
    // the next part of the share that has tiles
    auto settle = [&]() {
        while (at.left > 0) {
            pt = part_of(at, s);
            if (pt.n > 0) return true;
            at.left -= pt.units;
            slot = 1;
            if (at.left > 0) advance(s);
        }
        return false;
    };
    // q of the segment as operand words, and the accumulators' start, 8 rows a warp
    auto prepare = [&]() {
        if (warp < NT) {
            const int nt = warp, rows = s.qlen * p.group - at.rt * R;
            const int r = nt * 8 + g;
            const int rr = at.rt * R + r, i = rr / p.group;
            const bool there = r < rows;
            const uint16_t* src = p.q + (s.tok0 + (there ? i : 0)) * p.q_stride +
                                  static_cast<int64_t>(at.h * p.group + (there ? rr - i * p.group : 0)) * D;
            uint2 w[NB][2];      // values of byte j's low nibble, high nibble (bf16)
            uint32_t mx = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // the bytes of this lane's word: even blocks 4t+2..4t+5 and (t = 3) 0, 1, 14, 15;
                // odd blocks 4t..4t+3
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint16_t* a = src + 32 * b + 16 * hf;
                    if (b & 1) {
                        w[b][hf] = *reinterpret_cast<const uint2*>(a + 4 * t);
                    } else {
                        w[b][hf].x = *reinterpret_cast<const uint32_t*>(a + (t == 3 ? 0 : 4 * t + 2));
                        w[b][hf].y = *reinterpret_cast<const uint32_t*>(a + (t == 3 ? 14 : 4 * t + 4));
                    }
                    if (!there) w[b][hf] = make_uint2(0, 0);
                    mx = __vmaxu2(mx, __vmaxu2(w[b][hf].x & 0x7fff7fffu, w[b][hf].y & 0x7fff7fffu));
                }
            }
            mx = max(mx & 0xffffu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (mx >= 0x7f80u && p.err) atomicOr(p.err, KQ_DEV_X_RANGE);
            const int e = xscale_exp(mx, 13);
            // the scale's sign goes into q, so that yscale > 0; scale 0: q = 0
            const float up = p.scale == 0.f ? 0.f : copysignf(exp2_int(e), p.scale);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float v[8];      // lo of bytes 0..3, hi of bytes 0..3
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    v[4 * hf] = bf16lo_to_f32(w[b][hf].x) * up;
                    v[4 * hf + 1] = bf16hi_to_f32(w[b][hf].x) * up;
                    v[4 * hf + 2] = bf16lo_to_f32(w[b][hf].y) * up;
                    v[4 * hf + 3] = bf16hi_to_f32(w[b][hf].y) * up;
                }
                // high nibbles enter the MMA as 16 * code
                const uint32_t w4[4] = {pack_f16x2(v[0], v[2]), pack_f16x2(v[4] * 0.0625f, v[6] * 0.0625f),
                                        pack_f16x2(v[1], v[3]), pack_f16x2(v[5] * 0.0625f, v[7] * 0.0625f)};
                *reinterpret_cast<uint4*>(qmem + (nt * NB + b) * 512 + 16 * lane) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                float a = 0.f;   // of the rounded operands
#pragma unroll
                for (int k = 0; k < 4; ++k) a += (f16lo_to_f32(w4[k]) + f16hi_to_f32(w4[k])) * (k & 1 ? 16.f : 1.f);
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                a *= -8.f / 16777216.f;
                // row g is column g & 1 of t = g / 2, in both of its rows
                if (t == 0) {
                    float* st = reinterpret_cast<float*>(qmem + C::kQ + (nt * NB + b) * 64 + 16 * (g >> 1)) + (g & 1);
                    st[0] = a;
                    st[2] = a;
                }
            }
            if (t == 0) {
                yrow[r] = factor_of(p.scale, e, 24);   // (codes enter as 2^-24)
                const int pos = s.pos0 + i;
                hirow[r] = p.causal ? min(pos, s.len - 1) : s.len - 1;
                lorow[r] = p.window > 0 ? pos - p.window + 1 : 0;
            }
        }
    };
    bool go = settle();
    if (go) prepare();
    bar_sync(1, 32 * kWarps);
    while (go) {
        const int tiles = pt.n, tile0 = s.t0 + pt.t0;
        const bool whole = tiles == s.nt;
        const int rows = s.qlen * p.group - at.rt * R;   // rows of this tile that exist (may exceed R)
        float yscale[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            yscale[nt][0] = yrow[nt * 8 + 2 * t];
            yscale[nt][1] = yrow[nt * 8 + 2 * t + 1];
        }
        // keys that every row of the segment sees
        const int pos0 = s.pos0 + (at.rt * R) / p.group;
        const int last_row = min(at.rt * R + R, s.qlen * p.group) - 1;
        const int pos1 = s.pos0 + last_row / p.group;
        const int all_hi = p.causal ? min(pos0, s.len - 1) : s.len - 1;
        const int all_lo = p.window > 0 ? pos1 - p.window + 1 : 0;

        float o[2 * NB][NT][4];
        float pd[NT][NB];        // this lane's part of sum P d of row g
        float m[NT][2], l[NT][2];
        int ve = -14;            // exponent of the value scale
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) pd[nt][b] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }

        // this warp's tiles: list positions n with n % kWarps == warp
        int i = first;
        for (; i < tiles; i += kWarps) {
            const uint32_t st = stage;
            const bool ok = __all_sync(0xffffffffu, wait(&full[st], phase));
            stage += kWarps;
            if (stage >= NST) {
                stage -= NST;
                phase ^= 1;
            }
            if (!ok) continue;
            const uint32_t kb = ring + st * C::kStage, vb = kb + kTile * RB;
            const int key0 = (tile0 + i) * kTile;
            const uint32_t there = vmask[st];
            // ---- S
            float y[2][NT][4];
#pragma unroll
            for (int bp = 0; bp < NB / 2; ++bp) {
                uint4 qw[2][NT];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) qw[hf][nt] = lds128(qtab + (nt * NB + 2 * bp + hf) * 512);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t cw[2][2];   // [block of the pair][row]
                    float d[2][2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t a = kb + tau(j, g + 8 * r) * RB + 36 * bp;
                        const uint32_t w0 = lds32(a), w4 = lds32(a + 16), wx = lds32(a + 4 + 4 * t);
                        cw[1][r] = lds32(a + 20 + 4 * t);
                        cw[0][r] = __byte_perm(w0, wx, t == 3 ? 0x5432 : 0x7654);
                        d[0][r] = f16lo_to_f32(w0);
                        d[1][r] = f16hi_to_f32(w4);
                    }
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int b = 2 * bp + hf;
                        const uint32_t c0 = cw[hf][0], c1 = cw[hf][1];
                        const uint32_t e0 = c0 >> 8, e1 = c1 >> 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 st4 = lds128(ctab + (nt * NB + b) * 64 + 16 * t);
                            float acc[4] = {__uint_as_float(st4.x), __uint_as_float(st4.y), __uint_as_float(st4.z),
                                            __uint_as_float(st4.w)};
                            mma_f16(acc, c0 & 0x000f000fu, c1 & 0x000f000fu, c0 & 0x00f000f0u, c1 & 0x00f000f0u,
                                    qw[hf][nt].x, qw[hf][nt].y);
                            mma_f16(acc, e0 & 0x000f000fu, e1 & 0x000f000fu, e0 & 0x00f000f0u, e1 & 0x00f000f0u,
                                    qw[hf][nt].z, qw[hf][nt].w);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[j][nt][k] = b == 0 ? d[hf][k >> 1] * acc[k] : fmaf(d[hf][k >> 1], acc[k], y[j][nt][k]);
                        }
                    }
                }
            }
            // base-2 scores, rounded before the reference comes off them: were the
            // exact product inside one FMA with a rounded reference, the largest
            // P would be off by a power of two once scores pass 2^24 or so
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[j][nt][k] = __fmul_rn(y[j][nt][k], yscale[nt][k & 1]);
            const bool edge = there != 0xffffffffu || key0 + kTile - 1 > all_hi || key0 < all_lo;
            if (edge) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tk = tau(j, g + 8 * (k >> 1)), key = key0 + tk;
                            const int r = nt * 8 + 2 * t + (k & 1);
                            const bool ok = key <= hirow[r] && key >= lorow[r] && ((there >> tk) & 1u);
                            if (!ok) y[j][nt][k] = -INFINITY;
                        }
            }
            // ---- value scales, lane = key; a key that no row sees has 0
            uint32_t dv[NB];
            uint32_t dm = 0, km = 0;   // largest of the key's value and key scales
            {
#pragma unroll
                for (int b = 0; b < NB; ++b) dv[b] = lds_u16(vb + lane * RB + 18 * b);
#pragma unroll
                for (int b = 0; b < NB; ++b) km = max(km, lds_u16(kb + lane * RB + 18 * b) & 0x7fffu);
                if (edge) {
                    const int key = key0 + lane;
                    const bool seen = key < s.len && key >= s.lo && ((there >> lane) & 1u);
#pragma unroll
                    for (int b = 0; b < NB; ++b) dv[b] = seen ? dv[b] : 0;
                    km = seen ? km : 0;
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) dm = max(dm, dv[b] & 0x7fffu);
            }
            // a scale past 8188: the rows that see its key are not numbers (the
            // prompt kernel's rule, whose binary16 values end there)
            const unsigned who = __ballot_sync(0xffffffffu, max(dm, km) > 0x6fffu);
            if (who) {
                if ((who >> lane) & 1u) {
                    dm = 0;
#pragma unroll
                    for (int b = 0; b < NB; ++b) dv[b] = 0;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tk = tau(j, g + 8 * (k >> 1)), key = key0 + tk;
                            const int r = nt * 8 + 2 * t + (k & 1);
                            if ((who >> tk) & 1u) {
                                if (key <= hirow[r] && key >= lorow[r]) l[nt][k & 1] = __int_as_float(0x7fc00000);
                                y[j][nt][k] = -INFINITY;
                            }
                        }
            }
            const uint32_t dmx = __reduce_max_sync(0xffffffffu, dm);
            // ---- reference (kPBias below a maximum), value exponent
            int ne = exponent_of(dmx);
            if (ne <= ve && (ne >= ve - kDrop || dmx == 0)) ne = ve;
            bool grow = ne > ve + 1 || ne < ve;
            float mt[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = fmaxf(fmaxf(y[0][nt][c], y[0][nt][c + 2]), fmaxf(y[1][nt][c], y[1][nt][c + 2]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mt[nt][c] = fmaxf(m[nt][c], v - kPBias);
                    grow |= v - m[nt][c] > kPBias + kLazy;   // (a difference of near values is exact)
                }
            if (__any_sync(0xffffffffu, grow)) {
                const float fe = exp2_int(ve - ne);
                ve = ne;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        f[c] = m[nt][c] == mt[nt][c] ? 1.f : ex2(m[nt][c] - mt[nt][c]);
                        m[nt][c] = mt[nt][c];
                        mul_in_place(l[nt][c], f[c]);
                        f[c] *= fe;
#pragma unroll
                        for (int k = 0; k < 2 * NB; ++k) {
                            mul_in_place(o[k][nt][c], f[c]);
                            mul_in_place(o[k][nt][c + 2], f[c]);
                        }
                    }
                    // row g is column g & 1 of t = g / 2
                    const float fa = __shfl_sync(0xffffffffu, f[0], g >> 1), fb = __shfl_sync(0xffffffffu, f[1], g >> 1);
#pragma unroll
                    for (int b = 0; b < NB; ++b) mul_in_place(pd[nt][b], (g & 1) ? fb : fa);
                }
            }
            // ---- P (binary16), transposed into B operand words
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float mm[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) mm[c] = m[nt][c] == -INFINITY ? 0.f : m[nt][c];   // (all hidden: 2^-inf)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e[k] = ex2(y[j][nt][k] - mm[k & 1]);
                        l[nt][k & 1] += e[k];
                    }
                    pb[j][nt][0] = movm(pack_f16x2(e[0], e[1]));
                    pb[j][nt][1] = movm(pack_f16x2(e[2], e[3]));
                }
            }
            // ---- O, in passes over the scales' magnitudes: 2^ve times 2^-kBelow and
            // more, then what is smaller in units of its own (rare)
            uint32_t cut;
#pragma unroll 1
            for (;;) {
                const uint32_t vs = static_cast<uint32_t>((15 - ve) << 10) * 0x10001u;   // 2^-ve
                uint32_t two[NB / 2];
                bool small = false;
#pragma unroll
                for (int b = 0; b < NB; b += 2) {
                    two[b / 2] = hmul2_u32(dv[b] | (dv[b + 1] << 16), vs);
                    small |= !__hbge2(__habs2(*reinterpret_cast<__half2*>(&two[b / 2])), __float2half2_rn(1.f / (1 << kBelow)));
                }
                uint32_t late = 0;   // the largest scale that is left for later
                if (__any_sync(0xffffffffu, small)) {
                    cut = bits_of_exp2(ve - kBelow);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint32_t mag = dv[b] & 0x7fffu;
                        if (mag < cut) {
                            late = max(late, mag);
                            two[b / 2] &= b & 1 ? 0xffffu : 0xffff0000u;
                        }
                    }
                    late = __reduce_max_sync(0xffffffffu, late);
                }
#pragma unroll
                for (int b = 0; b < NB; b += 2) {
                    sts_u16(scale_at + 64 * b, two[b / 2]);
                    sts_u16(scale_at + 64 * b + 64, two[b / 2] >> 16);
                }
                __syncwarp();
                uint4 dq[NB];   // scales of the keys 2t, 2t + 1, 2t + 8, 2t + 9 of both 16s
#pragma unroll
                for (int b = 0; b < NB; ++b) dq[b] = lds128(scales + 64 * b + 16 * t);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t ra = vb + tau(j, 2 * t) * RB, rb = vb + tau(j, 2 * t + 1) * RB;
                    const uint32_t rc = vb + tau(j, 2 * t + 8) * RB, rd = vb + tau(j, 2 * t + 9) * RB;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint32_t c = 18 * b + 2 + 2 * g;
                        const uint32_t xa = lds_u16(ra + c), xb = lds_u16(rb + c), xc = lds_u16(rc + c), xd = lds_u16(rd + c);
                        // whole bytes (low code + 16 * high code) of both keys, and the low codes
                        const uint32_t x0 = __byte_perm(xa, xb, 0x6420), x1 = __byte_perm(xa, xb, 0x6521);
                        const uint32_t z0 = __byte_perm(xc, xd, 0x6420), z1 = __byte_perm(xc, xd, 0x6521);
                        const uint32_t d0 = j ? dq[b].z : dq[b].x, d1 = j ? dq[b].w : dq[b].y;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t b0 = hmul2_u32(pb[j][nt][0], d0), b1 = hmul2_u32(pb[j][nt][1], d1);
                            // rows g, g + 8: dims 2g, 2g + 1 of the block's first (then second) 16
                            mma_f16(o[2 * b][nt], x0 & 0x000f000fu, x1 & 0x000f000fu, z0 & 0x000f000fu, z1 & 0x000f000fu, b0, b1);
                            mma_f16(o[2 * b + 1][nt], x0, x1, z0, z1, b0, b1);
                            pd[nt][b] = add_f16hi(b1, add_f16lo(b1, add_f16hi(b0, add_f16lo(b0, pd[nt][b]))));
                        }
                    }
                }
                __syncwarp();
                if (late == 0) break;
                // (what no row sees may be larger than `late`, and must not overflow)
                const int key = key0 + lane;
                const bool seen = key < s.len && key >= s.lo && ((there & ~who) >> lane) & 1u;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    dv[b] = lds_u16(vb + lane * RB + 18 * b);
                    if (!seen || (dv[b] & 0x7fffu) >= cut) dv[b] = 0;
                }
                const int e = exponent_of(late);
                const float f = exp2_int(ve - e);
                ve = e;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                        for (int c = 0; c < 4; ++c) mul_in_place(o[k][nt][c], f);
#pragma unroll
                    for (int b = 0; b < NB; ++b) mul_in_place(pd[nt][b], f);
                }
            }
            if (lane == 0) mbar_arrive(&empty[st]);
        }

        first = i - tiles;
        // high codes (times 16) out of the bytes, and the codes' offset, 8 sum
        // P d, out of both
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float v = pd[nt][b];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                v *= -8.f / 16777216.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float x = __shfl_sync(0xffffffffu, v, 4 * (2 * t + c));
                    o[2 * b + 1][nt][c] = fmaf(x, 16.f, o[2 * b + 1][nt][c] - o[2 * b][nt][c]);
                    o[2 * b + 1][nt][c + 2] = fmaf(x, 16.f, o[2 * b + 1][nt][c + 2] - o[2 * b][nt][c + 2]);
                    o[2 * b][nt][c] += x;
                    o[2 * b][nt][c + 2] += x;
                }
            }

        // ---- join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[nt][c];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (g == 0) {
                    const int r = nt * 8 + 2 * t + c;
                    wm[warp * R + r] = m[nt][c];
                    wl[warp * R + r] = v;
                }
            }
        bar_sync(1, 32 * kWarps);
        float M[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = nt * 8 + 2 * t + c;
                float v = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v = fmaxf(v, wm[w * R + r]);
                M[nt][c] = v;
                // codes' 2^24, the second 16 dims' 1/16, the value scale
                const float f = m[nt][c] == -INFINITY ? 0.f : ex2(m[nt][c] - v) * 16777216.f * exp2_int(ve);
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) {
                    const float fk = k & 1 ? f * 0.0625f : f;
                    o[k][nt][c] *= fk;
                    o[k][nt][c + 2] *= fk;
                }
            }
        // three warps at a time leave or add theirs
        auto leave = [&](int w, bool add) {
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float2* q2 = reinterpret_cast<float2*>(join + (w * R + nt * 8 + 2 * t + c) * C::DP + 32 * (k >> 1) +
                                                               16 * (k & 1) + 2 * g);
                        const float2 v = add ? *q2 : make_float2(0.f, 0.f);
                        *q2 = make_float2(v.x + o[k][nt][c], v.y + o[k][nt][c + 2]);
                    }
        };
        for (int w = 0; w < kWarps; w += 3) {
            if (warp >= w && warp < w + 3) leave(warp - w, w != 0);
            bar_sync(1, 32 * kWarps);
        }
        // sum of the buffers: the output, or this CTA's partial result
        float* part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * C::kSlot;
        for (int i = tid; i < R * (D / 4); i += 32 * kWarps) {
            const int r = i / (D / 4), c4 = (i % (D / 4)) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(join + (w * R + r) * C::DP + c4);
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            float mx = -INFINITY, sm = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wm[w * R + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)   // (a warp without a maximum has 0, or NaN from a q that is none)
                sm += wm[w * R + r] == -INFINITY ? wl[w * R + r] : wl[w * R + r] * ex2(wm[w * R + r] - mx);
            if (whole) {
                if (r < rows) {
                    const int rr = at.rt * R + r, ti = rr / p.group;
                    const float inv = sm == 0.f ? 0.f : 1.f / sm;
                    uint2 out;
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * inv, v.y * inv);
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v.z * inv, v.w * inv);
                    out.x = *reinterpret_cast<const uint32_t*>(&a);
                    out.y = *reinterpret_cast<const uint32_t*>(&b);
                    const int64_t row = static_cast<int64_t>(s.tok0 + ti) * p.n_heads + at.h * p.group + (rr - ti * p.group);
                    if (sm == 0.f) out = make_uint2(0, 0);   // no key is seen
                    *reinterpret_cast<uint2*>(p.out + row * D + c4) = out;
                }
            } else {
                *reinterpret_cast<float4*>(part + r * D + c4) = v;
                if (c4 == 0) {
                    part[R * D + r] = mx;
                    part[R * D + R + r] = sm;
                }
            }
        }
        at.left -= pt.units;
        slot = 1;
        if (at.left > 0) advance(s);
        go = settle();
        if (go) prepare();
        bar_sync(1, 32 * kWarps);   // join, wm and wl are free again, q is there
    }
}

// Joins the partial results of the segments that span CTAs, in list order: CTA
// i takes the segment that the boundary between shares i - 1 and i cuts, if
// that is the first boundary inside it; blockIdx.y takes 64 of the D values.
template <int NB, int NT>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnParams p) {
    using C = Shape<NB, NT>;
    constexpr int R = C::R, D = C::D;
    __shared__ unsigned long long sum;
    __shared__ int64_t found[2];
    pdl_wait();
    const int64_t total = list_total<R>(p, &sum);
    const int64_t share = share_of(total, p.n_ctas);
    const int64_t u = share * (static_cast<int64_t>(blockIdx.x) + 1);
    if (u >= total) return;
    if (threadIdx.x < 32) {
        int64_t before;
        const int b = list_find<R>(p, u, before);
        if (threadIdx.x == 0) {
            found[0] = b;
            found[1] = before;
        }
    }
    __syncthreads();
    const int b = static_cast<int>(found[0]);
    const Seq s = seq_of<R>(p, b);
    const int64_t off = u - found[1], seg = off / (s.nt + kSegCost);
    const int64_t a = found[1] + seg * (s.nt + kSegCost), t = a + kSegCost, e = t + s.nt;   // units: the segment, its tiles
    if (t >= u || u - share > t) return;                     // its tiles are not cut here, or cut before
    const int h = static_cast<int>(seg / s.rt), rt = static_cast<int>(seg % s.rt);
    const int c0 = static_cast<int>(t / share), c1 = static_cast<int>((e - 1) / share);
    const int rows = s.qlen * p.group - rt * R;
    auto slot = [&](int64_t c) { return p.part + (c * 2 + (c * share >= a ? 0 : 1)) * C::kSlot; };   // (0: the share's first segment)
    for (int i = threadIdx.x; i < R * 16; i += blockDim.x) {
        const int r = i / 16, c4 = static_cast<int>(blockIdx.y) * 64 + (i % 16) * 4;
        if (r >= rows) continue;
        float mx = -INFINITY;
        for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, slot(c)[R * D + r]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sm = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const float* q = slot(c);
            const float mc = q[R * D + r];
            const float f = mc == -INFINITY ? 0.f : ex2(mc - mx);
            sm += mc == -INFINITY ? q[R * D + R + r] : f * q[R * D + R + r];
            const float4 x = *reinterpret_cast<const float4*>(q + r * D + c4);
            v.x += f * x.x;
            v.y += f * x.y;
            v.z += f * x.z;
            v.w += f * x.w;
        }
        const float inv = sm == 0.f ? 0.f : 1.f / sm;
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        const __nv_bfloat162 z = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        const int rr = rt * R + r, ti = rr / p.group;
        const int64_t row = static_cast<int64_t>(s.tok0 + ti) * p.n_heads + h * p.group + (rr - ti * p.group);
        *reinterpret_cast<uint2*>(p.out + row * D + c4) = sm == 0.f ? make_uint2(0, 0) :
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&z));
    }
}

template <int NB, int NT>
int launch_of(AttnParams p, cudaStream_t s) {
    using C = Shape<NB, NT>;
    p.n_ctas = device_sm_count() * (C::two ? 2 : 1);
    static bool ready[64] = {};   // the attribute is set once a device
    int dev = 0;
    int rc = record_cuda(cudaGetDevice(&dev));
    if (rc) return rc;
    if (dev >= 64 || !ready[dev]) {
        rc = record_cuda(cudaFuncSetAttribute(attn_kernel<NB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
        if (rc) return rc;
        if (dev < 64) ready[dev] = true;
    }
    rc = launch_pdl(attn_kernel<NB, NT>, dim3(static_cast<unsigned>(p.n_ctas)), C::kThreads, C::kSmem, s, p);
    if (rc) return rc;
    return launch_pdl(attn_join_kernel<NB, NT>, dim3(static_cast<unsigned>(p.n_ctas - 1), NB / 2), 128, 0, s, p);
}

// Sequences with more rows a key head than this go to the prompt kernel.  64
// rows: 16 sequences of 4000 keys 132 us here and 93 there, one of 8000 (48
// rows) 28 here and 36 there, where 256-row tiles leave SMs idle.
constexpr int kFew = 32;

// Rows of a segment: 8 where a sequence's rows of one key head fit, else 16.
int rows_of(int max_new, int group) { return static_cast<int64_t>(max_new) * group <= 8 ? 8 : 16; }
bool has_prompts(int head_dim, int max_new, int group) {
    return kv_prompt_covers(head_dim) && static_cast<int64_t>(max_new) * group > kFew;
}

}  // namespace

int64_t kv_attention_workspace(int n_heads, int n_kv, int head_dim, int max_new) {
    const int r = rows_of(max_new, n_heads / n_kv);
    const int ctas = device_sm_count() * 2;
    const int64_t few = static_cast<int64_t>(ctas) * 2 * (r * head_dim + 2 * r) * 4;
    const int64_t more = has_prompts(head_dim, max_new, n_heads / n_kv) ? kv_prompt_workspace(head_dim) : 0;
    return few > more ? few : more;   // the kernels run one after the other
}

int launch_kv_attention(const KvAttention& a, cudaStream_t s) {
    AttnParams p{};
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.n_tokens = static_cast<int>(a.n_tokens);
    p.n_heads = a.n_heads;
    p.n_kv = a.n_kv;
    p.group = a.n_heads / a.n_kv;
    p.cu = a.cu_new;
    p.lens = a.seq_lens;
    p.n_seqs = static_cast<int>(a.n_seqs);
    p.kp = static_cast<const uint8_t*>(a.k_pool);
    p.vp = static_cast<const uint8_t*>(a.v_pool);
    p.n_pages = static_cast<int>(a.n_pages);
    p.page = a.page_size;
    p.by_page = divisor_of(static_cast<uint64_t>(a.page_size));
    p.by_group = divisor_of(static_cast<uint64_t>(p.group));
    p.table = a.block_table;
    p.max_blocks = static_cast<int>(a.max_blocks);
    p.scale = a.scale * kLog2e;
    p.causal = a.causal;
    p.window = a.window;
    p.part = static_cast<float*>(a.workspace);
    p.err = a.err_flag;
    p.status = device_status_ptr();
    const bool small = rows_of(a.max_new, p.group) == 8;
    const bool prompts = has_prompts(a.head_dim, a.max_new, p.group);
    p.few = prompts ? kFew : 0x7fffffff;
    int rc = KQ_ERR_UNSUPPORTED;
    switch (a.head_dim / 32) {
    case 2: rc = small ? launch_of<2, 1>(p, s) : launch_of<2, 2>(p, s); break;
    case 4: rc = small ? launch_of<4, 1>(p, s) : launch_of<4, 2>(p, s); break;
    case 6: rc = small ? launch_of<6, 1>(p, s) : launch_of<6, 2>(p, s); break;
    case 8: rc = small ? launch_of<8, 1>(p, s) : launch_of<8, 2>(p, s); break;
    }
    if (rc || !prompts) return rc;
    return launch_kv_prompt(p, a.head_dim, s);
}

}  // namespace kq
