// kq_kv_attention for many rows a key head (prompts): tcgen05 tensor cores
// over tiles of 256 rows x 128 keys.
//
// Rows are (token, query head of the key head's group) pairs, so one key head's
// tile is decoded once for 256 rows.  Keys and values become binary16 values
// (code - 8) * d in shared memory (one rounding, 2^-11), S = Q K^T and O += P V
// accumulate in fp32 in tensor memory, P = 2^(y - m) goes back to tensor
// memory as binary16 and is the second product's A operand.  The reference m,
// 7 below the running maximum, is only moved when a row's new maximum is more
// than 15 above it, so O is rescaled rarely; P stays below 2^15.1, and weights
// below 2^-32 of the row's largest round to 0.
//
// Warp-specialized, one CTA an SM, 28 warps (one idle):
//   warps 0..15   softmax, two threads a row: warps 0..7 rows 0..127 (first
//                 half), 8..15 rows 128..255; in each the first four take keys
//                 0..63 of every tile (first side), the others 64..127.  q into
//                 shared memory, S from tensor memory, P back, the output
//   warps 16..23  decoders: wire rows -> binary16 key and value tiles in the
//                 128-byte-swizzled layout (thread = key and half of its
//                 blocks; the tile of keys is the K-major operand of Q K^T, the
//                 same layout of values the MN-major operand of P V)
//   warps 24, 25  tcgen05.mma issuers, one a half (the first also allocates
//                 tensor memory): the tensor cores' queue holds a few MMAs, so
//                 one warp's waits and loops run while the other's execute
//   warp 26       block table and bulk copies of 16-key runs
// A half's two sides take turns of 64 keys: S of both has its own 64 columns of
// tensor memory, P takes the first 32 of them, and a side's next Q K^T is issued
// after its P V (MMAs complete in order), while the other side computes.  All
// four groups of four warps are apart, but for the row's reference m: each
// side takes it over from the other's last 64 keys, and hands it on when it is
// half through its exponentials, which keeps the sides out of step.  The order
// of the 32 values inside a block is whatever the code masks give; q is stored
// in the same order and the output is put back in registers.
//
// Work is the list of (sequence, key head, 256 rows, 128 keys) tiles that the
// causal mask and window leave, cut into equal runs, one a CTA, as in the
// few-row kernel; a segment that spans CTAs leaves fp32 partial results.  The
// runs' places are found once, by one CTA, not by every CTA.
//
// Bound by the chain of waits of a side (S, softmax, P, its MMAs); neither the
// tensor pipe nor the exponentials (each about half of the time) are full:
// the last 2048 tokens of 8048, 32 heads over 8 of 128: 262 us (0.90 PFLOP/s;
// 284 after a second or so, when the power cap takes the clock to 1.8 GHz);
// ragged prompts of up to 2500 tokens and as many as 1500 keys before them, 24
// heads over 8 of 64: 290 us (0.45 PFLOP/s), where the exponentials of the
// visible scores alone are 109 us.  Registers are short: 60 bytes of a thread are
// spilled with 128-value heads, 264 with 64.
// What the steps were worth on the first of these: 16-row mma.sync tiles 2513
// us; this kernel with one softmax thread a row 402; two threads a row and the
// plan by one CTA 306; MMAs issued by an elected lane of a whole warp 286; S by
// 32 keys 278; 64 keys a side and one issuing warp 335, with two 279; the
// reference handed over in one look 267; handed on half way and fewer polls 255;
// scores of any size and out-of-range keys by row 262.  A cubic on the FMA pipe
// for 1/4 of the exponentials: 288 for 266; a side's 64 keys in registers at once: 292 for 266; Q K^T of both
// sides at once: 340 for 279 (64 keys cost 51 cycles an MMA, 128 67, but the
// sides wait for each other); polls without a pause: 302 for 266; P beside S
// with 64-value heads, the next Q K^T under the softmax: ragged 309 for 290.
#include "kq_kv.cuh"

namespace kq {
namespace {

constexpr int kRows = 256, kKeys = 128;
constexpr int kSoft = 16, kDec = 8;                 // warps: softmax, decoders
constexpr int kMmaWarp = kSoft + kDec, kLoadWarp = kMmaWarp + 2;
constexpr int kThreads = 32 * (kSoft + kDec + 4);   // seven warpgroups (one warp idle)
// A segment counts as its tiles and kSegCost more in the list: its queries,
// first tiles and output take about as long as that many tiles (ragged prompts:
// 304 us with 3, 290 with 4 or 5, 293 with 6; chosen on these 64-value heads,
// 128 take the same).
constexpr int kSegCost = 4;
constexpr int kRaw = 3;            // raw tiles in flight
constexpr int kMinShare = kSegCost + 3;   // least units of a CTA's share
// A row's reference is 7 below its maximum when it moves, which it does when the
// maximum is more than 15 above it.
constexpr float kPBias = 7.f, kLazy = 8.f;
// Exponents are one FMA of an exact product and the reference while |reference|
// is within this, so that the reference's own rounding is at most 2^-4; past it
// the products are rounded first, as the maximum is, or P could leave binary16.
constexpr float kFar = 1048576.f;

// ---------------------------------------------------------------- PTX glue
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// A and B from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
#define KQ_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                    "=r"(v[i + 6]), "=r"(v[i + 7])
#define KQ_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), \
                    "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of this warp's 32 lanes; the wait is part of the statement, so
// that no use of the registers can move before it.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : KQ_R8(v, 0), KQ_R8(v, 8), KQ_R8(v, 16), KQ_R8(v, 24)
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : KQ_R8(v, 0)
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), KQ_I8(v, 0) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(a),
        KQ_I8(v, 0), KQ_I8(v, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Two fp32 at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 128-byte swizzle, rows of 128 bytes in groups of 8 (1024 bytes).  As a
// K-major operand (rows = M or N) the leading offset is unused; as an MN-major
// operand (rows = K, 64 N values a row) it is the distance to the next 64 N
// values, `next64`.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t next64) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>(next64 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
// kind::f16: D fp32, A and B binary16, M = 128; B K-major or MN-major.
__device__ __forceinline__ constexpr uint32_t idesc_of(int n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// ---------------------------------------------------- order inside a block
// 16-byte chunk c of a row holds the eight values of one 32-bit word of codes:
// chunk 4b + i is word i of block b, whose bytes are (even blocks, 2 bytes off
// a word) 4i + 2 .. 4i + 5 and, for i = 3, 0, 1, 14, 15; (odd blocks) 4i .. 4i + 3.
__device__ __forceinline__ constexpr int byte_of(int b, int i, int k) {
    return (b & 1) ? 4 * i + k : (i < 3 ? 4 * i + 2 + k : (k < 2 ? k : 12 + k));
}
// Value index (0..31) of element e of word i: bytes 0, 2 low, 0, 2 high, 1, 3
// low, 1, 3 high.
__device__ __forceinline__ constexpr int value_of(int b, int i, int e) {
    const int k = 2 * (e & 1) + (e >> 2);
    return byte_of(b, i, k) + ((e & 2) ? 16 : 0);
}

struct Seq {
    int tok0, qlen, pos0, len, rows;
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int b) {
    const Given in = given_of(p, b);
    Seq s;
    s.tok0 = in.tok0;
    s.qlen = in.qlen;
    s.pos0 = in.pos0;
    s.len = in.len;
    s.rows = s.qlen * p.group;
    return s;
}
// Key tiles [t0, t0 + n) that the rows of row tile rt see; at least one, so
// that rows without keys are written.
struct Span {
    int t0, n, lo;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, const Seq& s, int rt) {
    const int first = s.pos0 + group_of(p, rt * kRows);
    const int end = min(rt * kRows + kRows, s.rows) - 1;
    const int last = s.pos0 + group_of(p, end);
    int hi = p.causal ? last + 1 : s.len;     // one past the last key
    hi = hi < 0 ? 0 : (hi > s.len ? s.len : hi);
    int lo = p.window > 0 ? first - p.window + 1 : 0;
    lo = lo < 0 ? 0 : (lo > hi ? hi : lo);
    Span r;
    r.lo = lo;
    r.t0 = lo / kKeys;
    const int n = (hi + kKeys - 1) / kKeys - r.t0;
    r.n = n < 1 ? 1 : n;
    return r;
}
// Units of a sequence for one key head.
__device__ __forceinline__ int64_t tiles_of(const AttnParams& p, const Seq& s) {
    if (s.rows <= p.few) return 0;
    int64_t n = 0;
    for (int rt = 0; rt * kRows < s.rows; ++rt) n += span_of(p, s, rt).n + kSegCost;
    return n;
}

// A place in the list (unit `unit` of a segment), and the units before the segment.
struct Place {
    int b, h, rt, unit;
    int64_t start;
};
// The share's part of the segment at a place: units, and tiles [t0, t0 + n) of
// the row tile's span.
struct Part {
    int units, t0, n;
};
__device__ __forceinline__ Part part_of(const Place& at, const Span& sp, int left) {
    Part r;
    r.units = min(left, sp.n + kSegCost - at.unit);
    r.t0 = max(at.unit - kSegCost, 0);
    r.n = max(at.unit + r.units - kSegCost - r.t0, 0);
    return r;
}
// The plan that one CTA leaves at the head of the work space: the list's
// length, a CTA's share of it and where every share begins.
struct Plan {
    int64_t total, share;
    Place at[1];
};
constexpr int kMostCtas = 255;
constexpr int64_t kPlanBytes = 8192;
static_assert(sizeof(Plan) + kMostCtas * sizeof(Place) <= kPlanBytes, "the plan's room");
__device__ __forceinline__ Plan* plan_of(const AttnParams& p) { return reinterpret_cast<Plan*>(p.part); }
__device__ __forceinline__ float* parts_of(const AttnParams& p) { return p.part + kPlanBytes / 4; }

// One CTA of 256 threads: thread b's tiles of sequence b (a warp a sequence
// where there are few, so that long prompts' row tiles are counted in
// parallel), their running sums, and thread c's place of unit c * share.
__global__ void __launch_bounds__(256) prompt_plan_kernel(const AttnParams p) {
    __shared__ int64_t sums[256];
    pdl_launch();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Plan* plan = plan_of(p);
    // running sums of the tiles of sequences b0 .. b0 + 255, all heads
    auto chunk = [&](int b0) {
        if (p.n_seqs <= 32) {
            if (tid < 256) sums[tid] = 0;
            __syncthreads();
            for (int b = warp; b < p.n_seqs; b += 8) {
                const Seq s = seq_of(p, b);
                int64_t n = 0;
                if (s.rows > p.few)
                    for (int rt = lane; static_cast<int64_t>(rt) * kRows < s.rows; rt += 32) n += span_of(p, s, rt).n + kSegCost;
#pragma unroll
                for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
                if (lane == 0) sums[b] = n * p.n_kv;
            }
        } else {
            sums[tid] = b0 + tid < p.n_seqs ? tiles_of(p, seq_of(p, b0 + tid)) * p.n_kv : 0;
        }
        __syncthreads();
        for (int o = 1; o < 256; o <<= 1) {
            const int64_t v = tid >= o ? sums[tid - o] : 0;
            __syncthreads();
            sums[tid] += v;
            __syncthreads();
        }
    };
    int64_t total = 0;
    for (int b0 = 0; b0 < p.n_seqs; b0 += 256) {
        chunk(b0);
        total += sums[255];
        __syncthreads();
    }
    int64_t share = (total + p.n_ctas - 1) / p.n_ctas;
    share = share < kMinShare ? kMinShare : share;
    if (tid == 0) {
        plan->total = total;
        plan->share = share;
    }
    const int64_t u = share * tid;
    int64_t base = 0;
    for (int b0 = 0; b0 < p.n_seqs && base < total; b0 += 256) {
        if (p.n_seqs > 256) chunk(b0);   // (one chunk is still there)
        if (tid < p.n_ctas && u >= base && u < base + sums[255]) {
            int lo = 0, hi = 255;
            while (lo < hi) {            // the first whose running sum is past u
                const int mid = (lo + hi) >> 1;
                if (base + sums[mid] > u) hi = mid;
                else lo = mid + 1;
            }
            Place at{b0 + lo, 0, 0, 0, 0};
            const int64_t before = base + (lo ? sums[lo - 1] : 0), per = (base + sums[lo] - before) / p.n_kv;
            at.h = static_cast<int>((u - before) / per);
            at.start = before + at.h * per;
            const Seq s = seq_of(p, at.b);
            for (;;) {
                const int k = span_of(p, s, at.rt).n + kSegCost;
                if (u < at.start + k) break;
                at.start += k;
                ++at.rt;
            }
            at.unit = static_cast<int>(u - at.start);
            plan->at[tid] = at;
        }
        base += sums[255];
        __syncthreads();
    }
}
// The next segment of the list (there is one).
__device__ __forceinline__ void advance(const AttnParams& p, Place& at, Seq& s) {
    at.unit = 0;
    ++at.rt;
    if (at.rt * kRows >= s.rows) {
        at.rt = 0;
        if (++at.h == p.n_kv) {
            at.h = 0;
            do {
                ++at.b;
                s = seq_of(p, at.b);
            } while (s.rows <= p.few);
        }
    }
}

template <int NB>
struct Shape {
    static constexpr int D = 32 * NB;
    static constexpr int RB = 18 * NB;
    static constexpr uint32_t kTileB = kKeys * D * 2;        // a key or value tile, a half of q
    static constexpr uint32_t kHalfB = kKeys * 128;          // its first 64 values
    static constexpr uint32_t kRawB = kKeys * RB;
    static constexpr uint32_t kEx = 1024;                    // exchange between the two sides of a row
    static constexpr uint32_t kQ = kEx + 5 * kRows * 4, kK = kQ + 2 * kTileB, kV = kK + 2 * kTileB, kRaw0 = kV + 2 * kTileB;
    static constexpr uint32_t kSmem = kRaw0 + kRaw * kRawB + 1024;
    static constexpr int kSlot = kRows * D + 2 * kRows;      // floats of a partial result
    // Tensor memory: S of both halves and sides (64 columns each, P takes the
    // first 32), O of both halves.
    static constexpr uint32_t kO = 256;
};

struct Bars {
    uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[4], p_full[4], o_full[4], q_full[2];   // [2 half + side]
    uint64_t m_full[16];                                   // [softmax warp]
    uint64_t idle;                                         // second half: a segment without its rows has begun
};

template <int NB>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const AttnParams p) {
    using C = Shape<NB>;
    constexpr int D = C::D, RB = C::RB, HB = NB / 2;   // HB: blocks of one side
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    extern __shared__ uint8_t smem_[];
    uint8_t* smem = smem_ + ((1024u - (smem_u32(smem_) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    Bars& bar = *reinterpret_cast<Bars*>(smem);
    static_assert(sizeof(Bars) <= 512, "barriers");
    volatile uint32_t* tmask = reinterpret_cast<volatile uint32_t*>(smem + 512);  // [16] runs of a tile that are there
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + 576);   // tensor memory, abort
    // [8] segments in turn: first and last key with a scale past 8188
    int* bad_lo = reinterpret_cast<int*>(smem + 640);
    int* bad_hi = bad_lo + 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], kDec);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.k_full[i], kDec);
            mbar_init(&bar.k_empty[i], 2);
            mbar_init(&bar.v_full[i], kDec);
            mbar_init(&bar.v_empty[i], 2);
            mbar_init(&bar.q_full[i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_full[i], 1);
        }
        for (int i = 0; i < 16; ++i) mbar_init(&bar.m_full[i], 1);
        mbar_init(&bar.idle, 1);
        for (int i = 0; i < 8; ++i) {
            bad_lo[i] = 0x7fffffff;
            bad_hi[i] = -1;
        }
        misc[1] = 0;
        fence_barrier_init();
    }
    pdl_launch();
    pdl_wait();
    const Plan* plan = plan_of(p);
    const int64_t total = plan->total, share = plan->share;
    const int64_t u0 = share * blockIdx.x;
    if (u0 >= total) return;
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sb + 576));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    Place at = plan->at[blockIdx.x];
    Seq s = seq_of(p, at.b);
    int left = static_cast<int>(total - u0 < share ? total - u0 : share);
    auto wait = [&](uint64_t* b, uint32_t parity) { return kv_wait(b, parity, misc + 1, p.status); };

    if (warp >= kMmaWarp) {
        regs_dec<56>();
        if (warp < kLoadWarp) {
            // ------------------------------------------------ MMA issuers
            // The whole warp goes through the loop and one elected lane issues:
            // operands that are the same in all lanes by construction (what was
            // loaded comes through a shuffle) sit in uniform registers, where an
            // instruction issued from one lane's own registers takes a loop of
            // its own each time, about 100 cycles, longer than the MMA.
            constexpr uint32_t iqk = idesc_of(kKeys / 2, false), ipv = idesc_of(D, true);
            const int i = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);   // half
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), ts = tm + i * 128, to = tm + C::kO + i * D;
            const uint64_t qd = sw128_desc(sb + C::kQ + i * C::kTileB, 16), kd = sw128_desc(sb + C::kK, 16),
                           vd = sw128_desc(sb + C::kV, C::kHalfB);
            uint32_t n = 0;           // tiles so far
            uint32_t hn = 0, hs = 0;  // tiles of this half (the second may be idle), segments
            bool ok = true;
            auto await = [&](uint64_t* b, uint32_t parity) { ok = __all_sync(0xffffffffu, ok && wait(b, parity)); };
            auto qk = [&](int z, uint32_t m) {   // S of side z = q K^T, tile number m
                const uint64_t b = kd + (((m & 1) * C::kTileB + z * 64 * 128) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t o = ((k >> 2) * C::kHalfB + (k & 3) * 32) >> 4;
                    mma_ss(ts + z * 64, qd + o, b + o, iqk, k != 0);
                }
                tc_commit(&bar.s_full[2 * i + z]);
            };
            while (left > 0 && ok) {
                const Part pt = part_of(at, span_of(p, s, at.rt), left);
                const int tiles = __shfl_sync(0xffffffffu, pt.n, 0);
                const bool used = __shfl_sync(0xffffffffu, tiles > 0 && (i == 0 || s.rows - at.rt * kRows > 128), 0);
                if (tiles > 0) {
                    // (an idle half's softmax warps are waited for all the same, so that
                    // they have read the notes on the segment before)
                    await(&bar.q_full[i], hs & 1);
                    ++hs;
                    if (ok && !used && elect_one()) mbar_arrive(&bar.idle);
                    __syncwarp();
                    await(&bar.k_full[n & 1], (n >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (used) {
                            qk(0, n);
                            qk(1, n);
                        }
                        tc_commit(&bar.k_empty[n & 1]);
                    }
                    __syncwarp();
                }
                for (int j = 0; j < tiles; ++j, ++n) {
                    const bool more = j + 1 < tiles;
                    await(&bar.v_full[n & 1], (n >> 1) & 1);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        if (used) await(&bar.p_full[2 * i + z], hn & 1);
                        if (more && z == 0) await(&bar.k_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            if (used) {
                                // O += P V of this side
                                const uint64_t b = vd + (((n & 1) * C::kTileB + 4 * z * 2048) >> 4);
#pragma unroll
                                for (int k = 0; k < 4; ++k) mma_ts(to, ts + z * 64 + 8 * k, b + (k * 2048 >> 4), ipv, j > 0 || z != 0 || k != 0);
                                tc_commit(&bar.o_full[2 * i + z]);
                                // S shares its room with P: after P V in the same queue
                                if (more) qk(z, n + 1);
                            }
                            if (z == 1) {
                                if (more) tc_commit(&bar.k_empty[(n + 1) & 1]);
                                tc_commit(&bar.v_empty[n & 1]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (used) ++hn;
                }
                left = __shfl_sync(0xffffffffu, left - pt.units, 0);
                if (left > 0) advance(p, at, s);
            }
            // nothing of this CTA's may arrive after its end
            if (n > 0 && ok) wait(&bar.v_empty[(n - 1) & 1], ((n - 1) >> 1) & 1);
        } else if (warp == kLoadWarp) {
            // ------------------------------------------------ loader
            // raw tiles in the order K0, then K(j+1), V(j), over the share
            uint32_t n = 0, st = 0, par = 1;
            auto load = [&](const uint8_t* pool, uint32_t mask, int64_t off) {
                bool ok = true;
                if (lane == 0) {
                    ok = wait(&bar.raw_empty[st], par);
                    if (ok) mbar_arrive_expect_tx(&bar.raw_full[st], __popc(mask) * 16 * RB);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok && ((mask >> lane) & 1u)) bulk_g2s(smem + C::kRaw0 + st * C::kRawB + lane * 16 * RB, pool + off, 16 * RB, &bar.raw_full[st]);
                if (++st == kRaw) {
                    st = 0;
                    par ^= 1;
                }
            };
            uint32_t vmask = 0;    // of the tile whose values come next
            int64_t voff = 0;
            bool pending = false;
            while (left > 0) {
                const Span sp = span_of(p, s, at.rt);
                const Part pt = part_of(at, sp, left);
                for (int j = 0; j < pt.n; ++j, ++n) {
                    // lane i < 8: keys 16 i .. of the tile
                    const int key = (sp.t0 + pt.t0 + j) * kKeys + 16 * lane;
                    int64_t off = 0;
                    bool in = lane < 8 && key < s.len && key + 16 > sp.lo;
                    if (in) {
                        const int blk = page_of(p, key);
                        const int pg = p.table[static_cast<int64_t>(at.b) * p.max_blocks + blk];
                        if (pg < 0 || pg >= p.n_pages) {
                            in = false;
                            if (p.err) atomicOr(p.err, KQ_DEV_BAD_RANGE);
                        } else {
                            off = ((static_cast<int64_t>(pg) * p.n_kv + at.h) * p.page + (key - blk * p.page)) * RB;
                        }
                    }
                    const uint32_t mask = __ballot_sync(0xffffffffu, in);
                    if (lane == 0) tmask[n & 15] = mask;
                    __syncwarp();
                    load(p.kp, mask, off);
                    if (pending) load(p.vp, vmask, voff);
                    vmask = mask;
                    voff = off;
                    pending = true;
                }
                left -= pt.units;
                if (left > 0) advance(p, at, s);
            }
            if (pending) load(p.vp, vmask, voff);
        }
    } else if (warp >= kSoft) {
        regs_dec<48>();
        // ---------------------------------------------------- decoders
        // thread = key and half of its blocks
        const int row = tid & 127, side = (warp - kSoft) >> 2;
        uint32_t st = 0, par = 0, n = 0, seg = 0;
        const uint32_t sw = (row & 7) << 4;
        // tile number m into `base`, from the next raw tile; a key that is not
        // there is zero, and so is a block whose scale passes 8188 (its key is
        // noted for the rows of segment sg, before the tile is handed over)
        auto decode = [&](uint32_t base, uint64_t* full, uint64_t* empty, uint32_t m, bool there, int key, uint32_t sg) {
            bool ok = wait(&bar.raw_full[st], par);
            ok = wait(&empty[m & 1], ((m >> 1) & 1) ^ 1) && ok;
            ok = __all_sync(0xffffffffu, ok);
            bool bad = false;
            if (ok) {
                // NB = 4: a pair of blocks, 9 words; NB = 2: the even block's words
                // 0..4 or the odd one's 4..8
                const uint32_t src = sb + C::kRaw0 + st * C::kRawB + row * RB + side * (NB == 4 ? 36 : 16);
                constexpr int W = NB == 4 ? 9 : 5;
                uint32_t x[W];
#pragma unroll
                for (int i = 0; i < W; ++i) x[i] = lds32(src + 4 * i);
                const uint32_t dst = base + (m & 1) * C::kTileB + row * 128 + (NB == 4 ? side * C::kHalfB : 0);
#pragma unroll
                for (int b = 0; b < HB; ++b) {
                    const bool odd = NB == 4 ? (b & 1) : side != 0;
                    uint32_t d = NB == 4 ? (b ? __byte_perm(x[4], x[4], 0x3232) : __byte_perm(x[0], x[0], 0x1010))
                                         : __byte_perm(x[0], x[0], odd ? 0x3232 : 0x1010);
                    if (!there) d = 0;
                    if ((d & 0x7fffu) > 0x6fffu) {   // past 8188: 8 d is no binary16 value
                        bad = true;
                        d = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t c;
                        if constexpr (NB == 4) {
                            c = b ? x[(5 + i) % W] : (i < 3 ? x[1 + i] : __byte_perm(x[0], x[4], 0x5432));
                        } else {
                            c = i < 3 ? x[1 + i] : (odd ? x[4] : __byte_perm(x[0], x[4], 0x5432));
                        }
                        const uint32_t e = c >> 8;
                        // 1024 + code - 1032 and (1024 + 16 code) / 16 - 72: code - 8, exact
                        const uint32_t v0 = hsub2_u32(and_or(c, 0x000f000fu, 0x64006400u), 0x64086408u);
                        const uint32_t v1 = hfma2_u32(and_or(c, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
                        const uint32_t v2 = hsub2_u32(and_or(e, 0x000f000fu, 0x64006400u), 0x64086408u);
                        const uint32_t v3 = hfma2_u32(and_or(e, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
                        const uint32_t ch = NB == 4 ? 4 * b + i : 4 * side + i;
                        sts128(dst + ((ch << 4) ^ sw), hmul2_u32(v0, d), hmul2_u32(v1, d), hmul2_u32(v2, d), hmul2_u32(v3, d));
                    }
                }
                if (bad) {
                    atomicMin(&bad_lo[sg & 7], key);
                    atomicMax(&bad_hi[sg & 7], key);
                }
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0 && ok) {
                mbar_arrive(&bar.raw_empty[st]);
                mbar_arrive(&full[m & 1]);
            }
            if (++st == kRaw) {
                st = 0;
                par ^= 1;
            }
        };
        bool pending = false, vthere = false;   // of the tile whose values come next
        int vkey = 0;
        uint32_t vseg = 0;
        auto values = [&]() { decode(sb + C::kV, bar.v_full, bar.v_empty, n - 1, vthere, vkey, vseg); };
        while (left > 0) {
            const Span sp = span_of(p, s, at.rt);
            const Part pt = part_of(at, sp, left);
            for (int j = 0; j < pt.n; ++j, ++n) {
                const int key = (sp.t0 + pt.t0 + j) * kKeys + row;
                wait(&bar.raw_full[st], par);   // the loader's mask is there with the raw tile
                const bool there = key < s.len && key >= sp.lo && ((tmask[n & 15] >> (row >> 4)) & 1u);
                decode(sb + C::kK, bar.k_full, bar.k_empty, n, there, key, seg);
                if (pending) values();
                vthere = there;
                vkey = key;
                vseg = seg;
                pending = true;
            }
            seg += pt.n > 0;
            left -= pt.units;
            if (left > 0) advance(p, at, s);
        }
        if (pending) values();
    } else {
        regs_inc<88>();
        // ------------------------------------------------------ softmax
        // Two threads a row: keys 0..63 and 64..127 of every tile (`side`), the
        // first and second half of q's and the output's values.
        const int half = warp >> 3, side = (warp >> 2) & 1, row = 32 * (warp & 3) + lane, pr = 128 * half + row;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // this warp's 32 lanes of tensor memory
        const uint32_t ts = tmem + half * 128 + 64 * side + lanes;
        const uint32_t to = tmem + C::kO + half * D + lanes;
        // exchange with the row's other thread: double-buffered, so that one
        // barrier of the two warps is enough
        float* ex = reinterpret_cast<float*>(smem + C::kEx) + pr;
        uint32_t flip = 0;
        const int pair = 1 + 4 * half + (warp & 3);
        // the reference that the row's two threads hand each other: one word,
        // written by whichever has its turn
        float* mex = reinterpret_cast<float*>(smem + C::kEx) + 4 * kRows + pr;
        uint64_t *mine = &bar.m_full[warp], *theirs = &bar.m_full[warp ^ 4];
        auto other = [&](float v) {
            ex[(flip + side) * kRows] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            const float o = ex[(flip + (side ^ 1)) * kRows];
            flip ^= 2;
            return o;
        };
        uint32_t n = 0;                // tiles so far
        uint32_t hn = 0, seg = 0;      // tiles of this half, segments
        uint32_t idle = 0;             // segments without rows of this half
        int slot = 0;
        for (; left > 0;) {
            const Span sp = span_of(p, s, at.rt);
            const Part pt = part_of(at, sp, left);
            const int tiles = pt.n;
            const bool used = tiles > 0 && (half == 0 || s.rows - at.rt * kRows > 128);
            if (used) {
                const bool whole = tiles == sp.n;
                const int rr = at.rt * kRows + pr;
                const bool there = rr < s.rows;
                const int ti = there ? group_of(p, rr) : 0;
                const int64_t qhead = static_cast<int64_t>(at.h) * p.group + (there ? rr - ti * p.group : 0);
                const int pos = s.pos0 + ti;
                int hi = p.causal ? min(pos, s.len - 1) : s.len - 1;
                int lo = p.window > 0 ? pos - p.window + 1 : 0;
                if (!there) {
                    hi = 0x7fffffff;
                    lo = 0;
                }
                // keys that every row of this warp sees
                const int all_hi = __reduce_min_sync(0xffffffffu, hi), all_lo = __reduce_max_sync(0xffffffffu, lo);
                // ---- q: scaled by a power of two, in the blocks' order
                float c = 1.f;       // of S, to base-2 scores
                {
                    const uint16_t* src = p.q + (s.tok0 + ti) * p.q_stride + qhead * D + D / 2 * side;
                    uint32_t w[D / 4];
                    uint32_t mx = 0;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint4 v = there ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
                        w[4 * i] = v.x;
                        w[4 * i + 1] = v.y;
                        w[4 * i + 2] = v.z;
                        w[4 * i + 3] = v.w;
                        mx = absmax8_bf16(mx, v);
                    }
                    mx = max(mx & 0xffffu, mx >> 16);
                    if (mx >= 0x7f80u && p.err) atomicOr(p.err, KQ_DEV_X_RANGE);
                    mx = max(mx, __float_as_uint(other(__uint_as_float(mx))));
                    const int e = xscale_exp(mx, 13);
                    // the scale's sign goes into q, so that c > 0; scale 0: q = 0
                    const float up = p.scale == 0.f ? 0.f : copysignf(exp2_int(e), p.scale);
                    c = factor_of(p.scale, e, 0);
                    const uint32_t dst = sb + C::kQ + half * C::kTileB + row * 128 + (NB == 4 ? side * C::kHalfB : 0);
#pragma unroll
                    for (int b = 0; b < HB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t o[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float f[2];
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    // (NB = 2: the side is the block's parity)
                                    const int v0 = 32 * b + value_of(NB == 4 ? b : 0, i, 2 * k + z);
                                    const int v1 = 32 * b + value_of(NB == 4 ? b : 1, i, 2 * k + z);
                                    const float a0 = (v0 & 1) ? bf16hi_to_f32(w[v0 >> 1]) : bf16lo_to_f32(w[v0 >> 1]);
                                    const float a1 = (v1 & 1) ? bf16hi_to_f32(w[v1 >> 1]) : bf16lo_to_f32(w[v1 >> 1]);
                                    f[z] = (NB == 2 && side ? a1 : a0) * up;
                                }
                                o[k] = pack_f16x2(f[0], f[1]);
                            }
                            const uint32_t ch = NB == 4 ? 4 * b + i : 4 * side + i;
                            sts128(dst + ((ch << 4) ^ ((row & 7) << 4)), o[0], o[1], o[2], o[3]);
                        }
                    fence_proxy_async();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_full[half]);
                }
                float m = -INFINITY;     // reference of the base-2 exponents
                bool far = false;        // a reference of this warp's has been past kFar:
                float cf = c;            // S is multiplied when it is loaded, and cf is 1
                float2 l2 = make_float2(0.f, 0.f);
                if (!side) *mex = m;
                auto times = [](uint32_t a, float f) { return __float_as_uint(__fmul_rn(__uint_as_float(a), f)); };
                // moves the sum to another reference; the factor
                auto follow = [&](float nm) {
                    const float f = m == nm ? 1.f : ex2(m - nm);
                    m = nm;
                    l2.x *= f;
                    l2.y *= f;
                    return f;
                };
                for (int j = 0; j < tiles; ++j) {
                    // (where a wait has run out the CTA goes through its barriers all
                    // the same, on whatever is there)
                    wait(&bar.s_full[2 * half + side], (hn + j) & 1);
                    // the reference after the 64 keys before these
                    float before = m;
                    if (side || j > 0) {
                        wait(theirs, (hn + j - (side ^ 1)) & 1);
                        before = *mex;
                    }
                    __syncwarp();
                    tc_fence_after();
                    const int key0 = (sp.t0 + pt.t0 + j) * kKeys + 64 * side;
                    const uint32_t mask = (tmask[(n + j) & 15] >> (4 * side)) & 15u;
                    bool edge = key0 + 63 > all_hi || key0 < all_lo || mask != 15u || far;
                    // 32 keys of S at a time (keys 32 w ..), hidden ones -inf: the
                    // second 32, then the first, which stay in registers, and the
                    // second again after those are done
                    uint32_t x[32];
                    auto load = [&](int w) {
                        tmem_ld32(ts + 32 * w, x);
                        if (edge) {
                            // bits of the keys that this row sees
                            const int h0 = hi - key0 - 32 * w, l0 = lo - key0 - 32 * w;
                            uint32_t bits = h0 < 0 ? 0u : (h0 >= 31 ? ~0u : (2u << h0) - 1u);
                            bits &= l0 <= 0 ? ~0u : (l0 > 31 ? 0u : ~0u << l0);
                            bits &= ((mask >> (2 * w)) & 1u ? 0xffffu : 0u) | ((mask >> (2 * w)) & 2u ? 0xffff0000u : 0u);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((bits >> k) & 1u)) x[k] = 0xff800000u;
                            if (far) {
#pragma unroll
                                for (int k = 0; k < 32; ++k) x[k] = times(x[k], c);
                            }
                        }
                    };
                    auto largest = [&]() {
                        float mx[4];     // (one chain would wait for each step)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 4]));
#pragma unroll
                        for (int k = 8; k < 32; k += 8)
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                mx[z] = fmaxf(mx[z], fmaxf(__uint_as_float(x[k + z]), __uint_as_float(x[k + z + 4])));
                        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    };
                    load(1);
                    float mt = largest();
                    load(0);
                    mt = __fmul_rn(fmaxf(mt, largest()), cf);
                    if (__any_sync(0xffffffffu, before != m || mt - before > kPBias + kLazy)) {
                        follow(before);
                        const bool grow = __any_sync(0xffffffffu, mt - m > kPBias + kLazy);
                        const float nm = grow ? fmaxf(m, mt - kPBias) : m;
                        *mex = nm;
                        const float f = follow(nm);
                        if (!far && __any_sync(0xffffffffu, fabsf(m) > kFar && m != -INFINITY)) {
                            far = edge = true;
                            cf = 1.f;
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = times(x[k], c);
                        }
                        if (grow && (side || j > 0)) {
                            // O is the sum up to those keys once their P V is done
                            wait(&bar.o_full[2 * half + (side ^ 1)], (hn + j - (side ^ 1)) & 1);
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < D / 8; ++k) {
                                uint32_t o[8];
                                tmem_ld8(to + 8 * k, o);
#pragma unroll
                                for (int z = 0; z < 8; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * f);
                                tmem_st8(to + 8 * k, o);
                            }
                        }
                    }
                    const float bias = m == -INFINITY ? 0.f : -m;
                    const float2 cc = make_float2(cf, cf), bb = make_float2(bias, bias);
                    auto power = [&](int w) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float2 y = make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
                            y = fma2(y, cc, bb);
                            y.x = ex2(y.x);
                            y.y = ex2(y.y);
                            l2 = add2(l2, y);
                            x[k] = pack_f16x2(y.x, y.y);
                        }
                        tmem_st16(ts + 16 * w, x);
                    };
                    power(0);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(mine);
                    load(1);
                    power(1);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[2 * half + side]);
                }
                // ---- output
                if (!side) {
                    wait(theirs, (hn + tiles - 1) & 1);
                    follow(*mex);
                }
                float l = l2.x + l2.y;
                l += other(l);
                if (__all_sync(0xffffffffu, wait(&bar.o_full[2 * half + 1], (hn + tiles - 1) & 1))) {
                    tc_fence_after();
                    // a row that sees a key with a scale past 8188
                    const int b0 = bad_lo[seg & 7], b1 = bad_hi[seg & 7];
                    bool bad = there && b1 >= lo && b0 <= hi;
                    if (bad && b0 < lo && b1 > hi) {
                        // one before and one behind the row's keys: look at its own
                        bad = false;
                        const int end = min(hi, (sp.t0 + pt.t0 + tiles) * kKeys - 1);
#pragma unroll 1
                        for (int key = max(lo, (sp.t0 + pt.t0) * kKeys); key <= end && !bad; ++key) {
                            const int blk = page_of(p, key), pg = p.table[static_cast<int64_t>(at.b) * p.max_blocks + blk];
                            if (pg < 0 || pg >= p.n_pages) continue;
                            const int64_t off = ((static_cast<int64_t>(pg) * p.n_kv + at.h) * p.page + (key - blk * p.page)) * RB;
#pragma unroll 1
                            for (int b = 0; b < NB; ++b) {
                                const int kd = *reinterpret_cast<const uint16_t*>(p.kp + off + 18 * b) & 0x7fff;
                                const int vd = *reinterpret_cast<const uint16_t*>(p.vp + off + 18 * b) & 0x7fff;
                                bad |= max(kd, vd) > 0x6fff;
                            }
                        }
                    }
                    __syncwarp();
                    if (bad) l = __int_as_float(0x7fc00000);
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    float* part = parts_of(p) + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * C::kSlot;
                    uint16_t* out = p.out + (static_cast<int64_t>(s.tok0 + ti) * p.n_heads + qhead) * D + D / 2 * side;
#pragma unroll
                    for (int b = 0; b < HB; ++b) {
                        uint32_t o[32];
                        tmem_ld32(to + D / 2 * side + 32 * b, o);
                        auto at_value = [&](int v) {   // value v of the block, from its place in the codes' order
                            float r = 0.f;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    if (NB == 4 && value_of(b, i, e) == v) r = __uint_as_float(o[8 * i + e]);
                                    if (NB == 2 && value_of(0, i, e) == v && side == 0) r = __uint_as_float(o[8 * i + e]);
                                    if (NB == 2 && value_of(1, i, e) == v && side == 1) r = __uint_as_float(o[8 * i + e]);
                                }
                            return r;
                        };
                        if (whole) {
                            if (there) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    uint32_t h[4];
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const __nv_bfloat162 t2 = __floats2bfloat162_rn(at_value(8 * i + 2 * k) * inv, at_value(8 * i + 2 * k + 1) * inv);
                                        h[k] = l == 0.f ? 0u : *reinterpret_cast<const uint32_t*>(&t2);
                                    }
                                    *reinterpret_cast<uint4*>(out + 32 * b + 8 * i) = make_uint4(h[0], h[1], h[2], h[3]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<float4*>(part + pr * D + D / 2 * side + 32 * b + 4 * i) =
                                    make_float4(at_value(4 * i), at_value(4 * i + 1), at_value(4 * i + 2), at_value(4 * i + 3));
                        }
                    }
                    if (!whole && side == 0) {
                        part[kRows * D + pr] = m;
                        part[kRows * D + kRows + pr] = l;
                    }
                }
                hn += tiles;
            } else if (tiles > 0) {
                // this half has no rows here, but keeps in step with its issuer
                if (lane == 0) mbar_arrive(&bar.q_full[half]);
                wait(&bar.idle, idle & 1);
                ++idle;
            }
            // the slot of the segment four on: the halves are at most two tiles
            // apart, the decoders at most two tiles ahead of the slower one
            if (tiles > 0 && tid == 0) {
                bad_lo[(seg + 4) & 7] = 0x7fffffff;
                bad_hi[(seg + 4) & 7] = -1;
            }
            seg += tiles > 0;
            n += tiles;
            left -= pt.units;
            slot = 1;
            if (left > 0) advance(p, at, s);
        }
    }
    if (misc[1]) {   // let copies and MMAs in flight finish before the CTA's memory goes
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 2000000ull) __nanosleep(10000);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the partial results of a segment that spans CTAs, in list order: the
// first boundary between shares inside a segment takes it, 8 rows a block.
template <int NB>
__global__ void __launch_bounds__(256) prompt_join_kernel(const AttnParams p) {
    using C = Shape<NB>;
    constexpr int D = C::D, per = D / 4;
    pdl_wait();
    const Plan* plan = plan_of(p);
    const int64_t share = plan->share, u = share * (static_cast<int64_t>(blockIdx.x) + 1);
    if (u >= plan->total) return;
    const Place at = plan->at[blockIdx.x + 1];
    const Seq s = seq_of(p, at.b);
    const int64_t a = at.start, t = a + kSegCost, e = t + span_of(p, s, at.rt).n;   // units: the segment, its tiles
    if (t >= u || u - share > t) return;   // its tiles are not cut here, or cut before
    const int c0 = static_cast<int>(t / share), c1 = static_cast<int>((e - 1) / share);
    auto slot = [&](int64_t c) { return parts_of(p) + (c * 2 + (c * share >= a ? 0 : 1)) * C::kSlot; };   // (0: the share's first segment)
    for (int i = threadIdx.x; i < 8 * per; i += 256) {
        const int r = blockIdx.y * 8 + i / per, c4 = (i % per) * 4, rr = at.rt * kRows + r;
        if (rr >= s.rows) continue;
        float mx = -INFINITY;
        for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, slot(c)[kRows * D + r]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const float* q = slot(c);
            const float mc = q[kRows * D + r], lc = q[kRows * D + kRows + r];
            const float f = mc == -INFINITY ? 0.f : ex2(mc - mx);
            l += mc == -INFINITY ? lc : f * lc;
            const float4 x = *reinterpret_cast<const float4*>(q + r * D + c4);
            v.x += f * x.x;
            v.y += f * x.y;
            v.z += f * x.z;
            v.w += f * x.w;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        const __nv_bfloat162 z = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        const int ti = group_of(p, rr);
        const int64_t row = static_cast<int64_t>(s.tok0 + ti) * p.n_heads + at.h * p.group + (rr - ti * p.group);
        *reinterpret_cast<uint2*>(p.out + row * D + c4) = l == 0.f ? make_uint2(0, 0) :
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&z));
    }
}

int prompt_ctas() { return device_sm_count() < kMostCtas ? device_sm_count() : kMostCtas; }

template <int NB>
int launch_of(AttnParams p, cudaStream_t s) {
    using C = Shape<NB>;
    p.n_ctas = prompt_ctas();
    static bool ready[64] = {};   // the attribute is set once a device
    int dev = 0;
    int rc = record_cuda(cudaGetDevice(&dev));
    if (rc) return rc;
    if (dev >= 64 || !ready[dev]) {
        rc = record_cuda(cudaFuncSetAttribute(prompt_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
        if (rc) return rc;
        if (dev < 64) ready[dev] = true;
    }
    rc = launch_pdl(prompt_plan_kernel, dim3(1), 256, 0, s, p);
    if (rc) return rc;
    rc = launch_pdl(prompt_kernel<NB>, dim3(static_cast<unsigned>(p.n_ctas)), kThreads, C::kSmem, s, p);
    if (rc || p.n_ctas == 1) return rc;
    return launch_pdl(prompt_join_kernel<NB>, dim3(static_cast<unsigned>(p.n_ctas - 1), kRows / 8), 256, 0, s, p);
}

}  // namespace

bool kv_prompt_covers(int head_dim) { return head_dim == 64 || head_dim == 128; }

int64_t kv_prompt_workspace(int head_dim) {
    return kPlanBytes + static_cast<int64_t>(prompt_ctas()) * 2 * (kRows * head_dim + 2 * kRows) * 4;
}

int launch_kv_prompt(AttnParams p, int head_dim, cudaStream_t s) {
    return head_dim == 64 ? launch_of<2>(p, s) : launch_of<4>(p, s);
}

}  // namespace kq
