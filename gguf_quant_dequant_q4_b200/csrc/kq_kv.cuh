// Shared by the KV-cache kernels (plan, append, attention).
//
// A pool is [n_pages, n_kv_heads, page_size, row] bytes, row = head_dim / 32
// q4_0 wire blocks of 18 bytes, so the rows of one head in one page are one
// contiguous run; page_size is a multiple of 16, so every run of 16 tokens
// starts on a 16-byte boundary and is a multiple of 16 bytes (288 * blocks).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kq_device.cuh"
#include "kq_launch.h"

namespace kq {

// Programmatic dependent launch: a kernel may start while the one before it
// on the stream still runs; nothing is read or written before this wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class K, class... A>
int launch_pdl(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = use_pdl() ? 1 : 0;
    return record_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

constexpr float kLog2e = 1.4426950408889634f;

// Division of n < 2^31 by a divisor known on the host: umulhi(n, mul) >> shift
// with 2^k < d <= 2^(k + 1) (k = shift) and mul = ceil(2^(32 + k) / d) < 2^32:
// mul d exceeds 2^(32 + k) by less than d, and n 2^(k + 1) < 2^(32 + k), so the
// product's error stays below 1 / d.  d = 1 has mul 0.
struct Divisor {
    uint32_t mul;
    int shift;
};
inline Divisor divisor_of(uint64_t d) {
    Divisor r{0, 0};
    if (d < 2) return r;
    while ((uint64_t(2) << r.shift) < d) ++r.shift;
    r.mul = static_cast<uint32_t>(((uint64_t(1) << (32 + r.shift)) + d - 1) / d);
    return r;
}
__device__ __forceinline__ int divide(int n, const Divisor& d) {
    return d.mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), d.mul) >> d.shift) : n;
}

// An attention call as its kernels take it.
struct AttnParams {
    const uint16_t* q;
    int64_t q_stride;            // elements between tokens
    uint16_t* out;               // [n_tokens, n_heads, D]
    int n_tokens;
    int n_heads, n_kv, group;
    Divisor by_group, by_page;
    const int32_t* cu;
    const int32_t* lens;
    int n_seqs;
    const uint8_t* kp;
    const uint8_t* vp;
    int n_pages, page;
    const int32_t* table;
    int max_blocks;
    float scale;                 // times log2(e)
    int causal, window;
    float* part;                 // partial results, two slots a CTA
    int n_ctas;
    int few;                     // sequences of at most this many rows a key head go to the few-row kernel
    int32_t* err;
    int* status;
};

// Bounded wait of a pipeline (all threads of a warp, or one): the timer's read
// paces the polls, so that warps that wait leave the issue slots to those that
// work (32 polls a read: prompts 267 us for 257).  False once the limit has passed, or where another wait of the CTA has
// run out before (*gone).
__device__ __forceinline__ bool kv_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* gone, int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (*gone) return false;
        if (mbar_try_wait(bar, parity)) return true;
        if (global_ns() - t0 > kWaitLimitNs) break;
    }
    *gone = 1;
    if (status) atomicOr(status, KQ_DEV_TIMEOUT);
    return false;
}

// Rows and keys of sequence b.  Its tokens keep the places that the given
// lengths say, whatever the tokens and the table row hold: the one at tok0 + i
// stands at pos0 + i, and keys behind the row count as hidden.
struct Given {
    int tok0, qlen, pos0, len;   // first token, tokens, its position, keys that the table row holds
    int bad;                     // KQ_DEV_* of lengths that do not fit
};
__device__ __forceinline__ Given given_of(const AttnParams& p, int b) {
    Given s;
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    const int end = c1 < 0 ? 0 : (c1 > p.n_tokens ? p.n_tokens : c1);
    s.tok0 = c0 < 0 ? 0 : (c0 > end ? end : c0);
    s.qlen = end - s.tok0;
    const int len = p.lens[b] < 0 ? 0 : p.lens[b], most = p.max_blocks * p.page;
    s.len = len < most ? len : most;
    // (positions below -qlen see as little as -qlen)
    const int64_t pos = static_cast<int64_t>(len) - c1 + s.tok0;
    s.pos0 = pos < -s.qlen ? -s.qlen : static_cast<int>(pos);
    s.bad = (c0 < 0 || c1 > p.n_tokens || c1 < c0 ? KQ_DEV_BAD_RANGE : 0) | (len > most && s.qlen > 0 ? KQ_DEV_TOO_MANY : 0);
    return s;
}

// Token of a row, table place of a key.
__device__ __forceinline__ int group_of(const AttnParams& p, int row) { return divide(row, p.by_group); }
__device__ __forceinline__ int page_of(const AttnParams& p, int key) { return divide(key, p.by_page); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The factor of a row's products q . k (q scaled by 2^e, the products by 2^-up)
// to base-2 scores, kept among fp32's normal numbers.  Where it is cut the
// softmax is the same: below, the scores are 0 to all bits; above, two products
// that differ (by 2^-72 at least, the operands being binary16) are 2^55 apart.
__device__ __forceinline__ float factor_of(float scale, int e, int up) {
    if (scale == 0.f) return 1.f;   // (and q is 0)
    const float f = fabsf(scale) * exp2_int(-e) * exp2_int(up);
    return fminf(fmaxf(f, 1.17549435e-38f), 3.40282347e38f);
}

// The prompt kernel (kq_kv_prompt.cu) on tcgen05: head sizes that it covers,
// its work space and its launch.
bool kv_prompt_covers(int head_dim);
int64_t kv_prompt_workspace(int head_dim);
int launch_kv_prompt(AttnParams p, int head_dim, cudaStream_t s);

}  // namespace kq
