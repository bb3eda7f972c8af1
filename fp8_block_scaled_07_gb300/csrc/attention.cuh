// attention.cuh -- attention of bf16 queries over the paged 8-bit cache: what
// the kernel for few rows (attention_few.cu: single tokens), the kernel for
// many rows (attention_many.cu: prompts) and the entry point (attention.cu)
// share.
//
//   S[j, t] = sm_scale * q[j] . (k_code[t] * k_scale[page(t), h])
//   out[j]  = sum_t softmax_t(S[j, t]) * v_code[t] * v_scale[page(t), h]
// over the tokens t < len - n + j + 1 of the request (j counts its n queries;
// its last query sees the whole cache).  A query that sees nothing gives
// zeros, and an lse of -inf.  What a query does not see has no part in its
// result, a NaN in K (masked after the product) or in V (note_nans) neither.
//
// Both products run on the tensor core: the e4m3 bytes go from HBM by TMA into
// shared memory.  K is read there by tcgen05.mma as it is, and so is V for few
// rows; for many rows V is converted to fp16 first, exactly, once for 256 rows.
// What meets an e4m3 operand is split instead:
//   * a bf16 q has 8 significant bits.  Scaled by a power of two (its row's
//     largest magnitude into [128, 256)) it is exactly hi + lo / 32 with two
//     e4m3 numbers of 4 significant bits each: hi rounds q to 4 bits, and the
//     rest, at most half a unit of hi, is a multiple of its last bit.  (Below
//     2^-13 of the row's largest element hi is subnormal and the rest is kept
//     to 2^-22 of that element.)
//   * few rows: a probability p in fp32 becomes hi + lo / 32 the same way: 9
//     significant bits, one more than bf16's, down to 2^-9 of the row's
//     largest p; below that a multiple of 2^-18 of it, rounded so that the
//     errors of many cancel (attention_few.cu).  Many rows: p is rounded to
//     fp16, 11 significant bits.
// Few rows: one MMA serves both halves, which are separate columns of its N
// side.  Many rows: two MMAs add to one accumulator.
//
// Scales: with x = S log2(e) + log2(v_scale[page]) and M the running maximum
// of x, the second product's operand is 2^(x - M), V's scale included, and
// the softmax's sum is that of 2^(x - M) / v_scale[page].  So pages of any
// scale share one accumulator, and nothing is multiplied after the product.
#pragma once

#include "common.cuh"

#include <algorithm>

namespace fp8bs {

// 3-D map over a paged cache (gemm.cu)
bool make_cache_map(CUtensorMap* m, const void* base, int64_t n_pages, int64_t rows, int64_t row_bytes, int box_x,
                    int box_rows, bool swizzle128);

struct AttnParams {
    const uint16_t* q;
    int64_t q_ts, q_hs;
    const float *k_scale, *v_scale;
    const int32_t *tables, *lens, *offsets;
    __nv_bfloat16* out;
    float* lse;
    int32_t* next;       // many rows: items taken so far; zero between calls
    int32_t* info;       // few rows: [0] the number of ranges, then a record for each (attn_join_kernel)
    float* parts;        // few rows: partial results, two slots per range
    int64_t T, n_pages, row0;   // row0: first query row of request 0 (offsets == null)
    int32_t B, Hq, Hkv, G, width, bs_log2;
    int32_t few_rows;    // requests of at most this many rows (queries x heads per cache head) are the few-rows kernel's
    int32_t fill_tail;   // this launch writes the rows past offsets[B]
    int32_t debug_skip;  // test hook: a CTA's first tile of V is never loaded
    float scale;         // sm_scale * log2(e)
};

// Tensor maps of the cache: K's first 128 bytes of a row (dk >= 128) and its
// last 64 (dk % 128 == 64), V's rows.
struct AttnMaps {
    CUtensorMap k0, k1, v;
};

// Rows of queries per tile of the few-rows kernel, and its workspace bytes.
int few_rows_per_tile(int G, bool ragged);
size_t few_workspace(int ru, int dv, int sms);
void few_workspace_split(AttnParams& p, void* base, int ru, int sms);
cudaError_t launch_few(int dk, int ru, const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st);
cudaError_t launch_many(int dk, const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st);
int few_read_and_clear_status(cudaStream_t st);
int many_read_and_clear_status(cudaStream_t st);
bool few_set_wait_limit(long long cycles);
bool many_set_wait_limit(long long cycles);
constexpr int kFewB = 256;     // requests per launch of the two kernels
constexpr int kManyB = 256;
constexpr int kMostSegment = 3;   // cost of a segment of the few-rows kernel in tiles, at most (attention_few.cu)

namespace {

__device__ int g_attention_status;   // FP8_OK or FP8_ERR_TIMEOUT; one per translation unit

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLoInv = 1.0f / 32.0f;
constexpr int kRing = 8;            // tiles whose page constants are staged

// Whether a page's scale of V is one: its logarithm and its reciprocal are finite.
__device__ __forceinline__ bool is_scale(float v) { return v >= 0x1p-126f && v < INFINITY; }

__device__ __forceinline__ void attn_abort(volatile int* abort_flag) {
    *abort_flag = 1;
    atomicExch(&g_attention_status, static_cast<int>(FP8_ERR_TIMEOUT));
}

// Maximum over the warp.
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Barrier of `n` threads that also tells whether all of them say ok.
__device__ __forceinline__ bool bar_all(int id, int n, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"(ok ? 1 : 0)
        : "memory");
    return r != 0;
}

// Whether the phase of the given parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// 3-D tiled load: x within a page row's bytes, y the row within a page, z the page.
__device__ __forceinline__ void tma_load_page(void* dst, const void* tmap, uint64_t* bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Shared-memory descriptor with the 64-byte swizzle (K-major, 64-byte rows: atoms of 8 rows, 512 bytes).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(512 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(4) << 61;
    return d;
}

// MN-major operand of 128-byte rows (one row per K index, 128 M or N values),
// 128-byte swizzle: groups of 8 K indices every 1024 bytes; one group wide.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1024 >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Whether any of 16 e4m3 codes is a NaN (0x7F, 0xFF): not 0.
__device__ __forceinline__ uint32_t e4m3_nans(const uint4& v) {
    constexpr uint32_t kAbs = 0x7F7F7F7Fu, kOne = 0x01010101u;
    return (((v.x & kAbs) + kOne) | ((v.y & kAbs) + kOne) | ((v.z & kAbs) + kOne) | ((v.w & kAbs) + kOne)) & 0x80808080u;
}

// V of a token that only some rows see must not hold a NaN: 0 x NaN would enter
// the sums of the others.  Such a NaN becomes 0, and where it stood is noted:
// key[d], for each value d, is the first token with one, as an offset from a
// token that the rows have in common, above a tag that says whose note it is
// (a later one's passes over an earlier one's, so notes are never cleared).
// The results of the rows that see that token are made NaN in the end.
template <int kBits>
__device__ __forceinline__ uint32_t nan_key(uint32_t tag, int offset) {
    return (tag << kBits) | ((1u << kBits) - 1u - static_cast<uint32_t>(offset));
}
// Notes the NaNs among 16 codes of values d .. d + 15 (key: d's).
__device__ __forceinline__ void note_nans(const uint4& v, uint32_t* key, uint32_t mine) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll 1
        for (int b = 0; b < 4; ++b)
            if (((w[i] >> (8 * b)) & 0x7Fu) == 0x7Fu) atomicMax(key + 4 * i + b, mine);
}
// 16 codes, 0 for every NaN.
__device__ __forceinline__ uint4 without_nans(uint4 v) {
    auto of = [](uint32_t x) {
        const uint32_t n = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
        return x & ~(n | (n - (n >> 7)));
    };
    return make_uint4(of(v.x), of(v.y), of(v.z), of(v.w));
}
// Whether a row that sees the tokens below `limit` (as an offset) sees the noted one.
template <int kBits>
__device__ __forceinline__ bool sees_nan(uint32_t key, uint32_t tag, int limit) {
    return (key >> kBits) == tag && limit > static_cast<int>((1u << kBits) - 1u - (key & ((1u << kBits) - 1u)));
}

// N consecutive TMEM columns of this thread's lane, as fp32.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
    static_assert(N == 8 || N % 16 == 0, "columns");
    if constexpr (N == 8) {
        uint32_t r[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 16) {
            uint32_t r[16];
            tmem_ld16(taddr + c, r);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[c + i] = __uint_as_float(r[i]);
        }
    }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

// Two values as e4m3 pairs hi and lo with value = hi + lo / 32: through fp16,
// whose 11 significant bits hold the difference exactly.  `dither` (two fp16)
// is added to lo before it is rounded.
__device__ __forceinline__ void split_e4m3x2(float a, float b, uint16_t& hi, uint16_t& lo, uint32_t dither = 0) {
    uint32_t p2, h2;
    hi = f32x2_to_e4m3x2(a, b);   // (from fp16 it takes twice the issue slots)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p2) : "f"(b), "f"(a));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(hi));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(p2) : "r"(p2), "r"(h2));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p2) : "r"(p2), "r"(0x50005000u), "r"(dither));   // 32, 32
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(p2));
}

int read_and_clear_attention_status(cudaStream_t st) {
    int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_attention_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return -1;
    if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbolAsync(g_attention_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) != cudaSuccess)
            return -1;
        if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
    }
    return v;
}

bool set_attention_wait_limit(long long cycles) {
    return cudaMemcpyToSymbol(g_wait_limit_cycles, &cycles, sizeof(cycles)) == cudaSuccess;
}

}  // namespace
}  // namespace fp8bs
