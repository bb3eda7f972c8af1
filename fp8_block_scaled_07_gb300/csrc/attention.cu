// attention.cu -- fp8_kv_attention: argument checks, tensor maps, launches
// (kernels: attention_few.cu, attention_many.cu).
#include <cmath>

#include "attention.cuh"

namespace fp8bs {
int take_debug_skip();   // gemm.cu

namespace {

bool block_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
bool dims_ok(int32_t dk, int32_t dv) {
    return (dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128);
}

constexpr size_t kCounterBytes = 16 * 1024;   // as fp8_gemm's, zero between calls: one workspace serves both

}  // namespace

int attention_read_and_clear_status(cudaStream_t st) {
    const int f = few_read_and_clear_status(st), m = many_read_and_clear_status(st);
    return f != 0 ? f : m;
}
bool attention_set_wait_limit(long long cycles) { return few_set_wait_limit(cycles) && many_set_wait_limit(cycles); }

}  // namespace fp8bs

using namespace fp8bs;

extern "C" size_t fp8_kv_attention_workspace_size(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t dk, int32_t dv) {
    if (T <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !dims_ok(dk, dv)) return 0;
    return kCounterBytes + few_workspace(few_rows_per_tile(Hq / Hkv, T != B), dv, device_sm_count());
}

extern "C" fp8_status fp8_kv_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                       const void* k_cache, const float* k_scale, const void* v_cache,
                                       const float* v_scale, int64_t n_pages, int32_t block_size,
                                       const int32_t* tables, int32_t width, const int32_t* lens,
                                       const int32_t* offsets, int32_t B, int64_t T, int32_t Hq, int32_t Hkv,
                                       int32_t dk, int32_t dv, float sm_scale, void* out, float* lse, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (T < 0 || B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || n_pages <= 0 || width <= 0) return FP8_ERR_INVALID_ARG;
    // (tiles of 128 tokens, the last one's end included, are counted in 31 bits)
    if (!block_size_ok(block_size) || static_cast<int64_t>(width) * block_size > (1LL << 31) - 128)
        return FP8_ERR_INVALID_ARG;
    if (!(sm_scale > 0.0f) || std::isinf(sm_scale) || q_token_stride < 0 || q_head_stride < 0 || q_token_stride % 8 || q_head_stride % 8)
        return FP8_ERR_INVALID_ARG;
    if (!offsets && T != B) return FP8_ERR_INVALID_ARG;
    if (!dims_ok(dk, dv) || T > (1LL << 31) - 1 || n_pages > (1LL << 31) - 1) return FP8_ERR_UNSUPPORTED;
    if (T == 0) return FP8_OK;
    if (B == 0 || !q || !tables || !lens || !out || !k_cache || !k_scale || !v_cache || !v_scale)
        return FP8_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(out) & 31))
        return FP8_ERR_INVALID_ARG;
    const int G = Hq / Hkv, sms = device_sm_count();
    const int ru = few_rows_per_tile(G, T != B);
    if (!workspace || !aligned16(workspace) || workspace_bytes < kCounterBytes + few_workspace(ru, dv, sms))
        return FP8_ERR_WORKSPACE;
    AttnParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.next = static_cast<int32_t*>(workspace);   // (zero again after every call)
    few_workspace_split(p, static_cast<uint8_t*>(workspace) + kCounterBytes, ru, sms);
    p.T = T;
    p.n_pages = n_pages;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = G;
    p.width = width;
    while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
    p.scale = sm_scale * 1.4426950408889634f;
    p.debug_skip = take_debug_skip();
    // The few-rows kernel reads a request's cache once for every ru rows, but
    // spreads it over the GPU; the many-rows kernel once for 256 rows, on one
    // SM for each of them and each cache head.  So a request stays with the
    // former for two passes (64 requests of 4096 tokens, 8 cache heads of 128:
    // 16 rows 113 us, 32 rows 210, where a third pass would make it 304; the
    // other kernel 198 to 202 for 40 to 128 rows, so that two passes are about
    // even with it), and for four where the latter could not fill the GPU (4
    // requests: 32 rows 27 us, 64 rows 36, 128 rows 58; the other kernel 71).
    p.few_rows = offsets ? (static_cast<int64_t>(B) * Hkv < sms ? 4 : 2) * ru : G;
    // maps over [n_pages][Hkv * block_size] rows
    const int64_t rows = static_cast<int64_t>(Hkv) * block_size;
    AttnMaps m;
    bool ok = true;
    if (dk >= 128) ok = make_cache_map(&m.k0, k_cache, n_pages, rows, dk, 128, block_size, true);
    if (dk % 128) ok = ok && make_cache_map(&m.k1, k_cache, n_pages, rows, dk, 64, block_size, false);
    // (the few-rows kernel reads V of 64 values as rows of token pairs)
    ok = ok && (dv == 64 ? make_cache_map(&m.v, v_cache, n_pages, rows / 2, 128, 128, block_size / 2, true)
                         : make_cache_map(&m.v, v_cache, n_pages, rows, 128, 128, block_size, true));
    if (!ok) return FP8_ERR_CUDA;
    if (dk < 128) m.k0 = m.k1;       // not read
    if (dk % 128 == 0) m.k1 = m.k0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    auto requests = [&](int32_t b0, int32_t n) {
        p.B = std::min(B - b0, n);
        p.tables = tables + static_cast<int64_t>(b0) * width;
        p.lens = lens + b0;
        p.offsets = offsets ? offsets + b0 : nullptr;
        p.row0 = b0;
        p.fill_tail = b0 + p.B == B;
    };
    // requests per launch: their tiles of one cache head are counted in 31 bits
    const int64_t most = (static_cast<int64_t>(width) * block_size / 128 + 1 + kMostSegment) * ((p.few_rows + ru - 1) / ru);
    const int32_t step = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(kFewB, ((1LL << 31) - 1) / most)));
    for (int32_t b0 = 0; b0 < B && e == cudaSuccess; b0 += step) {
        requests(b0, step);
        e = launch_few(dk, ru, m, p, sms, st);
    }
    if (offsets && T * G > p.few_rows && e == cudaSuccess) {   // (else no request can have more rows)
        if (dv == 64 && !make_cache_map(&m.v, v_cache, n_pages, rows, 64, 64, block_size, false)) return FP8_ERR_CUDA;
        for (int32_t b0 = 0; b0 < B && e == cudaSuccess; b0 += kManyB) {
            requests(b0, kManyB);
            e = launch_many(dk, m, p, sms, st);
        }
    }
    return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}
