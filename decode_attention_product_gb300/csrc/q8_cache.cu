// q8_cache.cu -- the 8-bit block-scaled cache: append of new tokens and the
// read-back of cached ones.
//
// Work is cut by block: a warp, or half of one, per (request, page, kv head, K or V), so
// a block's scale and its up to 16 rows belong to it and nothing is shared between
// warps.
//
// Measured, 32 kv heads: append of 7.7 k tokens in 5 prompts (INT8) 37 us for 188 MB,
// bound by issue (70 % of the slots: about 54 instructions per 128-element row) and
// the chain of dependent loads before it; read-back of the same 34 us, bound by that
// chain (request, length, page, codes).  One token for each of 256 requests: append 5
// us, read-back of its blocks 14 us for 53 MB.
//
// A ragged call knows its requests only on the device (cu_tokens).  Request b
// owns the work units from v_b = cu_tokens[b] / 16 + 2 b on: appending n tokens
// touches at most n / 16 + 2 pages, which v_{b+1} - v_b never undercuts, so the
// host can size the grid from the token count alone (T / 16 + 2 B + 1 units,
// two idle ones per request at most) and a warp finds its request by a search
// over v: 256 requests in one step, more by 32-way steps.
#include "common.cuh"
#include "internal.h"
#include "q8_common.cuh"

namespace aq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Q8CacheParams {
    __half *kv;                    // [T][Hkv][2][D]: read by the append, written by the read-back
    uint8_t *pages;                // [NP][Hkv][2][P][D]
    float *scales;                 // [NP][Hkv][2]
    const int32_t *block_table;    // [B][max_pages]
    const int32_t *seq_lens;       // [B]
    const int32_t *cu_tokens;      // [B + 1], or null: one token per request
    int32_t *status;
    int64_t num_pages;
    int32_t batch, num_tokens, num_kv_heads, max_pages;
};

__device__ __forceinline__ float4 halves(uint2 u) {
    const float2 a = h2_to_f2(u.x), b = h2_to_f2(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void load_row(const __half *src, uint2 (&x)[1]) { x[0] = ld_global_na_v2(src); }

__device__ __forceinline__ void load_row(const __half *src, uint2 (&x)[2]) {
    const uint4 v = ld_global_na_v4(src);
    x[0] = make_uint2(v.x, v.y);
    x[1] = make_uint2(v.z, v.w);
}

__device__ __forceinline__ void store_codes(uint32_t *dst, const uint32_t (&c)[1]) { *dst = c[0]; }

__device__ __forceinline__ void store_codes(uint32_t *dst, const uint32_t (&c)[2]) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
}

struct Unit {
    int page;                      // the block table's entry, not checked (kNoPage: no place in the cache)
    int s0, n;                     // slots [s0, s0 + n) of the page; n == 0: nothing to do
    int64_t row;                   // token row of slot s0
};
constexpr int kNoPage = -2147483647 - 1;

// The unit's rows and block.  A request that does not fit is flagged here.
__device__ __forceinline__ Unit find_unit(const Q8CacheParams &p, int u, int lane) {
    constexpr int P = kPage;
    Unit w{kNoPage, 0, 0, 0};
    int b = u, first = u, n = 1, local = 0;
    if (p.cu_tokens) {
        int lo = 0, hi = p.batch;
        while (hi - lo > 256) {
            const int step = (hi - lo + 31) / 32;
            const int i = lo + lane * step;
            const bool le = i < hi && p.cu_tokens[i] / P + 2 * i <= u;
            const unsigned m = __ballot_sync(0xffffffffu, le);
            const int k = m ? 31 - __clz(static_cast<int>(m)) : 0;
            lo += k * step;
            hi = min(hi, lo + step);
        }
        int le = 0;                                    // the last 256 at once, 8 per lane
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = lo + 8 * lane + j;
            le += i < hi && p.cu_tokens[i] / P + 2 * i <= u;
        }
        b = lo + max(0, static_cast<int>(__reduce_add_sync(0xffffffffu, le)) - 1);
        first = p.cu_tokens[b];
        const int end = p.cu_tokens[b + 1];
        local = u - (first / P + 2 * b);
        if (first < 0 || end < first || end > p.num_tokens) {
            if (lane == 0) flag_status(p.status, AQ_DEV_BAD_LENGTH);
            return w;
        }
        n = end - first;
        if (n == 0 || local < 0) return w;
    }
    const int L = p.seq_lens[b];
    const int64_t start = static_cast<int64_t>(L) - n;
    const bool long_ = L < 0 || start < 0 || L > static_cast<int64_t>(p.max_pages) * P;
    const int p0 = long_ ? 0 : static_cast<int>(start / P);
    const int np = long_ ? (n + P - 1) / P : (L - 1) / P + 1 - p0;
    if (local >= np) return w;
    if (long_) {                                       // no place in the cache: its rows in pieces of 16
        if (lane == 0) flag_status(p.status, AQ_DEV_BAD_LENGTH);
        w.n = min(P, n - local * P);
        w.row = first + static_cast<int64_t>(local) * P;
        return w;
    }
    const int64_t at = static_cast<int64_t>(p0 + local) * P;
    w.s0 = static_cast<int>(max(start, at) - at);
    w.n = static_cast<int>(min(static_cast<int64_t>(L) - at, static_cast<int64_t>(P))) - w.s0;
    w.row = first + (at + w.s0 - start);
    w.page = p.block_table[static_cast<size_t>(b) * p.max_pages + p0 + local];
    return w;
}

// Whether the unit's page is one of the pool's; flags one that is not.
__device__ __forceinline__ bool page_ok(const Q8CacheParams &p, const Unit &w, int lane) {
    const bool ok = w.page >= 0 && w.page < p.num_pages;
    if (!ok && w.page != kNoPage && lane == 0) flag_status(p.status, AQ_DEV_BAD_PAGE);
    return ok;
}

// ROWS: the most rows that a block gets from the call.  16: a warp per head and K or V,
// 4 dims per lane (16 rows of 8 dims would hold 122 registers and half the warps: 45 us
// against 37 us for the 5 prompts above).  1, a decode step's single tokens: lanes 0-15 a
// head's key row, lanes 16-31 its value row, 8 dims each (5.0 us against 6.1 us for 256).
template <int FMT, int ROWS>
__global__ void __launch_bounds__(kThreads, ROWS == 1 ? 6 : 4) q8_append_kernel(const __grid_constant__ Q8CacheParams p) {
    constexpr int D = kHeadDim, P = kPage;
    constexpr int DL = ROWS == 1 ? 8 : 4, LANES = D / DL, W = DL / 4;      // dims per lane, lanes per row, words of codes
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LANES;
    const Unit w = find_unit(p, blockIdx.x, lane);
    const int n = w.n, pairs = 2 * p.num_kv_heads;
    if (n == 0 || w.page == kNoPage) return;
    const size_t row = static_cast<size_t>(pairs) * D;
    for (int hp = (blockIdx.y * kWarps + warp) * W + lane / LANES; hp < pairs; hp += gridDim.y * kWarps * W) {
        const __half *src = p.kv + static_cast<size_t>(w.row) * row + static_cast<size_t>(hp) * D + DL * sub;
        uint2 x[ROWS][W];
        uint32_t top = 0;                              // largest |half| bits of each 16-bit lane
#pragma unroll
        for (int s = 0; s < ROWS; ++s) {
#pragma unroll
            for (int j = 0; j < W; ++j) x[s][j] = make_uint2(0u, 0u);
            if (s < n) load_row(src + s * row, x[s]);
        }
        if (!page_ok(p, w, lane)) return;              // (the rows were on their way meanwhile)
        const size_t block = static_cast<size_t>(w.page) * pairs + hp;
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.pages + block * (P * D)) + W * sub;
        const float old = w.s0 > 0 ? p.scales[block] : 0.f;
#pragma unroll
        for (int s = 0; s < ROWS; ++s)
#pragma unroll
            for (int j = 0; j < W; ++j)
                top = __vmaxu2(top, __vmaxu2(x[s][j].x & 0x7fff7fffu, x[s][j].y & 0x7fff7fffu));
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int off = 1; off < LANES; off *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        // a block that holds a non-finite value is NaN as a whole (codes 0)
        const float want = top >= 0x7c00u ? __int_as_float(0x7fc00000)
                                          : scale_for<FMT>(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
        const float scale = old != old ? old : (want > old || want != want) ? want : old;
        if (w.s0 > 0 && scale != old && old == old) {  // earlier tokens of the block, under the grown scale
            // four rows under way together; rolled, so that its code does not crowd out the rest
#pragma unroll 1
            for (int s = 0; s < w.s0; s += 4) {
                uint32_t c[4][W];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < W; ++j) c[k][j] = s + k < w.s0 ? dst[(s + k) * (D / 4) + j] : 0u;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (s + k < w.s0) dst[(s + k) * (D / 4) + j] = rescale4<FMT>(c[k][j], old, scale);
            }
        }
        const Encoder enc = encoder_of<FMT>(scale);
        dst += w.s0 * (D / 4);
        uint32_t redo = 0;
#pragma unroll
        for (int s = 0; s < ROWS; ++s) {
            if (s < n) {
                uint32_t c[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    bool again;
                    c[j] = encode4<FMT>(halves(x[s][j]), enc, again);
                    redo |= again ? 1u << s : 0u;
                }
                store_codes(dst + s * (D / 4), c);
            }
        }
        while (redo) {                                 // few rows, if any: fetched again, decided exactly
            const int s = __ffs(redo) - 1;
            redo &= redo - 1;
            uint2 y[W];
            load_row(src + s * row, y);
#pragma unroll
            for (int j = 0; j < W; ++j) dst[s * (D / 4) + j] = encode4_exact<FMT>(halves(y[j]), scale);
        }
        if (sub == 0 && (w.s0 == 0 || scale != old)) p.scales[block] = scale;
    }
}

// The read-back: lanes 0-15 a head's key rows, lanes 16-31 its value rows, 8 dims each, so
// that a token's row is 512 contiguous bytes (against 256 and 4 dims per lane: 34 us
// against 41 us for the same prompts, 14 us against 19 us for the step's blocks).
template <int FMT>
__global__ void __launch_bounds__(kThreads, 4) q8_load_kernel(const __grid_constant__ Q8CacheParams p) {
    constexpr int D = kHeadDim, P = kPage;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Unit w = find_unit(p, blockIdx.x, lane);
    const int n = w.n;
    if (n == 0) return;
    const bool bad = !page_ok(p, w, lane);
    const size_t row = static_cast<size_t>(p.num_kv_heads) * 2 * D;
    for (int h = blockIdx.y * kWarps + warp; h < p.num_kv_heads; h += gridDim.y * kWarps) {
        __half *dst = p.kv + static_cast<size_t>(w.row) * row + static_cast<size_t>(h) * 2 * D + 8 * lane;
        const size_t block = (static_cast<size_t>(bad ? 0 : w.page) * p.num_kv_heads + h) * 2 + (lane >> 4);
        const float scale = bad ? __int_as_float(0x7fc00000) : p.scales[block];
        const uint8_t *src = p.pages + block * (P * D) + w.s0 * D + 8 * (lane & 15);
        uint2 c[P];
#pragma unroll
        for (int s = 0; s < P; ++s) {
            c[s] = make_uint2(0u, 0u);
            if (!bad && s < n) c[s] = ld_global_na_v2(src + s * D);
        }
#pragma unroll
        for (int s = 0; s < P; ++s) {
            if (s < n) {
                uint32_t v[4], r[4];
                widen4<FMT>(c[s].x, v[0], v[1]);
                widen4<FMT>(c[s].y, v[2], v[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = h2_to_f2(v[j]);
                    const __half2 h2 = __floats2half2_rn(a.x * scale, a.y * scale);
                    r[j] = *reinterpret_cast<const uint32_t *>(&h2);
                }
                *reinterpret_cast<uint4 *>(dst + s * row) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
    }
}

aq_status q8_cache_call(bool append, const aq_pq_config *cfg, int32_t format, int32_t batch, int32_t num_tokens,
                        int32_t num_kv_heads, const void *kv, void *code_pages, float *page_scales,
                        int64_t num_pages, const int32_t *block_table, int32_t max_pages, const int32_t *seq_lens,
                        const int32_t *cu_tokens, int32_t *device_status, aq_stream_t stream) {
    if (!cfg || cfg->head_dim <= 0 || cfg->page_size <= 0) return AQ_ERR_INVALID_ARGUMENT;
    if (cfg->head_dim != kHeadDim || cfg->page_size != kPage) return AQ_ERR_UNSUPPORTED;
    if (format != AQ_Q8_INT8 && format != AQ_Q8_E4M3) return AQ_ERR_INVALID_ARGUMENT;
    if (batch < 0 || num_tokens < 0 || num_kv_heads < 1 || num_pages < 0 || max_pages < 0) return AQ_ERR_INVALID_ARGUMENT;
    if (!cu_tokens && num_tokens != batch) return AQ_ERR_INVALID_ARGUMENT;
    if (num_kv_heads > 65535 || batch > 65535) return AQ_ERR_UNSUPPORTED;
    if (batch == 0 || num_tokens == 0) return AQ_OK;
    if (!kv || !code_pages || !page_scales || !block_table || !seq_lens) return AQ_ERR_INVALID_ARGUMENT;
    auto off16 = [](const void *a) { return (reinterpret_cast<uintptr_t>(a) & 15u) != 0; };
    if (off16(kv) || off16(code_pages) || off16(page_scales)) return AQ_ERR_INVALID_ARGUMENT;
    Q8CacheParams p{};
    p.kv = static_cast<__half *>(const_cast<void *>(kv));
    p.pages = static_cast<uint8_t *>(code_pages);
    p.scales = page_scales;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.cu_tokens = cu_tokens;
    p.status = device_status;
    p.num_pages = num_pages;
    p.batch = batch;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.max_pages = max_pages;
    const unsigned units = cu_tokens ? static_cast<unsigned>(num_tokens / kPage) + 2u * batch + 1u
                                     : static_cast<unsigned>(batch);
    // a unit's heads over several CTAs only as far as that fills the GPU (6 CTAs per SM,
    // twice): a CTA's first loads depend on one another, its heads' do not.  (The 5
    // prompts' append and the step's read-back: 37.5 and 14.2 us; filled once 38.7 and
    // 15.1, four times 40.2 and 15.2)
    const int warps = append && cu_tokens ? 2 * num_kv_heads : num_kv_heads;
    unsigned split = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
    if (split > 2u * 6u * 152u / units + 1u) split = 2u * 6u * 152u / units + 1u;
    const dim3 grid(units, split);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool int8 = format == AQ_Q8_INT8;
    auto kern = !append      ? (int8 ? q8_load_kernel<kInt8> : q8_load_kernel<kE4m3>)
                : cu_tokens ? (int8 ? q8_append_kernel<kInt8, kPage> : q8_append_kernel<kE4m3, kPage>)
                            : (int8 ? q8_append_kernel<kInt8, 1> : q8_append_kernel<kE4m3, 1>);
    const cudaError_t e = launch_dependent(kern, grid, dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess) return AQ_OK;
    record_cuda_error(e);
    return AQ_ERR_CUDA;
}

}  // namespace

}  // namespace aq

using namespace aq;

extern "C" {

aq_status aq_q8_append(const aq_pq_config *cfg, int32_t format, int32_t batch, int32_t num_tokens,
                       int32_t num_kv_heads, const void *kv_f16, void *code_pages, float *page_scales,
                       int64_t num_pages, const int32_t *block_table, int32_t max_pages, const int32_t *seq_lens,
                       const int32_t *cu_tokens, int32_t *device_status, aq_stream_t stream) {
    return q8_cache_call(true, cfg, format, batch, num_tokens, num_kv_heads, kv_f16, code_pages, page_scales,
                         num_pages, block_table, max_pages, seq_lens, cu_tokens, device_status, stream);
}

aq_status aq_q8_load(const aq_pq_config *cfg, int32_t format, int32_t batch, int32_t num_tokens,
                     int32_t num_kv_heads, void *kv_f16, const void *code_pages, const float *page_scales,
                     int64_t num_pages, const int32_t *block_table, int32_t max_pages, const int32_t *seq_lens,
                     const int32_t *cu_tokens, int32_t *device_status, aq_stream_t stream) {
    return q8_cache_call(false, cfg, format, batch, num_tokens, num_kv_heads, kv_f16, const_cast<void *>(code_pages),
                         const_cast<float *>(page_scales), num_pages, block_table, max_pages, seq_lens, cu_tokens,
                         device_status, stream);
}

}  // extern "C"
