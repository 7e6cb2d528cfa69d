// q8_attention.cu -- decode attention over the 8-bit block-scaled cache:
//   s_t = scale * kscale(page of t) * (q . kcode_t),   p = softmax(s),
//   out = sum_t p_t * vscale(page of t) * vcode_t      (PAM article §2.2.3 for
// the blockwise softmax whose (max, sum, output) partials merge over splits).
//
// Both products run on warp-level tensor-core tiles (m16n8k16, fp16 operands,
// fp32 accumulators).  An 8-bit code is exact in fp16.  The fp32 operand of
// each product is split into a rounded fp16 part and the rounded remainder (22
// bits); the tile's 16 rows hold the 8 query heads of a group twice, high parts
// in rows 0-7 and remainders in rows 8-15, so one instruction multiplies both
// and a group of up to 8 heads costs no more than one head.
//
// A warp takes whole pages.  The contraction order of a tile is free as long
// as both operands agree, so every lane reads 16-byte pieces of rows straight
// from the page: lane (r, c) = (lane / 4, lane % 4) reads keys 8 t + r, bytes
// [16 c, 16 c + 16) and [64 + 16 c, ...) -- 32 dims, two per register pair --
// and values of tokens 2c, 2c + 1, 2c + 8, 2c + 9, bytes [16 r, 16 r + 16),
// interleaved token by token.  The score tile leaves lane (r, c) with head r's
// scores of tokens 8 t + 2 c + {0, 1}, which is what the value product wants.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "q8_common.cuh"

namespace aq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 8;              // query heads of a tile
constexpr float kWeightTop = 32768.f;  // weights enter the fp16 product as p * 2^15

struct Q8AttnParams {
    const float *q;                // [B][Hq][D]
    const uint8_t *pages;          // [NP][Hkv][2][P][D]
    const float *scales;           // [NP][Hkv][2]
    const int32_t *block_table;    // [B][max_pages]
    const int32_t *seq_lens;       // [B]
    float *out;                    // [B][Hq][D]
    float *part_o;                 // [B][Hq][S][D]
    float *part_ml;                // [B][Hq][S][2]
    int32_t *status;
    int64_t num_pages;
    int32_t num_q_heads, num_kv_heads, group, chunks, max_pages, max_seq_len, num_splits;
    int64_t split_len;             // tokens, a multiple of P
    float scale_log2;
};

__device__ __forceinline__ uint4 ldg_page(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Column pairs of two tokens' words: byte i of a and of b as one fp16 pair.
template <int FMT>
__device__ __forceinline__ void pair4(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
    const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
    widen4<FMT>(x, h[0], h[1]);
    widen4<FMT>(y, h[2], h[3]);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) q8_attention_kernel(const __grid_constant__ Q8AttnParams p) {
    constexpr int D = kHeadDim, P = kPage;
    __shared__ float wm[kWarps][kGroup], wl[kWarps][kGroup];
    __shared__ __align__(16) float wacc[kWarps][kGroup][D];
    __shared__ int sbad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int split = blockIdx.x, kvh = blockIdx.y / p.chunks, chunk = blockIdx.y % p.chunks, b = blockIdx.z;
    const int heads = min(kGroup, p.group - chunk * kGroup);
    const size_t bh0 = static_cast<size_t>(b) * p.num_q_heads + static_cast<size_t>(kvh) * p.group + chunk * kGroup;
    const int S_ = p.num_splits;
    const float nan = __int_as_float(0x7fc00000);

    const int L = p.seq_lens[b];
    const bool badlen = L < 0 || L > static_cast<int64_t>(p.max_pages) * P || L > p.max_seq_len;
    const int64_t ts64 = static_cast<int64_t>(split) * p.split_len;
    const int te = badlen ? 0 : static_cast<int>(min(static_cast<int64_t>(L), ts64 + p.split_len));
    if (badlen || ts64 >= te) {
        if (badlen && tid == 0) flag_status(p.status, AQ_DEV_BAD_LENGTH);
        for (int i = tid; i < heads * D; i += kThreads) {
            const size_t bh = bh0 + i / D;
            if (S_ == 1) p.out[bh * D + i % D] = badlen ? nan : 0.f;
            else if (i % D == 0) {
                p.part_ml[(bh * S_ + split) * 2] = badlen ? nan : -INFINITY;
                p.part_ml[(bh * S_ + split) * 2 + 1] = badlen ? nan : 0.f;
            }
        }
        return;
    }
    const int ts = static_cast<int>(ts64);
    if (tid == 0) sbad = 0;

    // the query of head r: lane c's 32 dims, scaled by a power of two to
    // [2^13, 2^14) at its largest magnitude, as fp16 parts
    uint32_t qa[8][4];
    float qinv;
    {
        float4 x[8];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < heads)
                x[j] = *reinterpret_cast<const float4 *>(p.q + (bh0 + r) * D + (j / 4) * 64 + c * 16 + (j % 4) * 4);
            top = fmaxf(fmaxf(fmaxf(top, fabsf(x[j].x)), fmaxf(fabsf(x[j].y), fabsf(x[j].z))), fabsf(x[j].w));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(253, max(1, 267 - static_cast<int>(__float_as_uint(top) >> 23)));
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        qinv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23) * p.scale_log2;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f16x2_split(x[j].x * up, x[j].y * up, qa[j][0], qa[j][1]);
            f16x2_split(x[j].z * up, x[j].w * up, qa[j][2], qa[j][3]);
        }
    }
    float m = -INFINITY, l = 0.f, vref = 0.f;
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    __syncthreads();

    const int32_t *bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const int pg1 = (te + P - 1) / P;
    bool badpage = false;
#pragma unroll 1
    for (int pi = ts / P + warp; pi < pg1; pi += kWarps) {
        const int pg = bt[pi];
        if (pg < 0 || pg >= p.num_pages) {
            badpage = true;
            continue;
        }
        const size_t block = (static_cast<size_t>(pg) * p.num_kv_heads + kvh) * 2;
        const uint8_t *base = p.pages + block * (P * D);
        uint4 k[2][2], v[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) k[t][i] = ldg_page(base + (8 * t + r) * D + 64 * i + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ldg_page(base + P * D + (2 * c + (i & 1) + 8 * (i >> 1)) * D + 16 * r);
        const float2 sc = __ldg(reinterpret_cast<const float2 *>(p.scales + block));
        const int n = min(P, te - pi * P);

        float s[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t b0, b1;
                widen4<FMT>(word(k[t][j / 4], j % 4), b0, b1);
                mma_16816(d, qa[j], b0, b1);
            }
            const float f = qinv * sc.x;
            s[t][0] = 8 * t + 2 * c < n ? (d[0] + d[2]) * f : -INFINITY;
            s[t][1] = 8 * t + 2 * c + 1 < n ? (d[1] + d[3]) * f : -INFINITY;
        }
        float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx, m);
        // the frame of the value sums: 2^-15 of a power of two >= every value scale seen
        const float vtop = __uint_as_float((__float_as_uint(sc.y) + 0x7fffffu) & 0x7f800000u);
        const float vnew = sc.y > vref ? vtop : vref;
        if (__any_sync(0xffffffffu, mx > m || vnew != vref)) {
            const float a = mx == -INFINITY ? 1.f : fast_exp2(m - mx);
            l *= a;
            const float av = vref > 0.f ? a * (vref / vnew) : 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                o[j][0] *= av;
                o[j][1] *= av;
                o[j][2] *= av;
                o[j][3] *= av;
            }
            m = mx;
            vref = vnew;
        }
        const float vw = vref > 0.f ? kWeightTop * (sc.y / vref) : sc.y;
        uint32_t pa[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float p0 = fast_exp2(s[t][0] - m), p1 = fast_exp2(s[t][1] - m);
            l += p0 + p1;
            f16x2_split(p0 * vw, p1 * vw, pa[2 * t], pa[2 * t + 1]);
        }
        if (FMT == kE4m3 && n < P) {                   // slots behind the last token may hold NaN codes
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (2 * c + (i & 1) + 8 * (i >> 1) >= n) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t b0[4], b1[4];
            pair4<FMT>(word(v[0], w), word(v[1], w), b0);
            pair4<FMT>(word(v[2], w), word(v[3], w), b1);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_16816(o[4 * w + j], pa, b0[j], b1[j]);
        }
    }
    if (badpage) atomicOr(&sbad, AQ_DEV_BAD_PAGE);

    // ---- merge the warps ------------------------------------------------------
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c == 0) {
        wm[warp][r] = m;
        wl[warp][r] = l;
    }
    const float back = vref * (1.f / kWeightTop);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        wacc[warp][r][32 * c + j] = (o[j][0] + o[j][2]) * back;
        wacc[warp][r][32 * c + 16 + j] = (o[j][1] + o[j][3]) * back;
    }
    __syncthreads();
    const int bad = sbad;
    if (bad && tid == 0) flag_status(p.status, bad);
    for (int i = tid; i < heads * D; i += kThreads) {
        const int g = i / D, d = i % D;
        float ms = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ms = fmaxf(ms, wm[w][g]);
        float num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (wm[w][g] > -INFINITY || wl[w][g] != wl[w][g]) {
                const float f = exp2f(wm[w][g] - ms);
                den += f * wl[w][g];
                num += f * wacc[w][g][d];
            }
        }
        const size_t bh = bh0 + g;
        if (S_ == 1) {
            p.out[bh * D + d] = bad ? nan : num / den;
        } else {
            p.part_o[(bh * S_ + split) * D + d] = num;
            if (d == 0) {
                p.part_ml[(bh * S_ + split) * 2] = bad ? nan : ms;
                p.part_ml[(bh * S_ + split) * 2 + 1] = bad ? nan : den;
            }
        }
    }
}

// out = sum over splits of 2^(m - max) o, over the same sum of l: one CTA per
// (request, query head), one thread per dim.
__global__ void __launch_bounds__(kHeadDim) q8_combine_kernel(const __grid_constant__ Q8AttnParams p) {
    const size_t bh = static_cast<size_t>(blockIdx.y) * p.num_q_heads + blockIdx.x;
    const int S_ = p.num_splits, d = threadIdx.x;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + bh * S_;
    const float *po = p.part_o + bh * S_ * kHeadDim + d;
    float ms = -INFINITY;
    bool nan = false;
    for (int s = 0; s < S_; ++s) {
        const float2 x = ml[s];
        nan |= x.y != x.y;
        if (x.y > 0.f) ms = fmaxf(ms, x.x);
    }
    float num = 0.f, den = 0.f;
    for (int s = 0; s < S_; ++s) {
        const float2 x = ml[s];
        if (x.y > 0.f) {
            const float f = exp2f(x.x - ms);
            den += f * x.y;
            num += f * po[static_cast<size_t>(s) * kHeadDim];
        }
    }
    p.out[bh * kHeadDim + d] = nan ? __int_as_float(0x7fc00000) : den > 0.f ? num / den : 0.f;
}

// Splits of a call (host arithmetic): enough CTAs for the GPU, at least 256
// tokens each.
struct Q8Plan {
    int32_t num_splits;
    int64_t split_len;
    size_t workspace;
};

Q8Plan q8_plan(int64_t batch, int64_t Hq, int64_t Hkv, int32_t max_seq_len, int32_t req) {
    const int64_t G = Hq / Hkv, units = batch * Hkv * ((G + kGroup - 1) / kGroup);
    const int64_t pages = (static_cast<int64_t>(max_seq_len) + kPage - 1) / kPage;
    int64_t S = req;
    if (S <= 0) {
        const int64_t want = units > 0 ? (4 * 152 + units - 1) / units : 1, most = max_seq_len / 256;
        S = want < most ? want : most;
    }
    if (S > 4096) S = 4096;
    if (S > pages) S = pages;
    if (S < 1) S = 1;
    const int64_t len = pages > 0 ? (pages + S - 1) / S : 1;
    S = pages > 0 ? (pages + len - 1) / len : 1;
    Q8Plan pl{};
    pl.num_splits = static_cast<int32_t>(S);
    pl.split_len = len * kPage;
    pl.workspace = S > 1 ? static_cast<size_t>(batch) * Hq * S * (kHeadDim + 2) * sizeof(float) : 0;
    return pl;
}

aq_status check_q8(const aq_pq_config *cfg, int32_t batch, int32_t Hq, int32_t Hkv, int32_t max_seq_len,
                   int32_t num_splits) {
    if (!cfg || cfg->head_dim <= 0 || cfg->page_size <= 0) return AQ_ERR_INVALID_ARGUMENT;
    if (cfg->head_dim != kHeadDim || cfg->page_size != kPage) return AQ_ERR_UNSUPPORTED;
    if (batch < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_seq_len < 0 || num_splits < 0)
        return AQ_ERR_INVALID_ARGUMENT;
    if (batch > 65535 || static_cast<int64_t>(Hkv) * ((Hq / Hkv + kGroup - 1) / kGroup) > 65535) return AQ_ERR_UNSUPPORTED;
    return AQ_OK;
}

}  // namespace

}  // namespace aq

using namespace aq;

extern "C" {

aq_status aq_q8_decode_plan(const aq_pq_config *cfg, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t max_seq_len, int32_t num_splits_req, int32_t *num_splits,
                            size_t *workspace_bytes) {
    const aq_status st = check_q8(cfg, batch, num_q_heads, num_kv_heads, max_seq_len, num_splits_req);
    if (st != AQ_OK) return st;
    const Q8Plan pl = q8_plan(batch, num_q_heads, num_kv_heads, max_seq_len, num_splits_req);
    if (num_splits) *num_splits = pl.num_splits;
    if (workspace_bytes) *workspace_bytes = pl.workspace;
    return AQ_OK;
}

aq_status aq_q8_decode_attention(const aq_pq_config *cfg, int32_t format, int32_t batch, int32_t num_q_heads,
                                 int32_t num_kv_heads, const float *q, const void *code_pages,
                                 const float *page_scales, int64_t num_pages, const int32_t *block_table,
                                 int32_t max_pages, const int32_t *seq_lens, int32_t max_seq_len, float scale,
                                 int32_t num_splits, float *out, void *workspace, size_t workspace_bytes,
                                 int32_t *device_status, aq_stream_t stream) {
    const aq_status st = check_q8(cfg, batch, num_q_heads, num_kv_heads, max_seq_len, num_splits);
    if (st != AQ_OK) return st;
    if (format != AQ_Q8_INT8 && format != AQ_Q8_E4M3) return AQ_ERR_INVALID_ARGUMENT;
    if (max_pages < 0 || num_pages < 0 || !std::isfinite(scale)) return AQ_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_pages) * kPage) return AQ_ERR_INVALID_ARGUMENT;
    if (batch == 0) return AQ_OK;
    if (!q || !code_pages || !page_scales || !block_table || !seq_lens || !out) return AQ_ERR_INVALID_ARGUMENT;
    auto off16 = [](const void *a) { return (reinterpret_cast<uintptr_t>(a) & 15u) != 0; };
    if (off16(q) || off16(code_pages) || off16(page_scales) || off16(out) || off16(workspace))
        return AQ_ERR_INVALID_ARGUMENT;
    const Q8Plan pl = q8_plan(batch, num_q_heads, num_kv_heads, max_seq_len, num_splits);
    if (pl.workspace > 0 && (!workspace || workspace_bytes < pl.workspace)) return AQ_ERR_WORKSPACE_TOO_SMALL;
    Q8AttnParams p{};
    p.q = q;
    p.pages = static_cast<const uint8_t *>(code_pages);
    p.scales = page_scales;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.out = out;
    if (pl.num_splits > 1) {
        p.part_o = static_cast<float *>(workspace);
        p.part_ml = p.part_o + static_cast<size_t>(batch) * num_q_heads * pl.num_splits * kHeadDim;
    }
    p.status = device_status;
    p.num_pages = num_pages;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.chunks = (p.group + kGroup - 1) / kGroup;
    p.max_pages = max_pages;
    p.max_seq_len = max_seq_len;
    p.num_splits = pl.num_splits;
    p.split_len = pl.split_len;
    p.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(pl.num_splits), static_cast<unsigned>(num_kv_heads * p.chunks),
                    static_cast<unsigned>(batch));
    if (format == AQ_Q8_INT8) q8_attention_kernel<kInt8><<<grid, kThreads, 0, s>>>(p);
    else q8_attention_kernel<kE4m3><<<grid, kThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && pl.num_splits > 1) {
        q8_combine_kernel<<<dim3(static_cast<unsigned>(num_q_heads), static_cast<unsigned>(batch)), kHeadDim, 0, s>>>(p);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) return AQ_OK;
    record_cuda_error(e);
    return AQ_ERR_CUDA;
}

}  // extern "C"
