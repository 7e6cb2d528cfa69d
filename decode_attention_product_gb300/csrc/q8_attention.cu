// q8_attention.cu -- decode attention over the 8-bit block-scaled cache:
//   s_t = scale * kscale(page of t) * (q . kcode_t),   p = softmax(s),
//   out = sum_t p_t * vscale(page of t) * vcode_t      (PAM article §2.2.3 for
// the blockwise softmax whose (max, sum, output) partials merge over splits).
//
// Both products run on warp-level tensor-core tiles (m16n8k16, fp16 operands,
// fp32 accumulators): a group of at most 8 query heads is the 8-column operand,
// far too narrow for a 128-row tcgen05 tile, and the 8-bit codes have to be
// widened in registers anyway.  A code is exact in fp16.  The fp32 operand of each
// product (queries, weights) is split into a rounded fp16 part and the rounded
// remainder, 22 bits together, and both parts multiply into one accumulator.
//
// A page of one kv head is 4 KiB in one piece, keys then values: one TMA copy
// per page into the warp's own ring of kStages pages.  A warp takes whole pages
// and keeps its own running (max, sum, output); no other warp is waited for
// until the end.  The copy swizzles 16-byte chunk i of row t to i ^ (t % 8), which
// leaves every 16-byte shared load below free of bank conflicts.
//
// The contraction order of a tile is free as long as both operands agree, so a
// lane (r, c) = (lane / 4, lane % 4) takes whole 16-byte chunks:
//   scores   16 tokens x 8 heads: rows r, r + 8, dims [32 c, 32 c + 32) of the keys;
//            lane (r, c) gets tokens r, r + 8 of heads 2 c, 2 c + 1
//   values   16 dims x 8 heads, 8 tiles: dims [16 r, 16 r + 16) of tokens 2 c, 2 c + 1,
//            2 c + 8, 2 c + 9; the weights reach the other operand's layout by
//            8x8 transposes of register tiles
//
// The splits of a (request, kv head) are the CTAs of a cluster, up to 8: their
// results merge through distributed shared memory, in one launch and without
// workspace.  More splits (few, very long requests) go through partials.
#include <cudaTypedefs.h>

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "q8_common.cuh"

namespace aq {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;             // pages in a warp's ring
constexpr int kGroup = 8;              // query heads of a tile
constexpr int kMaxCluster = 8;
constexpr int kPageBytes = 2 * kPage * kHeadDim;
constexpr float kWeightTop = 32768.f;  // weights enter the fp16 product as p * 2^15
constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kStages * kPageBytes + 1024;

struct Q8AttnParams {
    CUtensorMap map;               // code pages as [NP * Hkv][32 rows][128 bytes], 128-byte swizzle
    const float *q;                // [B][Hq][D]
    const float *scales;           // [NP][Hkv][2]
    const int32_t *block_table;    // [B][max_pages]
    const int32_t *seq_lens;       // [B]
    float *out;                    // [B][Hq][D]
    float *part_o;                 // [B][Hq][S][D]
    float *part_ml;                // [B][Hq][S][2]
    int32_t *status;
    int64_t num_pages;
    unsigned long long wait_limit_ns;
    int32_t num_q_heads, num_kv_heads, group, chunks, max_pages, max_seq_len, num_splits, cluster;
    float scale_log2;
};

// One page to shared memory, counted in bytes on `bar`.
__device__ __forceinline__ void tma_page(void *dst, const CUtensorMap *map, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3}], [%4];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Transpose of an 8x8 fp16 tile held as (row lane / 4, columns 2 (lane % 4) + {0, 1}).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Byte i of two tokens' words as one fp16 pair, i = 0 .. 3.
template <int FMT>
__device__ __forceinline__ void pair4(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
    const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
    widen4<FMT>(x, h[0], h[1]);
    widen4<FMT>(y, h[2], h[3]);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 4) q8_attention_kernel(const __grid_constant__ Q8AttnParams p) {
    constexpr int D = kHeadDim, P = kPage;
    extern __shared__ unsigned char ring_raw[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ float wm[kWarps][kGroup], wl[kWarps][kGroup];
    __shared__ __align__(16) float co[kGroup][D];          // this CTA's sums, read by the cluster
    __shared__ float cm[kGroup], cl[kGroup];
    __shared__ int cbad;
    // the ring starts on the swizzle's period
    unsigned char *ring = ring_raw + ((1024u - (smem_u32(ring_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int split = blockIdx.x, kvh = blockIdx.y / p.chunks, chunk = blockIdx.y % p.chunks, b = blockIdx.z;
    const int heads = min(kGroup, p.group - chunk * kGroup);
    const size_t bh0 = static_cast<size_t>(b) * p.num_q_heads + static_cast<size_t>(kvh) * p.group + chunk * kGroup;
    const int S_ = p.num_splits;
    const float nan = __int_as_float(0x7fc00000);

    // the request's pages, shared out evenly over its splits
    const int L = p.seq_lens[b];
    const bool badlen = L < 0 || L > static_cast<int64_t>(p.max_pages) * P || L > p.max_seq_len;
    const int np = badlen ? 0 : (L + P - 1) / P;
    const int pg0 = static_cast<int>(static_cast<int64_t>(np) * split / S_);
    const int pg1 = static_cast<int>(static_cast<int64_t>(np) * (split + 1) / S_);
    const int mine = pg1 - pg0 > warp ? (pg1 - pg0 - warp + kWarps - 1) / kWarps : 0;      // pg0 + warp, + kWarps, ...
    const int32_t *bt = p.block_table + static_cast<size_t>(b) * p.max_pages + pg0 + warp;
    unsigned char *stage = ring + static_cast<size_t>(warp) * kStages * kPageBytes;

    // page ids (-1: outside the pool) and scales of the warp's pages [k, k + 32), one per lane
    auto page_id = [&](int k) {
        const int pg = k < mine ? bt[static_cast<size_t>(k) * kWarps] : -1;
        return pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    auto page_scales = [&](int pg) {
        return pg >= 0 ? __ldg(reinterpret_cast<const float2 *>(p.scales) + static_cast<size_t>(pg) * p.num_kv_heads + kvh)
                       : make_float2(0.f, 0.f);
    };
    int id = page_id(lane);
    if (tid == 0) cbad = badlen ? AQ_DEV_BAD_LENGTH : 0;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&bars[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    // page k into its ring slot (lane 0); a page outside the pool only arrives
    auto issue = [&](int k, int pg) {
        if (lane == 0) {
            uint64_t *bar = &bars[warp][k % kStages];
            if (pg >= 0) {
                mbar_arrive_expect_tx(bar, kPageBytes);
                tma_page(stage + (k % kStages) * kPageBytes, &p.map, pg * p.num_kv_heads + kvh, bar);
            } else {
                mbar_arrive(bar);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
        const int pg = __shfl_sync(0xffffffffu, id, k);
        if (k < mine) issue(k, pg);
    }
    float2 sc = page_scales(id);
    int next_id = mine > 32 ? page_id(32 + lane) : -1;

    // the query of head r: this lane's 32 dims, scaled by a power of two to
    // [2^13, 2^14) at its largest magnitude, as fp16 parts
    uint32_t qh[8][2], ql[8][2];
    float qs0, qs1;                                    // what undoes it, with the softmax scale: heads 2c, 2c + 1
    {
        float4 x[8];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < heads) x[j] = *reinterpret_cast<const float4 *>(p.q + (bh0 + r) * D + 32 * c + 4 * j);
            top = fmaxf(fmaxf(fmaxf(top, fabsf(x[j].x)), fmaxf(fabsf(x[j].y), fabsf(x[j].z))), fabsf(x[j].w));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(253, max(1, 267 - static_cast<int>(__float_as_uint(top) >> 23)));
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23) * p.scale_log2;
        qs0 = __shfl_sync(0xffffffffu, down, 8 * c);
        qs1 = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f16x2_split(x[j].x * up, x[j].y * up, qh[j][0], ql[j][0]);
            f16x2_split(x[j].z * up, x[j].w * up, qh[j][1], ql[j][1]);
        }
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, vref = 0.f;
    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    int bad = 0, k = 0;

#pragma unroll 1
    for (; k < mine; ++k) {
        if (k && (k & 31) == 0) {                      // the next 32 pages' ids were fetched 32 pages ago
            id = next_id;
            sc = page_scales(id);
            next_id = page_id(k + 32 + lane);
        }
        const int pg = __shfl_sync(0xffffffffu, id, k & 31);
        const float ks = __shfl_sync(0xffffffffu, sc.x, k & 31), vs = __shfl_sync(0xffffffffu, sc.y, k & 31);
        uint64_t *bar = &bars[warp][k % kStages];
        const uint32_t phase = (k / kStages) & 1;
        bool ok = mbar_test_wait(bar, phase);
        if (!ok && p.wait_limit_ns) ok = mbar_wait_limit(bar, phase, p.wait_limit_ns);
        if (!__all_sync(0xffffffffu, ok)) {
            bad |= AQ_DEV_TIMEOUT;
            break;
        }
        const unsigned char *base = stage + (k % kStages) * kPageBytes;
        uint4 kr[2][2], v[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                kr[t][i] = *reinterpret_cast<const uint4 *>(base + (8 * t + r) * D + (((2 * c + i) ^ r) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * c + (i & 1) + 8 * (i >> 1);
            v[i] = *reinterpret_cast<const uint4 *>(base + (P + t) * D + ((r ^ (t & 7)) << 4));
        }
        // every lane has read the slot: refill it
        __syncwarp();
        {
            const int n = k + kStages;
            const int from = __shfl_sync(0xffffffffu, (n ^ k) & 32 ? next_id : id, n & 31);
            if (n < mine) issue(n, from);
        }
        if (pg < 0) {
            bad |= AQ_DEV_BAD_PAGE;
            continue;
        }
        const int n = min(P, L - (pg0 + warp + k * kWarps) * P);

        float d[2][4] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t a[4];
            widen4<FMT>(word(kr[0][j / 4], j % 4), a[0], a[2]);
            widen4<FMT>(word(kr[1][j / 4], j % 4), a[1], a[3]);
            mma_16816(d[0], a, qh[j][0], qh[j][1]);
            mma_16816(d[1], a, ql[j][0], ql[j][1]);
        }
        const float f0 = qs0 * ks, f1 = qs1 * ks;
        const float s00 = r < n ? (d[0][0] + d[1][0]) * f0 : -INFINITY;
        const float s01 = r < n ? (d[0][1] + d[1][1]) * f1 : -INFINITY;
        const float s10 = r + 8 < n ? (d[0][2] + d[1][2]) * f0 : -INFINITY;
        const float s11 = r + 8 < n ? (d[0][3] + d[1][3]) * f1 : -INFINITY;
        float x0 = fmaxf(s00, s10), x1 = fmaxf(s01, s11);
        // a new maximum, or a value scale above the frame of the value sums (a power
        // of two >= every value scale seen): bring the sums to the new frame
        if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1 || vs > vref)) {
#pragma unroll
            for (int off = 4; off < 32; off *= 2) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            }
            x0 = fmaxf(x0, m0);
            x1 = fmaxf(x1, m1);
            const float vnew = vs > vref ? __uint_as_float((__float_as_uint(vs) + 0x7fffffu) & 0x7f800000u) : vref;
            const float a0 = x0 == -INFINITY ? 1.f : fast_exp2(m0 - x0), a1 = x1 == -INFINITY ? 1.f : fast_exp2(m1 - x1);
            const float vr = vref > 0.f ? vref / vnew : 0.f;
            l0 *= a0;
            l1 *= a1;
            m0 = x0;
            m1 = x1;
            vref = vnew;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j][0] *= a0 * vr;
                o[j][1] *= a1 * vr;
                o[j][2] *= a0 * vr;
                o[j][3] *= a1 * vr;
            }
        }
        const float vw = vref > 0.f ? kWeightTop * (vs / vref) : vs;
        const float p00 = fast_exp2(s00 - m0), p01 = fast_exp2(s01 - m1), p10 = fast_exp2(s10 - m0), p11 = fast_exp2(s11 - m1);
        l0 += p00 + p10;
        l1 += p01 + p11;
        uint32_t wh[2], wr[2];
        f16x2_split(p00 * vw, p01 * vw, wh[0], wr[0]);
        f16x2_split(p10 * vw, p11 * vw, wh[1], wr[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            wh[t] = transpose8(wh[t]);
            wr[t] = transpose8(wr[t]);
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
            for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1]};
                mma_16816(o[2 * w + j], a, wh[0], wh[1]);
                mma_16816(o[2 * w + j], a, wr[0], wr[1]);
            }
        }
    }
    grid_launch_dependents();                          // the combine may be set up
    // a wait that ran out: every copy under way still has to land
    if (bad & AQ_DEV_TIMEOUT)
        for (int j = k; j < min(mine, k + kStages); ++j) mbar_wait_bounded(&bars[warp][j % kStages], (j / kStages) & 1);

    // ---- merge the warps (their rings are free now) ------------------------------
#pragma unroll
    for (int off = 4; off < 32; off *= 2) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    __syncwarp();
    float(*acc)[D] = reinterpret_cast<float(*)[D]>(stage);
    const float back = vref * (1.f / kWeightTop);
    if (2 * c < heads) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float2 *>(&acc[2 * c][16 * r + 2 * j]) = make_float2(o[j][0] * back, o[j][2] * back);
    }
    if (2 * c + 1 < heads) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float2 *>(&acc[2 * c + 1][16 * r + 2 * j]) = make_float2(o[j][1] * back, o[j][3] * back);
    }
    if (r == 0) {
        wm[warp][2 * c] = m0;
        wm[warp][2 * c + 1] = m1;
        wl[warp][2 * c] = l0;
        wl[warp][2 * c + 1] = l1;
    }
    __syncthreads();
    if (bad && lane == 0) atomicOr(&cbad, bad);
    for (int i = tid; i < heads * D; i += kThreads) {
        const int g = i / D, dim = i % D;
        float ms = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ms = fmaxf(ms, wm[w][g]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (wm[w][g] > -INFINITY || wl[w][g] != wl[w][g]) {
                const float f = exp2f(wm[w][g] - ms);
                den += f * wl[w][g];
                num += f * reinterpret_cast<const float *>(ring + static_cast<size_t>(w) * kStages * kPageBytes)[i];
            }
        }
        co[g][dim] = num;
        if (dim == 0) {
            cm[g] = ms;
            cl[g] = den;
        }
    }
    __syncthreads();
    if (cbad && tid == 0) flag_status(p.status, cbad);
    if (p.cluster > 1) {
        // ---- merge the cluster: this CTA's share of the outputs ------------------
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        cluster_wait_acquire();
        const uint32_t a_o = smem_u32(&co[0][0]), a_m = smem_u32(cm), a_l = smem_u32(cl), a_b = smem_u32(&cbad);
        for (int i = split * kThreads + tid; i < heads * D; i += S_ * kThreads) {
            const int g = i / D;
            float m[kMaxCluster], l[kMaxCluster], x[kMaxCluster], ms = -INFINITY, num = 0.f, den = 0.f;
            bool flagged = false;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                m[s] = -INFINITY;
                l[s] = x[s] = 0.f;
                if (s < S_) {
                    m[s] = ld_cluster_f32(mapa_u32(a_m + 4 * g, s));
                    l[s] = ld_cluster_f32(mapa_u32(a_l + 4 * g, s));
                    x[s] = ld_cluster_f32(mapa_u32(a_o + 4 * i, s));
                    flagged |= __float_as_int(ld_cluster_f32(mapa_u32(a_b, s))) != 0;
                }
                ms = fmaxf(ms, m[s]);
            }
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                if (m[s] > -INFINITY || l[s] != l[s]) {
                    const float f = exp2f(m[s] - ms);
                    den += f * l[s];
                    num += f * x[s];
                }
            }
            p.out[bh0 * D + i] = flagged ? nan : L == 0 ? 0.f : num / den;
        }
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
        cluster_wait_acquire();                        // peers have read this CTA's sums
        return;
    }
    for (int i = tid; i < heads * D; i += kThreads) {
        const int g = i / D, dim = i % D;
        if (S_ == 1) {
            p.out[bh0 * D + i] = cbad ? nan : L == 0 ? 0.f : co[g][dim] / cl[g];
        } else {
            p.part_o[((bh0 + g) * S_ + split) * D + dim] = co[g][dim];
            if (dim == 0) {
                p.part_ml[((bh0 + g) * S_ + split) * 2] = cbad ? nan : cm[g];
                p.part_ml[((bh0 + g) * S_ + split) * 2 + 1] = cbad ? nan : cl[g];
            }
        }
    }
}

// out = sum over splits of 2^(m - max) o, over the same sum of l: one CTA per
// (request, query head), one thread per dim; the splits' weights are computed
// once per CTA, 128 at a time.
__global__ void __launch_bounds__(kHeadDim) q8_combine_kernel(const __grid_constant__ Q8AttnParams p) {
    __shared__ float wgt[kHeadDim], red[2][kHeadDim / 32];
    grid_dependency_wait();                            // launched as a dependent of the attention kernel
    const size_t bh = static_cast<size_t>(blockIdx.y) * p.num_q_heads + blockIdx.x;
    const int S_ = p.num_splits, d = threadIdx.x;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + bh * S_;
    const float *po = p.part_o + bh * S_ * kHeadDim + d;
    float ms = -INFINITY;
    int nan = 0;
    for (int s = d; s < S_; s += kHeadDim) {
        const float2 x = ml[s];
        nan |= x.y != x.y;
        if (x.y > 0.f) ms = fmaxf(ms, x.x);
    }
    ms = warp_max_f32(ms);
    if ((d & 31) == 0) red[0][d / 32] = ms;
    nan = __syncthreads_or(nan);
    ms = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float num = 0.f, den = 0.f;
    for (int s0 = 0; s0 < S_; s0 += kHeadDim) {
        const int n = min(kHeadDim, S_ - s0);
        float w = 0.f;
        if (d < n) {
            const float2 x = ml[s0 + d];
            if (x.y > 0.f) {
                w = exp2f(x.x - ms);
                den += w * x.y;
            }
        }
        __syncthreads();
        wgt[d] = w;
        __syncthreads();
#pragma unroll 8
        for (int s = 0; s < n; ++s)
            if (wgt[s] > 0.f) num += wgt[s] * po[static_cast<size_t>(s0 + s) * kHeadDim];
    }
#pragma unroll
    for (int off = 16; off; off /= 2) den += __shfl_xor_sync(0xffffffffu, den, off);
    if ((d & 31) == 0) red[1][d / 32] = den;
    __syncthreads();
    den = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    p.out[bh * kHeadDim + d] = nan ? __int_as_float(0x7fc00000) : den > 0.f ? num / den : 0.f;
}

// Splits of a call (host arithmetic): enough CTAs to fill the GPU (4 per SM),
// each with a page per warp at least; up to kMaxCluster of them are a cluster.
struct Q8Plan {
    int32_t num_splits;
    size_t workspace;
};

Q8Plan q8_plan(int64_t batch, int64_t Hq, int64_t Hkv, int32_t max_seq_len, int32_t req) {
    const int64_t G = Hq / Hkv, units = batch * Hkv * ((G + kGroup - 1) / kGroup);
    const int64_t pages = (static_cast<int64_t>(max_seq_len) + kPage - 1) / kPage;
    int64_t S = req;
    if (S <= 0) {
        const int64_t slots = 4 * 152, most = pages / kWarps;
        S = units > 0 ? slots / units : 1;
        if (S > most) S = most;
        // one cluster of a power of two CTAs (they fit the GPU's groups of SMs
        // evenly) until partials give twice as many
        if (S > 1 && S < 2 * kMaxCluster) S = S >= 8 ? 8 : S >= 4 ? 4 : 2;
    }
    if (S > 4096) S = 4096;
    if (S > pages) S = pages;
    if (S < 1) S = 1;
    Q8Plan pl{};
    pl.num_splits = static_cast<int32_t>(S);
    pl.workspace = S > kMaxCluster ? static_cast<size_t>(batch) * Hq * S * (kHeadDim + 2) * sizeof(float) : 0;
    return pl;
}

// The code pages of [NP][Hkv] as boxes of 32 rows of 128 bytes.
cudaError_t page_map(CUtensorMap *map, const void *pages, int64_t boxes) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {kHeadDim, 2 * kPage, static_cast<cuuint64_t>(boxes > 0 ? boxes : 1)};
    const cuuint64_t strides[2] = {kHeadDim, kPageBytes};
    const cuuint32_t box[3] = {kHeadDim, 2 * kPage, 1}, step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(pages), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int FMT>
cudaError_t launch_q8(const Q8AttnParams &p, dim3 grid, cudaStream_t s) {
    auto kern = q8_attention_kernel<FMT>;
    static SmemAttr attr_state;
    if (cudaError_t e = ensure_smem_attr(attr_state, reinterpret_cast<const void *>(kern), kRingBytes); e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRingBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
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
    if (num_pages * num_kv_heads > 0x7fffffffll) return AQ_ERR_UNSUPPORTED;        // a copy's page coordinate
    Q8AttnParams p{};
    cudaError_t e = page_map(&p.map, code_pages, num_pages * num_kv_heads);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return AQ_ERR_CUDA;
    }
    p.q = q;
    p.scales = page_scales;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.out = out;
    if (pl.workspace > 0) {
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
    p.cluster = pl.num_splits <= kMaxCluster ? pl.num_splits : 1;
    p.wait_limit_ns = decode_wait_limit_ns();
    p.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(pl.num_splits), static_cast<unsigned>(num_kv_heads * p.chunks),
                    static_cast<unsigned>(batch));
    e = format == AQ_Q8_INT8 ? launch_q8<kInt8>(p, grid, s) : launch_q8<kE4m3>(p, grid, s);
    if (e == cudaSuccess && pl.workspace > 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(num_q_heads), static_cast<unsigned>(batch));
        cfg.blockDim = dim3(kHeadDim);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, q8_combine_kernel, p);
    }
    if (e == cudaSuccess) return AQ_OK;
    record_cuda_error(e);
    return AQ_ERR_CUDA;
}

}  // extern "C"
