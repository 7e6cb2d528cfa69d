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
//
// Measured (INT8 unless said; of the measured copy rate): ragged (256 requests, 421 k
// tokens, 32 heads, 3.5 GB) 511 us, 1.0; long (131072 tokens, 32 heads) 168 us with the
// combine, 0.94 (E4M3 190 us: the ALU, its widening takes 15 integer operations where
// INT8's takes 11); page1 (4 x 2048 tokens, 32 heads) 16.6 us, 0.60; qwen_gqa (8 x 1000
// tokens, 64 query and 8 kv heads, E4M3) 8.7 us, 0.29; 512 tokens of 2 heads 3.7 us.  The large ones are bound by HBM;
// the small ones by the chain release - ids and length - first page - merge, 5 to 6 us
// of it without a page's work, and by issue while their few pages per warp run.
// Tried and slower: pages loaded straight to registers (one page in flight per warp
// at 158 registers: long 295 us), 8 splits pushed to their owners (a release barrier
// in the prologue, 3 us under load), sums of the warps in row order (8-way bank
// conflicts, 2 us at a group of 8).
#include <cudaTypedefs.h>

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "q8_common.cuh"

namespace aq {

namespace {

constexpr int kWarps = 4;
static_assert(kWarps == 4, "the warps' flags are read by name");
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;             // pages in a warp's ring
constexpr int kGroup = 8;              // query heads of a tile
constexpr int kMaxCluster = 8;
constexpr int kQueryPitch = 80;        // words of a query's fp16 pairs: 4 groups of 16 + 4
constexpr int kSumPitch = 132;         // floats between heads of a warp's sums
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
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3}], [%4];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Transpose of an 8x8 fp16 tile held as (row lane / 4, columns 2 (lane % 4) + {0, 1}).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_arrive_release() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The codes as fp16 operands: INT8 as they are, E4M3 times 2^-8 by integer operations
// (the conversion instruction takes as long, long E4M3 189 against 190 us, but turns the
// NaN codes that unused slots may hold into NaN, which would have to be masked).
template <int FMT>
constexpr float kUnwiden = FMT == kE4m3 ? 256.f : 1.f;

template <int FMT>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (FMT == kE4m3) shift4_e4m3(w, lo, hi);
    else widen4<FMT>(w, lo, hi);
}

// Byte i of two tokens' words as one fp16 pair, i = 0 .. 3.
template <int FMT>
__device__ __forceinline__ void pair4(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
    const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
    widen<FMT>(x, h[0], h[1]);
    widen<FMT>(y, h[2], h[3]);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 4) q8_attention_kernel(const __grid_constant__ Q8AttnParams p) {
    constexpr int D = kHeadDim, P = kPage;
    extern __shared__ unsigned char ring_raw[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ float wm[kWarps][kGroup], wl[kWarps][kGroup];
    // first the queries' fp16 parts (qw), then this CTA's sums, read by the cluster (co)
    __shared__ __align__(16) uint32_t qw[2][kGroup][kQueryPitch];
    __shared__ float qdown[kGroup];
    float *co = reinterpret_cast<float *>(qw);
    static_assert(sizeof(qw) >= sizeof(float) * kGroup * kHeadDim, "the sums take the queries' place");
    __shared__ __align__(8) float2 cml[kGroup];
    __shared__ int wbad[kWarps], cflag;
    // the ring starts on the swizzle's period
    unsigned char *ring = ring_raw + ((1024u - (smem_u32(ring_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int split = blockIdx.x, kvh = blockIdx.y / p.chunks, chunk = blockIdx.y % p.chunks, b = blockIdx.z;
    const int heads = min(kGroup, p.group - chunk * kGroup);
    const size_t bh0 = static_cast<size_t>(b) * p.num_q_heads + static_cast<size_t>(kvh) * p.group + chunk * kGroup;
    const int S_ = p.num_splits;
    const float nan = __int_as_float(0x7fc00000);

    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&bars[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    grid_dependency_wait();
    grid_launch_dependents();
    // Small loads go out before the page copies: behind those they would queue for
    // microseconds (page1: all 512 CTAs' first copies take 3.5 us).  First the queries: 16 threads per head.
    uint4 xq[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (tid / 16 < heads) {
#pragma unroll
        for (int j = 0; j < 2; ++j) xq[j] = ld_global_na_v4(p.q + (bh0 + tid / 16) * D + 8 * (tid % 16) + 4 * j);
    }
    // page w0 + k * stride of the request is this warp's k-th: known before the length is,
    // so the first ids and the length are fetched together
    const int w0 = split * kWarps + warp, stride = S_ * kWarps;
    const int32_t *bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const uint32_t stage = smem_u32(ring) + warp * kStages * kPageBytes, bar0 = smem_u32(&bars[warp][0]);
    // this lane's first 16-byte chunks of keys (row r, chunk 2 c) and values (row 2 c, chunk r)
    const uint32_t at_k = r * D + (((2 * c) ^ r) << 4), at_v = (P + 2 * c) * D + ((r ^ (2 * c)) << 4);
    // page ids (-1: outside the pool) and scales of the warp's pages [k, k + 32), one per lane
    auto page_id = [&](int k) {
        const int64_t i = w0 + static_cast<int64_t>(k) * stride;
        const int pg = i < p.max_pages ? bt[i] : -1;
        return pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    // (a coherent load: the kernel may be resident while the one before still writes scales)
    auto page_scales = [&](int pg) {
        if (pg < 0) return make_float2(0.f, 0.f);
        const uint2 u = ld_global_na_v2(p.scales + (static_cast<size_t>(pg) * p.num_kv_heads + kvh) * 2);
        return make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    };
    int id = page_id(lane);
    const int L = p.seq_lens[b];
    const bool badlen = L < 0 || L > static_cast<int64_t>(p.max_pages) * P || L > p.max_seq_len;
    const int np = badlen ? 0 : (L - 1) / P + (L > 0);
    const int mine = np > w0 ? (np - w0 - 1) / stride + 1 : 0;
    // page k into its ring slot (lane 0); a page outside the pool only arrives
    auto issue = [&](int slot, int pg) {
        if (lane == 0) {
            uint64_t *bar = &bars[warp][slot];
            if (pg >= 0) {
                mbar_arrive_expect_tx(bar, kPageBytes);
                tma_page(stage + slot * kPageBytes, &p.map, pg * p.num_kv_heads + kvh, bar0 + 8 * slot);
            } else {
                mbar_arrive(bar);
            }
        }
    };
    float2 sc = page_scales(id);
    int next_id = mine > 32 ? page_id(32 + lane) : -1;
    float2 next_sc = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
        const int pg = __shfl_sync(0xffffffffu, id, k);
        if (k < mine) issue(k, pg);
    }

    // The queries, once per CTA: a head's 16 threads scale it by a power of two to
    // [2^13, 2^14) at its largest magnitude and split it into fp16 parts; every warp
    // then takes its tiles' operand, lane (r, c) head r's dims [32 c, 32 c + 32).
    // (Groups of 16 words are 20 apart, heads 80: conflict-free both ways.)
    {
        const int h = tid / 16, t = tid % 16;
        float top = 0.f;
        float4 x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[j] = make_float4(__uint_as_float(xq[j].x), __uint_as_float(xq[j].y), __uint_as_float(xq[j].z),
                               __uint_as_float(xq[j].w));
            top = fmaxf(fmaxf(fmaxf(top, fabsf(x[j].x)), fmaxf(fabsf(x[j].y), fabsf(x[j].z))), fabsf(x[j].w));
        }
#pragma unroll
        for (int off = 1; off < 16; off *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const int e = min(253, max(1, 267 - static_cast<int>(__float_as_uint(top) >> 23)));
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        uint4 hi, lo;
        f16x2_split(x[0].x * up, x[0].y * up, hi.x, lo.x);
        f16x2_split(x[0].z * up, x[0].w * up, hi.y, lo.y);
        f16x2_split(x[1].x * up, x[1].y * up, hi.z, lo.z);
        f16x2_split(x[1].z * up, x[1].w * up, hi.w, lo.w);
        const int at = 20 * (t / 4) + 4 * (t % 4);
        *reinterpret_cast<uint4 *>(&qw[0][h][at]) = hi;
        *reinterpret_cast<uint4 *>(&qw[1][h][at]) = lo;
        // what undoes the scaling, with the softmax scale
        if (t == 0)
            qdown[h] = __uint_as_float(static_cast<uint32_t>(254 - e) << 23) * p.scale_log2 * kUnwiden<FMT>;
    }
    __syncthreads();
    // the operand stays in shared memory, read once per page: in registers (32) it would
    // leave none for the page's own sums
    const uint32_t at_q = smem_u32(&qw[0][r][20 * c]);
    constexpr uint32_t kPart = kGroup * kQueryPitch * 4;
    const float qs0 = qdown[2 * c], qs1 = qdown[2 * c + 1];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, vref = 0.f, vinv = 1.f;
    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    int bad = badlen ? AQ_DEV_BAD_LENGTH : 0, k = 0, slot = 0;
    uint32_t phase = 0;

#pragma unroll 1
    for (; k < mine; ++k) {
        // the next 32 pages: ids fetched 32 pages ahead, scales 16
        if ((k & 31) == 16) next_sc = page_scales(next_id);
        if (k && (k & 31) == 0) {
            id = next_id;
            sc = next_sc;
            next_id = page_id(k + 32 + lane);
        }
        const int pg = __shfl_sync(0xffffffffu, id, k & 31);
        const float ks = __shfl_sync(0xffffffffu, sc.x, k & 31), vs = __shfl_sync(0xffffffffu, sc.y, k & 31);
        uint64_t *bar = &bars[warp][slot];
        bool ok = mbar_test_wait(bar, phase);
        if (!ok && p.wait_limit_ns) ok = mbar_wait_limit(bar, phase, p.wait_limit_ns);
        if (!__all_sync(0xffffffffu, ok)) {
            bad |= AQ_DEV_TIMEOUT;
            break;
        }
        const uint32_t base = stage + slot * kPageBytes;
        // page k + kStages into this slot, once every lane has read it
        auto refill = [&]() {
            __syncwarp();
            const int n = k + kStages;
            const int from = __shfl_sync(0xffffffffu, (n ^ k) & 32 ? next_id : id, n & 31);
            if (n < mine) issue(slot, from);
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
        };
        if (pg < 0) {
            bad |= AQ_DEV_BAD_PAGE;
            refill();
            continue;
        }
        uint4 kr[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) kr[t][i] = lds_v4(base + 8 * t * D + (at_k ^ (16 * i)));
        const int n = min(P, L - (w0 + k * stride) * P);

        float d[2][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 qh = lds_v4(at_q + 16 * i), ql = lds_v4(at_q + kPart + 16 * i);
#pragma unroll
            for (int j = 2 * i; j < 2 * i + 2; ++j) {
                uint32_t a[4];
                widen<FMT>(word(kr[0][j / 4], j % 4), a[0], a[2]);
                widen<FMT>(word(kr[1][j / 4], j % 4), a[1], a[3]);
                mma_16816(d[0], a, j & 1 ? qh.z : qh.x, j & 1 ? qh.w : qh.y);
                mma_16816(d[1], a, j & 1 ? ql.z : ql.x, j & 1 ? ql.w : ql.y);
            }
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
            vinv = vref > 0.f ? kWeightTop / vref : 1.f;   // exact: powers of two
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j][0] *= a0 * vr;
                o[j][1] *= a1 * vr;
                o[j][2] *= a0 * vr;
                o[j][3] *= a1 * vr;
            }
        }
        const float vw = vs * vinv;
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
        // values are read (and the slot refilled) this late to stay within 128 registers
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lds_v4(base + 8 * (i >> 1) * D + ((i & 1) ? (at_v + D) ^ 16 : at_v));
        refill();
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t b0[4], b1[4];
            pair4<FMT>(word(v[0], w), word(v[1], w), b0);
            pair4<FMT>(word(v[2], w), word(v[3], w), b1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1]};
                // a page's sum by itself, then added with rounding: the tensor cores' own
                // accumulation truncates, a bias that grows with the pages (long: 3.3e-6
                // of the output against 3.3e-7)
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816(t, a, wr[0], wr[1]);
                mma_16816(t, a, wh[0], wh[1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[2 * w + j][i] += t[i];
            }
        }
    }
    // a wait that ran out: every copy under way still has to land
    if (bad & AQ_DEV_TIMEOUT)
        for (int j = k; j < min(mine, k + kStages); ++j) {
            mbar_wait_bounded(&bars[warp][slot], phase);
            if (++slot == kStages) slot = 0, phase ^= 1;
        }

    // ---- merge the warps (their rings are free now) ------------------------------
#pragma unroll
    for (int off = 4; off < 32; off *= 2) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    __syncwarp();
    // sums in tile order: position 16 j + 2 r + e of a head is dim 16 r + 2 j + e
    float *acc = reinterpret_cast<float *>(ring + warp * kStages * kPageBytes);
    const float back = vref * (kUnwiden<FMT> / kWeightTop);
    if (2 * c < heads) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float2 *>(acc + 2 * c * kSumPitch + 16 * j + 2 * r) = make_float2(o[j][0] * back, o[j][2] * back);
    }
    if (2 * c + 1 < heads) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float2 *>(acc + (2 * c + 1) * kSumPitch + 16 * j + 2 * r) =
                make_float2(o[j][1] * back, o[j][3] * back);
    }
    if (r == 0) {
        wm[warp][2 * c] = m0;
        wm[warp][2 * c + 1] = m1;
        wl[warp][2 * c] = l0;
        wl[warp][2 * c + 1] = l1;
    }
    if (lane == 0) wbad[warp] = bad;
    __syncthreads();
    const int n_out = heads * D, flags = wbad[0] | wbad[1] | wbad[2] | wbad[3];
    if (flags && tid == 0) flag_status(p.status, flags);
    const bool merge = p.cluster > 1;
    auto dim_of = [](int pos) { return (pos & 14) * 8 + (pos >> 4) * 2; };      // of an even position
    if (tid == 0) cflag = flags;
    for (int g = warp; g < heads; g += kWarps) {       // a warp per head, 4 positions per lane
        float f[kWarps], ms = -INFINITY, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ms = fmaxf(ms, wm[w][g]);
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float lw = wl[w][g];
            f[w] = lw != lw ? lw : wm[w][g] > -INFINITY ? fast_exp2(wm[w][g] - ms) : 0.f;
            const float4 x = *reinterpret_cast<const float4 *>(
                ring + static_cast<size_t>(w) * kStages * kPageBytes + (g * kSumPitch + 4 * lane) * 4);
            den += f[w] * lw;                          // (a warp without pages adds 0 * 0; a NaN stays one)
            num.x += f[w] * x.x;
            num.y += f[w] * x.y;
            num.z += f[w] * x.z;
            num.w += f[w] * x.w;
        }
        if (merge) {
            *reinterpret_cast<float4 *>(co + g * D + 4 * lane) = num;
            if (lane == 0) cml[g] = make_float2(ms, den);
        } else {
            float *dst = S_ == 1 ? p.out + (bh0 + g) * D : p.part_o + ((bh0 + g) * S_ + split) * D;
            if (S_ == 1) {
                const float inv = flags ? nan : L == 0 ? 0.f : 1.f;
                num.x = inv == 0.f ? 0.f : num.x / den * inv;
                num.y = inv == 0.f ? 0.f : num.y / den * inv;
                num.z = inv == 0.f ? 0.f : num.z / den * inv;
                num.w = inv == 0.f ? 0.f : num.w / den * inv;
            } else if (lane == 0) {
                float *ml = p.part_ml + ((bh0 + g) * S_ + split) * 2;
                ml[0] = flags ? nan : ms;
                ml[1] = flags ? nan : den;
            }
            *reinterpret_cast<float2 *>(dst + dim_of(4 * lane)) = make_float2(num.x, num.y);
            *reinterpret_cast<float2 *>(dst + dim_of(4 * lane + 2)) = make_float2(num.z, num.w);
        }
    }
    if (!merge) return;
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();                            // every peer's sums are there
    // pairs of outputs, shared out over the cluster's threads
    for (int i = 2 * (split * kThreads + tid); i < n_out; i += 2 * S_ * kThreads) {
        const int g = i / D;
        float2 ml[kMaxCluster], x[kMaxCluster];
        float ms = -INFINITY, den = 0.f;
        float2 num = make_float2(0.f, 0.f);
        int flagged = 0;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            ml[s] = make_float2(-INFINITY, 0.f);
            if (s < S_) {
                ml[s] = ld_cluster_f32x2(mapa_u32(smem_u32(&cml[g]), s));
                x[s] = ld_cluster_f32x2(mapa_u32(smem_u32(co + i), s));
                flagged |= ld_cluster_s32(mapa_u32(smem_u32(&cflag), s));
            }
            ms = fmaxf(ms, ml[s].x);
        }
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            if (s < S_ && (ml[s].x > -INFINITY || ml[s].y != ml[s].y)) {
                const float f = fast_exp2(ml[s].x - ms);
                den += f * ml[s].y;
                num.x += f * x[s].x;
                num.y += f * x[s].y;
            }
        }
        *reinterpret_cast<float2 *>(p.out + (bh0 + g) * D + dim_of(i % D)) =
            flagged ? make_float2(nan, nan) : L == 0 ? make_float2(0.f, 0.f) : make_float2(num.x / den, num.y / den);
    }
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait_acquire();                            // peers have read this CTA's sums
}

// out = sum over splits of 2^(m - max) o, over the same sum of l: one CTA per
// (request, query head), one thread per dim; the splits' weights are computed
// once per CTA, 128 at a time.
__global__ void __launch_bounds__(kHeadDim) q8_combine_kernel(const __grid_constant__ Q8AttnParams p) {
    __shared__ float wgt[kHeadDim], red[2][kHeadDim / 32];
    grid_dependency_wait();
    grid_launch_dependents();
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
            num += wgt[s] * po[static_cast<size_t>(s0 + s) * kHeadDim];    // (an empty split: 0 * 0)
    }
#pragma unroll
    for (int off = 16; off; off /= 2) den += __shfl_xor_sync(0xffffffffu, den, off);
    if ((d & 31) == 0) red[1][d / 32] = den;
    __syncthreads();
    den = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    p.out[bh * kHeadDim + d] = nan ? __int_as_float(0x7fc00000) : den > 0.f ? num / den : 0.f;
}

// Splits of a call (host arithmetic): the count with the least estimated time.  The
// estimate, in ns, was fitted to timings of 12 shapes (8 to 608 units, 2048 to 60000
// tokens, 1 to 64 splits): a CTA takes 180 per page while SMs hold one CTA, 220 with two,
// 350 with up to four (by then the memory's rate), and a fixed 2100 alone, 3000 + 150 S
// in a cluster of S, 5500 + 80 S with partials and their combine.  608 CTAs are a
// wave.  Against whole powers of two up to a wave: 96 units of 8192 tokens 36 us (6
// splits) instead of 47 (4), 192 of 2048 tokens 21 (3) instead of 27 (2), 8 of 4096
// tokens 7.9 (16) instead of 10.8 (64).
struct Q8Plan {
    int32_t num_splits;
    size_t workspace;
};

constexpr int64_t kSlots = 4 * 152;

int64_t q8_estimate(int64_t units, int64_t pages, int64_t S) {
    const int64_t per_cta = (pages + kWarps * S - 1) / (kWarps * S) * kWarps;
    const int64_t fixed = S == 1 ? 2100 : S <= kMaxCluster ? 3000 + 150 * S : 5500 + 80 * S;
    auto wave = [&](int64_t ctas) { return per_cta * (ctas <= kSlots / 4 ? 180 : ctas <= kSlots / 2 ? 220 : 350) + fixed; };
    const int64_t ctas = units * S, rest = ctas % kSlots;
    return ctas / kSlots * wave(kSlots) + (rest ? wave(rest) : 0);
}

Q8Plan q8_plan(int64_t batch, int64_t Hq, int64_t Hkv, int32_t max_seq_len, int32_t req) {
    const int64_t G = Hq / Hkv, units = batch * Hkv * ((G + kGroup - 1) / kGroup);
    const int64_t pages = (static_cast<int64_t>(max_seq_len) + kPage - 1) / kPage;
    int64_t S = req;
    if (S <= 0) {
        S = 1;
        const int64_t most = pages / kWarps;           // a page per warp at least
        auto consider = [&](int64_t c) {
            if (c > 1 && c <= most && c <= 4096 && q8_estimate(units, pages, c) < q8_estimate(units, pages, S)) S = c;
        };
        if (units > 0) {
            for (int64_t c = 2; c <= kMaxCluster; ++c) consider(c);
            for (int64_t c = 12; c <= 32; c += 4) consider(c);
            consider(kSlots / 4 / units);
            consider(kSlots / 2 / units);
            consider(kSlots / units);
        }
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
    if (cudaError_t e = ensure_smem_attr(attr_state, reinterpret_cast<const void *>(kern), kRingBytes, 100); e != cudaSuccess)
        return e;
    return launch_dependent(kern, grid, dim3(kThreads), kRingBytes, s, p.cluster, p);
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
        const dim3 rows(static_cast<unsigned>(num_q_heads), static_cast<unsigned>(batch));
        e = launch_dependent(q8_combine_kernel, rows, dim3(kHeadDim), 0, s, 1, p);
    }
    if (e == cudaSuccess) return AQ_OK;
    record_cuda_error(e);
    return AQ_ERR_CUDA;
}

}  // extern "C"
