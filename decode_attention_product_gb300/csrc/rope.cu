// rope.cu -- rotary positions of queries and new keys, ahead of the append and
// the decode step.
//
// y1 = mscale * (x1 cos a - x2 sin a), y2 = mscale * (x1 sin a + x2 cos a) for
// every pair (x1, x2) of the first rot_dim dims, a = position * inv_freq[pair];
// the transposed rotation (sin negated) is the gradient of the plain one.
//
// The angle is taken modulo a turn in 64-bit fixed point: inv_freq / (2 pi) as
// a fraction of a turn in units of 2^-64 (from the double, 53 bits), times the
// integer position, wrapping; the wrapped product's signed fraction goes to
// sincospif.  A far position therefore keeps its angle (position 2^31 and
// inv_freq 1: within 4e-7), where position * inv_freq in 32 bits would be off
// by whole radians, without double-precision sines.
//
// One warp turns one 128-element row at a time, lane l holding dims
// [4l, 4l + 4); in the half layout the partner dims are rot_dim / 8 lanes
// away (a shuffle), in the interleaved one they are the lane's own.  A warp's
// angles serve all its heads, and four rows are under way together (one at a time:
// 90 us below).  Bound by memory: 8192 tokens of 32 query and 32 kv heads, 537 MB
// read and written out of place, in 82 us, 0.96 of the measured copy rate; a decode
// step's 8 tokens are one launch's latency, 4.2 us.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace aq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;               // rows of a warp under way together

struct RopeParams {
    const int32_t *positions;      // [T]
    const double *inv_freq;        // [rot_dim / 2]
    const float *q;                // [T][Hq][D] or null
    float *q_out;
    const __half *kv;              // [T][Hkv][2][D] or null
    __half *kv_out;
    int32_t num_q_heads, num_kv_heads, rot_dim;
    float mscale;
    int32_t transpose, lengths;
};

// cos and sin (times mscale) of position * inv_freq.
__device__ __forceinline__ float2 turn_of(int position, double inv_freq, float mscale, bool transpose) {
    double t = inv_freq * 0.15915494309189533577;          // turns per position
    const bool fine = fabs(t) < 1e300;
    t -= floor(t);                                         // [0, 1]
    const unsigned long long frac =
        t >= 1.0 ? 0ull : static_cast<unsigned long long>(t * 18446744073709551616.0);
    const long long a = static_cast<long long>(frac * static_cast<unsigned long long>(position));
    float s, c;
    sincospif(static_cast<float>(a) * 1.0842021724855044e-19f, &s, &c);     // 2^-63: half turns in [-1, 1]
    if (!fine) s = c = __int_as_float(0x7fc00000);
    return make_float2(c * mscale, (transpose ? -s : s) * mscale);
}

template <bool INTERLEAVED>
__device__ __forceinline__ float4 turn(float4 x, const float2 (&cs)[4], int lane, int quarter) {
    if (INTERLEAVED)
        return make_float4(x.x * cs[0].x - x.y * cs[0].y, x.x * cs[0].y + x.y * cs[0].x,
                           x.z * cs[1].x - x.w * cs[1].y, x.z * cs[1].y + x.w * cs[1].x);
    // the pair's other half: cs holds -sin for the first half, +sin for the second
    const int from = lane < quarter ? lane + quarter : lane - quarter;
    const float px = __shfl_sync(0xffffffffu, x.x, from & 31), py = __shfl_sync(0xffffffffu, x.y, from & 31);
    const float pz = __shfl_sync(0xffffffffu, x.z, from & 31), pw = __shfl_sync(0xffffffffu, x.w, from & 31);
    return make_float4(x.x * cs[0].x + px * cs[0].y, x.y * cs[1].x + py * cs[1].y, x.z * cs[2].x + pz * cs[2].y,
                       x.w * cs[3].x + pw * cs[3].y);
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int D = kHeadDim;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const int pos = max(p.positions[t], -0x7fffffff) - p.lengths;
    const bool pad = pos < 0;
    const bool q_same = p.q == p.q_out, kv_same = p.kv == p.kv_out;
    if (pad && (!p.q || q_same) && (!p.kv || kv_same)) return;
    const int quarter = p.rot_dim / 8;                 // lanes of one half of the rotated dims
    const bool rot = !pad && 4 * lane < p.rot_dim;
    float2 cs[4] = {};
    if (rot) {
        if (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                cs[j] = turn_of(pos, p.inv_freq[2 * lane + j], p.mscale, p.transpose);
        } else {
            const bool second = lane >= quarter;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cs[j] = turn_of(pos, p.inv_freq[4 * (second ? lane - quarter : lane) + j], p.mscale, p.transpose);
                if (!second) cs[j].y = -cs[j].y;
            }
        }
    }
    const int w0 = blockIdx.y * kWarps + warp, nw = gridDim.y * kWarps;
    // kRows rows of a warp at a time: their loads are under way together
    if (p.q && !(pad && q_same)) {
        const size_t o = static_cast<size_t>(t) * p.num_q_heads * D + 4 * lane;
        for (int h0 = w0; h0 < p.num_q_heads; h0 += kRows * nw) {
            float4 x[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int h = h0 + j * nw;
                x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < p.num_q_heads) x[j] = *reinterpret_cast<const float4 *>(p.q + o + static_cast<size_t>(h) * D);
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int h = h0 + j * nw;
                const float4 y = turn<INTERLEAVED>(x[j], cs, lane, quarter);
                if (h < p.num_q_heads && (rot || !q_same))
                    *reinterpret_cast<float4 *>(p.q_out + o + static_cast<size_t>(h) * D) = rot ? y : x[j];
            }
        }
    }
    if (p.kv && !(pad && kv_same)) {
        const size_t o = static_cast<size_t>(t) * p.num_kv_heads * 2 * D + 4 * lane;
        for (int h0 = w0; h0 < p.num_kv_heads; h0 += kRows * nw) {
            uint2 u[kRows], v[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int h = h0 + j * nw;
                u[j] = v[j] = make_uint2(0u, 0u);
                if (h < p.num_kv_heads) {
                    const __half *row = p.kv + o + static_cast<size_t>(h) * 2 * D;
                    u[j] = *reinterpret_cast<const uint2 *>(row);
                    if (!kv_same) v[j] = *reinterpret_cast<const uint2 *>(row + D);
                }
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int h = h0 + j * nw;
                const float2 a = h2_to_f2(u[j].x), b = h2_to_f2(u[j].y);
                const float4 y = turn<INTERLEAVED>(make_float4(a.x, a.y, b.x, b.y), cs, lane, quarter);
                const __half2 lo = __floats2half2_rn(y.x, y.y), hi = __floats2half2_rn(y.z, y.w);
                uint2 r;
                r.x = *reinterpret_cast<const uint32_t *>(&lo);
                r.y = *reinterpret_cast<const uint32_t *>(&hi);
                if (h < p.num_kv_heads) {
                    __half *row = p.kv_out + o + static_cast<size_t>(h) * 2 * D;
                    if (rot || !kv_same) *reinterpret_cast<uint2 *>(row) = rot ? r : u[j];
                    if (!kv_same) *reinterpret_cast<uint2 *>(row + D) = v[j];
                }
            }
        }
    }
}

bool misaligned(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) != 0; }

}  // namespace

}  // namespace aq

using namespace aq;

extern "C" {

aq_status aq_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, int32_t original_len,
                              double beta_fast, double beta_slow, double *inv_freq, float *mscale) {
    if (rot_dim < 8 || rot_dim > kHeadDim || rot_dim % 8 != 0 || !inv_freq || !mscale) return AQ_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(factor) || factor < 1.0) return AQ_ERR_INVALID_ARGUMENT;
    if (scaling < AQ_ROPE_PLAIN || scaling > AQ_ROPE_YARN) return AQ_ERR_INVALID_ARGUMENT;
    const double r = rot_dim;
    double low = 0.0, high = 0.0;
    if (scaling == AQ_ROPE_YARN) {
        if (original_len < 1 || !(beta_fast > 0.0) || !(beta_slow > 0.0) || beta_fast < beta_slow ||
            !std::isfinite(beta_fast))
            return AQ_ERR_INVALID_ARGUMENT;
        // the (fractional) pair that turns `beta` times over the original context
        auto pair_of = [&](double beta) {
            return r * std::log(original_len / (beta * 6.283185307179586)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(beta_slow)), r - 1.0);
        if (high <= low) high = low + 0.001;
    }
    if (scaling == AQ_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = std::pow(base, -2.0 * i / r);
        if (scaling == AQ_ROPE_LINEAR) w /= factor;
        if (scaling == AQ_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
            w = w / factor * ramp + w * (1.0 - ramp);
        }
        inv_freq[i] = w;
    }
    *mscale = scaling == AQ_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return AQ_OK;
}

aq_status aq_rope(const aq_pq_config *cfg, int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                  const int32_t *positions, const double *inv_freq, int32_t rot_dim, float mscale, int32_t flags,
                  const float *q, float *q_out, const void *kv_f16, void *kv_out_f16, aq_stream_t stream) {
    if (!cfg || cfg->head_dim <= 0) return AQ_ERR_INVALID_ARGUMENT;
    if (cfg->head_dim != kHeadDim) return AQ_ERR_UNSUPPORTED;
    if (num_tokens < 0 || rot_dim < 8 || rot_dim > kHeadDim || rot_dim % 8 != 0 || !std::isfinite(mscale) ||
        (flags & ~(AQ_ROPE_INTERLEAVED | AQ_ROPE_TRANSPOSE | AQ_ROPE_LENGTHS)))
        return AQ_ERR_INVALID_ARGUMENT;
    if (q ? num_q_heads < 1 : q_out != nullptr) return AQ_ERR_INVALID_ARGUMENT;
    if (kv_f16 ? num_kv_heads < 1 : kv_out_f16 != nullptr) return AQ_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return AQ_OK;
    if (!positions || !inv_freq || (!q && !kv_f16) || (q && !q_out) || (kv_f16 && !kv_out_f16))
        return AQ_ERR_INVALID_ARGUMENT;
    if (misaligned(q) || misaligned(q_out) || misaligned(kv_f16) || misaligned(kv_out_f16) || misaligned(inv_freq))
        return AQ_ERR_INVALID_ARGUMENT;
    RopeParams p{};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.q = q;
    p.q_out = q_out;
    p.kv = static_cast<const __half *>(kv_f16);
    p.kv_out = static_cast<__half *>(kv_out_f16);
    p.num_q_heads = q ? num_q_heads : 0;
    p.num_kv_heads = kv_f16 ? num_kv_heads : 0;
    p.rot_dim = rot_dim;
    p.mscale = mscale;
    p.transpose = (flags & AQ_ROPE_TRANSPOSE) != 0;
    p.lengths = (flags & AQ_ROPE_LENGTHS) != 0;
    const int rows = p.num_q_heads > p.num_kv_heads ? p.num_q_heads : p.num_kv_heads;
    int split = (rows + kWarps - 1) / kWarps;          // head groups: fill the GPU when there are few tokens
    const int want = (2 * 152 + num_tokens - 1) / num_tokens;
    if (split > want) split = want;
    const dim3 grid(static_cast<unsigned>(num_tokens), static_cast<unsigned>(split));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto kern = flags & AQ_ROPE_INTERLEAVED ? rope_kernel<true> : rope_kernel<false>;
    const cudaError_t e = launch_dependent(kern, grid, dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess) return AQ_OK;
    record_cuda_error(e);
    return AQ_ERR_CUDA;
}

}  // extern "C"
