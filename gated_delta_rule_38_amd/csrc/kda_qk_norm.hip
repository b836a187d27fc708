// QK_NORM: the per-head norm of queries and keys and the rotation of their positions, in one pass.
//
// A row is one (token, head) vector of D channels, held by the smallest power of two of lanes that
// covers it at V channels a lane; the sum of squares is a butterfly over those lanes, in fp32.
// The bound is HBM (read and write every element once), so a wave keeps several rows in flight.
// A wave takes one token with all its heads (or every splits-th group of them when tokens are
// few): a token's angles are the same for every head, so cos and sin of position * inv_freq are
// formed once a wave, one or two pairs a lane, passed through a strip of LDS that only this wave
// touches, and kept in registers for all heads: no workgroup barrier anywhere.  Angles are formed
// in 64 bits up to the reduction to one turn (a 32-bit product would be off by 0.03 rad at position
// 2^20).
// Rotated pairs sit in one lane (interleaved) or rot / 2 channels apart (half).  When that distance
// and the offset are whole lanes, the partner's raw channels come by a lane exchange and its norm
// weight is kept beside the own one; else the row goes through the wave's LDS strip.
// The arithmetic is near the traffic (about 70 instructions a row and wave), so what is the same for a
// wave sits in scalar registers and no channel branches: 32,733 tokens, 32 + 8 heads of 128, bf16, half
// layout: 111 us, 6.1 TB/s of its 0.67 GB (153 us with token and addresses in vector registers and a
// branch for each channel's partner).
#include "kda_layer.hpp"

namespace kda {

// How a lane's channels find their partners.
enum { QK_PLAIN = 0, QK_INTER = 1, QK_LANES = 2, QK_STRIP = 3 };

template <int CTRL> __device__ __forceinline__ float dpp_mov(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum over the aligned group of `lanes` (a power of two) lanes, the same value in each: quad
// permutes, mirrors within 8 and 16 lanes (the groups below already hold equal sums), then
// exchanges across rows.
__device__ __forceinline__ float group_sum(float x, int lanes)
{
    if (lanes > 1) x += dpp_mov<0xB1>(x);       // lane ^ 1
    if (lanes > 2) x += dpp_mov<0x4E>(x);       // lane ^ 2
    if (lanes > 4) x += dpp_mov<0x141>(x);      // mirror of 8
    if (lanes > 8) x += dpp_mov<0x140>(x);      // mirror of 16
    if (lanes > 16) x += __shfl_xor(x, 16);
    if (lanes > 32) x += __shfl_xor(x, 32);
    return x;
}

// Norm weights at channel c (1 without them), aligned to nothing but their type.
template <int V>
__device__ __forceinline__ void weights_at(const float *w, int c, float (&f)[V])
{
    typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int v = 0; v < V; v += 4) {
        const f32x4_u q = w ? *(const f32x4_u *)(w + c + v) : f32x4_u{1.f, 1.f, 1.f, 1.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) f[v + k] = q[k];
    }
}

// V elements as they lie in memory, V sizeof(ET) / 4 words.
template <typename ET, int V> struct Raw {
    static constexpr int W = V * sizeof(ET) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const ET *p)
    {
        typedef uint32_t vec __attribute__((ext_vector_type(W)));
        const vec v = __builtin_nontemporal_load((const vec *)p);       // read once: 2% over a plain load
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = v[i];
    }
    __device__ __forceinline__ void unpack(float (&f)[V]) const
    {
        if constexpr (sizeof(ET) == 2) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = __builtin_bit_cast(float, w[i]);
        }
    }
};

template <typename ET, int V, int MODE>
__global__ __launch_bounds__(256) void qk_norm_kernel(const QkNormParams p, int lanes_log2)
{
    // Rows in flight a lane group (32,733 tokens, 40 heads of 128: 2 rows 116 us, 3 rows 115, 4 rows 113).
    constexpr int U = 4;
    constexpr bool ROT = MODE != QK_PLAIN;
    __shared__ __attribute__((aligned(16))) float2 sCS[ROT ? 4 : 1][ROT ? 128 : 1];      // a wave's cos and sin
    __shared__ __attribute__((aligned(16))) float sRow[MODE == QK_STRIP ? 4 : 1][MODE == QK_STRIP ? 64 * V : 4];
    // (what is the same for a wave is kept in scalar registers)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane64 = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + wave;
    const int split = (int)item & (p.splits - 1);           // splits: a power of two
    const int64_t tok = item >> __builtin_ctz(p.splits);
    if (tok >= p.tokens) return;
    const uint32_t b = p.batched ? (uint32_t)tok / (uint32_t)p.T : 0u;
    const int64_t t = tok - (int64_t)b * p.T;
    const int lanes = 1 << lanes_log2, per = 64 >> lanes_log2;
    const int lane = lane64 & (lanes - 1), slot = lane64 >> lanes_log2;
    const bool in = lane * V < p.D;
    const int c0 = in ? lane * V : 0;

    Raw<ET, V> x[U];
    // the rows of one operand: rounds r, r + splits, ... of `per` heads (past the last head: that one
    // again, not stored)
    const ET *src = nullptr;
    int heads = 0;
    auto load = [&](int s, int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (r0 + u * p.splits) * per + slot;
            x[u].load(src + min(h, heads - 1) * p.x_sh[s]);
        }
    };
    auto open = [&](int s) {
        src = (const ET *)p.x[s] + b * p.x_sb[s] + t * p.x_st[s] + c0;
        heads = p.heads[s];
        if (heads > 0) load(s, split);
    };
    open(0);

    // this lane's pairs: cos, and sin with the sign its channels take the partner with
    const int half = p.rot >> 1, i0 = c0 - p.offset;
    float cs[ROT ? V : 1], sn[ROT ? V : 1];
    int partner = lane64;
    bool turns = false;
    if constexpr (ROT) {
        const double pos = (double)p.pos[b * p.pos_sb + t * p.pos_st] * 0.15915494309189533577;     // 1 / (2 pi)
        for (int e = lane64; e < half; e += 64) {
            const double a = pos * (double)p.freq[e];
            float s, c;
            sincospif(2.f * (float)(a - __builtin_rint(a)), &s, &c);
            sCS[wave][e] = make_float2(c * p.scale, s * p.scale);
        }
        __builtin_amdgcn_wave_barrier();            // one wave's LDS accesses keep their order
        if constexpr (MODE == QK_LANES) {
            turns = i0 >= 0 && i0 < p.rot;
            const bool first = i0 < half;
            if (turns) partner = lane64 + (first ? half : -half) / V;
            const float2 *q = sCS[wave] + (turns ? (first ? i0 : i0 - half) : 0);
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                const float4 two = *(const float4 *)(q + v);
                cs[v] = turns ? two.x : 1.f;
                cs[v + 1] = turns ? two.z : 1.f;
                sn[v] = first ? -two.y : two.y;
                sn[v + 1] = first ? -two.w : two.w;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = i0 + v;
                const bool rot = i >= 0 && i < p.rot, first = MODE == QK_INTER ? !(i & 1) : i < half;
                const int e = MODE == QK_INTER ? i >> 1 : (first ? i : i - half);
                const float2 q = sCS[wave][rot ? e : 0];
                cs[v] = rot ? q.x : 1.f;
                sn[v] = first ? -q.y : q.y;
            }
        }
    }
    // what a channel that does not turn takes of its partner is 0, whatever the partner holds
    auto turning = [&](int v) { return (unsigned)(i0 + v) < (unsigned)p.rot; };

    for (int s = 0; s < 2; ++s) {
        if (s) open(1);
        if (heads == 0) continue;
        ET *dst = (ET *)p.o[s] + b * p.o_sb[s] + t * p.o_st[s] + c0;
        // out = rn (own A + partner B): the norm weights (own, partner's) and the rotation in one
        float A[V], B[ROT ? V : 1];
        weights_at<V>(p.w[s], c0, A);
        if constexpr (MODE == QK_LANES) weights_at<V>(p.w[s], turns ? c0 + (i0 < half ? half : -half) : c0, B);
        if constexpr (MODE == QK_INTER) {
#pragma unroll
            for (int v = 0; v < V; ++v) B[v] = A[v ^ 1];
        }
        if constexpr (MODE == QK_STRIP) {
#pragma unroll
            for (int v = 0; v < V; ++v) B[v] = p.w[s] ? p.w[s][c0 + v + (turning(v) ? (i0 + v < half ? half : -half) : 0)] : 1.f;
        }
        if constexpr (ROT) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] *= cs[v];
                B[v] = turning(v) ? B[v] * sn[v] : 0.f;
            }
        }
        const int rounds = (heads + per - 1) / per;
        for (int r0 = split; r0 < rounds; r0 += U * p.splits) {
            if (r0 != split) load(s, r0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u * p.splits >= rounds) break;     // the same for the whole wave
                const int h = (r0 + u * p.splits) * per + slot;
                float y[V];
                x[u].unpack(y);
                float rn = 1.f;
                if (p.norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) ss = __builtin_fmaf(y[v], y[v], ss);
                    rn = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum(in ? ss : 0.f, lanes), p.inv_d, p.eps));
                }
                float z[V];
#pragma unroll
                for (int v = 0; v < V; ++v) z[v] = y[v] * A[v];
                if constexpr (MODE == QK_INTER) {
#pragma unroll
                    for (int v = 0; v < V; ++v) z[v] = __builtin_fmaf(turning(v) ? y[v ^ 1] : 0.f, B[v], z[v]);
                } else if constexpr (MODE == QK_LANES) {
                    Raw<ET, V> far;
                    float other[V];
#pragma unroll
                    for (int i = 0; i < Raw<ET, V>::W; ++i) {
                        const uint32_t w = __builtin_amdgcn_ds_bpermute(partner << 2, x[u].w[i]);
                        far.w[i] = turns ? w : 0u;
                    }
                    far.unpack(other);
#pragma unroll
                    for (int v = 0; v < V; ++v) z[v] = __builtin_fmaf(other[v], B[v], z[v]);
                } else if constexpr (MODE == QK_STRIP) {
                    float *strip = sRow[wave] + slot * (lanes * V);
#pragma unroll
                    for (int v = 0; v < V; v += 4) *(float4 *)(strip + lane * V + v) = make_float4(y[v], y[v + 1], y[v + 2], y[v + 3]);
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float other = strip[c0 + v + (turning(v) ? (i0 + v < half ? half : -half) : 0)];
                        z[v] = __builtin_fmaf(turning(v) ? other : 0.f, B[v], z[v]);
                    }
                    __builtin_amdgcn_wave_barrier();
                }
#pragma unroll
                for (int v = 0; v < V; ++v) z[v] *= rn;
                if (h < heads && in) store_once<ET, V>(dst + h * p.o_sh[s], z);
            }
        }
    }
}

template <typename ET, int V>
static hipError_t launch_qk_t(const QkNormParams &p, bool interleaved, hipStream_t st)
{
    int lg = 0;
    while ((V << lg) < p.D) ++lg;
    const int64_t blocks = (p.tokens * p.splits + 3) / 4;
    if (blocks <= 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), thr(256);
    if (p.rot == 0) hipLaunchKernelGGL((qk_norm_kernel<ET, V, QK_PLAIN>), grid, thr, 0, st, p, lg);
    else if (interleaved) hipLaunchKernelGGL((qk_norm_kernel<ET, V, QK_INTER>), grid, thr, 0, st, p, lg);
    else if (p.rot / 2 % V == 0 && p.offset % V == 0) hipLaunchKernelGGL((qk_norm_kernel<ET, V, QK_LANES>), grid, thr, 0, st, p, lg);
    else hipLaunchKernelGGL((qk_norm_kernel<ET, V, QK_STRIP>), grid, thr, 0, st, p, lg);
    return hipGetLastError();
}

hipError_t launch_qk_norm(const QkNormParams &p, bool io_f32, int vec, bool interleaved, hipStream_t st)
{
    if (io_f32) return launch_qk_t<float, 4>(p, interleaved, st);
    return vec == 8 ? launch_qk_t<bf16, 8>(p, interleaved, st) : launch_qk_t<bf16, 4>(p, interleaved, st);
}

}  // namespace kda
