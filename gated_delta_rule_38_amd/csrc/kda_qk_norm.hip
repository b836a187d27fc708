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

// V elements as they lie in memory, V sizeof(ET) / 4 words.
template <typename ET, int V> struct Raw {
    static constexpr int W = V * sizeof(ET) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const ET *p)
    {
        typedef uint32_t vec __attribute__((ext_vector_type(W)));
        const vec v = *(const vec *)p;
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
    // Rows in flight a lane group.  Packed prefill batch, 40 heads: 2 rows 158 us, 4 rows 172, 8 rows 194
    // (more registers, fewer waves); one row more requested ahead of each pair 162.
    constexpr int U = 2;
    constexpr bool ROT = MODE != QK_PLAIN;
    __shared__ float2 sCS[ROT ? 4 : 1][ROT ? 128 : 1];      // a wave's cos and sin
    __shared__ __attribute__((aligned(16))) float sRow[MODE == QK_STRIP ? 4 : 1][MODE == QK_STRIP ? 64 * V : 4];
    const int wave = threadIdx.x >> 6, lane64 = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + wave;
    const int64_t tok = p.splits == 1 ? item : item / p.splits;
    const int split = (int)(item - tok * p.splits);
    if (tok >= p.tokens) return;
    const int64_t b = p.batched ? tok / p.T : 0, t = tok - b * p.T;
    const int lanes = 1 << lanes_log2, lane = lane64 & (lanes - 1), slot = lane64 >> lanes_log2, per = 64 >> lanes_log2;
    const int c0 = lane * V;
    const bool in = c0 < p.D;

    Raw<ET, V> x[U];
    // the rows of one operand: rounds r, r + splits, ... of `per` heads
    const ET *src = nullptr;
    int heads = 0;
    auto load = [&](int s, int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (r0 + u * p.splits) * per + slot;
            if (h < heads && in) x[u].load(src + h * p.x_sh[s]);
            else
#pragma unroll
                for (int i = 0; i < Raw<ET, V>::W; ++i) x[u].w[i] = 0u;
        }
    };
    auto open = [&](int s) {
        src = (const ET *)p.x[s] + b * p.x_sb[s] + t * p.x_st[s] + c0;
        heads = p.heads[s];
    };
    open(0);
    load(0, split);

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
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = i0 + v;
            const bool rot = i >= 0 && i < p.rot, first = MODE == QK_INTER ? !(i & 1) : i < half;
            const int e = MODE == QK_INTER ? i >> 1 : (first ? i : i - half);
            const float2 q = sCS[wave][rot ? e : 0];
            cs[v] = rot ? q.x : 1.f;
            sn[v] = rot ? (first ? -q.y : q.y) : 0.f;
        }
        if constexpr (MODE == QK_LANES) {
            turns = i0 >= 0 && i0 < p.rot;
            if (turns) partner = lane64 + (i0 < half ? half : -half) / V;
        }
    }

    for (int s = 0; s < 2; ++s) {
        if (s) {
            open(1);
            load(1, split);
        }
        if (heads == 0) continue;
        ET *dst = (ET *)p.o[s] + b * p.o_sb[s] + t * p.o_st[s] + c0;
        // out = rn (own A + partner B): the norm weights (own, partner's) and the rotation in one
        float A[V], B[ROT ? V : 1];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float w = (p.w[s] && in) ? p.w[s][c0 + v] : 1.f;
            A[v] = ROT ? w * cs[ROT ? v : 0] : w;
            if constexpr (ROT) {
                const int i = i0 + v;
                int far = c0 + v;
                if (i >= 0 && i < p.rot) far += MODE == QK_INTER ? ((i & 1) ? -1 : 1) : (i < half ? half : -half);
                B[v] = ((p.w[s] && in) ? p.w[s][far] : 1.f) * sn[v];
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
                    rn = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum(ss, lanes), p.inv_d, p.eps));
                }
                float z[V];
                if constexpr (MODE == QK_PLAIN) {
#pragma unroll
                    for (int v = 0; v < V; ++v) z[v] = y[v] * A[v];
                } else if constexpr (MODE == QK_INTER) {
#pragma unroll
                    for (int v = 0; v < V; v += 2) {
                        // a pair that does not turn takes nothing of each other, not even a NaN
                        const bool rot = i0 + v >= 0 && i0 + v < p.rot;
                        z[v] = rot ? __builtin_fmaf(y[v + 1], B[v], y[v] * A[v]) : y[v] * A[v];
                        z[v + 1] = rot ? __builtin_fmaf(y[v], B[v + 1], y[v + 1] * A[v + 1]) : y[v + 1] * A[v + 1];
                    }
                } else if constexpr (MODE == QK_LANES) {
                    Raw<ET, V> far;
                    float other[V];
#pragma unroll
                    for (int i = 0; i < Raw<ET, V>::W; ++i) far.w[i] = __builtin_amdgcn_ds_bpermute(partner << 2, x[u].w[i]);
                    far.unpack(other);
#pragma unroll
                    for (int v = 0; v < V; ++v) z[v] = turns ? __builtin_fmaf(other[v], B[v], y[v] * A[v]) : y[v] * A[v];
                } else {
                    float *strip = sRow[wave] + slot * (lanes * V);
#pragma unroll
                    for (int v = 0; v < V; v += 4) *(float4 *)(strip + c0 + v) = make_float4(y[v], y[v + 1], y[v + 2], y[v + 3]);
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int i = i0 + v;
                        z[v] = y[v] * A[v];
                        if (i >= 0 && i < p.rot) z[v] = __builtin_fmaf(strip[c0 + v + (i < half ? half : -half)], B[v], z[v]);
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
