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
    constexpr int U = 4;                            // rows in flight a lane group
    __shared__ float2 sCS[4][128];                  // a wave's cos and sin
    __shared__ __attribute__((aligned(16))) float sRow[MODE == QK_STRIP ? 4 : 1][MODE == QK_STRIP ? 64 * V : 4];
    const int wave = threadIdx.x >> 6, lane64 = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + wave;
    const int64_t tok = item / p.splits;
    const int split = (int)(item % p.splits);
    if (tok >= p.tokens) return;
    const int64_t b = p.batched ? tok / p.T : 0, t = tok - b * p.T;
    const int lanes = 1 << lanes_log2, lane = lane64 & (lanes - 1), slot = lane64 >> lanes_log2, per = 64 >> lanes_log2;
    const int c0 = lane * V;
    const bool in = c0 < p.D;
    const int heads0 = p.heads[0], heads = heads0 + p.heads[1], rounds = (heads + per - 1) / per;
    const ET *xq = (const ET *)p.x[0] + b * p.x_sb[0] + t * p.x_st[0] + c0;
    const ET *xk = (const ET *)p.x[1] + b * p.x_sb[1] + t * p.x_st[1] + c0;
    ET *oq = (ET *)p.o[0] + b * p.o_sb[0] + t * p.o_st[0] + c0;
    ET *ok = (ET *)p.o[1] + b * p.o_sb[1] + t * p.o_st[1] + c0;

    Raw<ET, V> x[U];
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = (r0 + u * p.splits) * per + slot;
            if (hh < heads && in) x[u].load(hh < heads0 ? xq + hh * p.x_sh[0] : xk + (hh - heads0) * p.x_sh[1]);
            else
#pragma unroll
                for (int i = 0; i < Raw<ET, V>::W; ++i) x[u].w[i] = 0u;
        }
    };
    load(split);

    // this lane's pairs: cos, sin with the sign its channels take it with
    const int half = p.rot >> 1, i0 = c0 - p.offset;
    constexpr int NP = MODE == QK_INTER ? V / 2 : V;
    float cs[MODE == QK_PLAIN ? 1 : NP], sn[MODE == QK_PLAIN ? 1 : NP];
    int partner = lane64;
    bool turns = false;
    if constexpr (MODE != QK_PLAIN) {
        const double pos = (double)p.pos[b * p.pos_sb + t * p.pos_st] * 0.15915494309189533577;     // 1 / (2 pi)
        for (int e = lane64; e < half; e += 64) {
            const double a = pos * (double)p.freq[e];
            float s, c;
            sincospif(2.f * (float)(a - __builtin_rint(a)), &s, &c);
            sCS[wave][e] = make_float2(c * p.scale, s * p.scale);
        }
        __builtin_amdgcn_wave_barrier();            // one wave's LDS accesses keep their order
#pragma unroll
        for (int v = 0; v < NP; ++v) {
            // channel of pair v: whether it is rotated, and its pair
            const int i = MODE == QK_INTER ? i0 + 2 * v : i0 + v;
            const bool rot = i >= 0 && i < p.rot, first = i < half;
            const int e = MODE == QK_INTER ? i >> 1 : (first ? i : i - half);
            const float2 q = sCS[wave][rot ? e : 0];
            cs[v] = rot ? q.x : 1.f;
            sn[v] = rot ? (MODE != QK_INTER && first ? -q.y : q.y) : 0.f;
        }
        if constexpr (MODE == QK_LANES) {
            turns = i0 >= 0 && i0 < p.rot;
            if (turns) partner = lane64 + (i0 < half ? half : -half) / V;
        }
    }
    // norm weights of this lane's channels, and of its partner's
    float wt[2][V], wp[MODE == QK_LANES ? 2 : 1][MODE == QK_LANES ? V : 1];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            wt[s][v] = (p.w[s] && in) ? p.w[s][c0 + v] : 1.f;
            if constexpr (MODE == QK_LANES) wp[s][v] = (p.w[s] && in) ? p.w[s][(partner - lane64) * V + c0 + v] : 1.f;
        }

    for (int r0 = split; r0 < rounds; r0 += U * p.splits) {
        if (r0 != split) load(r0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = (r0 + u * p.splits) * per + slot;
            if (r0 + u * p.splits >= rounds) break;     // the same for the whole wave
            const int s = hh >= heads0;
            float y[V], other[V];
            x[u].unpack(y);
            if constexpr (MODE == QK_LANES) {
                Raw<ET, V> far;
#pragma unroll
                for (int i = 0; i < Raw<ET, V>::W; ++i)
                    far.w[i] = __builtin_amdgcn_ds_bpermute(partner << 2, x[u].w[i]);
                far.unpack(other);
            }
            if (p.norm) {
                float ss = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) ss = __builtin_fmaf(y[v], y[v], ss);
                ss = group_sum(ss, lanes);
                const float rn = 1.f / sqrtf(__builtin_fmaf(ss, p.inv_d, p.eps));
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    y[v] *= rn * (s ? wt[1][v] : wt[0][v]);
                    if constexpr (MODE == QK_LANES) other[v] *= rn * (s ? wp[1][v] : wp[0][v]);
                }
            }
            if constexpr (MODE == QK_INTER) {
#pragma unroll
                for (int v = 0; v < V / 2; ++v) {
                    const float a = y[2 * v], c = y[2 * v + 1];
                    y[2 * v] = a * cs[v] - c * sn[v];
                    y[2 * v + 1] = c * cs[v] + a * sn[v];
                }
            } else if constexpr (MODE == QK_LANES) {
#pragma unroll
                for (int v = 0; v < V; ++v) y[v] = turns ? y[v] * cs[v] + other[v] * sn[v] : y[v];
            } else if constexpr (MODE == QK_STRIP) {
                float *strip = sRow[wave] + slot * (lanes * V);
#pragma unroll
                for (int v = 0; v < V; v += 4) *(float4 *)(strip + c0 + v) = make_float4(y[v], y[v + 1], y[v + 2], y[v + 3]);
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = i0 + v;
                    if (i >= 0 && i < p.rot) y[v] = y[v] * cs[v] + strip[c0 + v + (i < half ? half : -half)] * sn[v];
                }
                __builtin_amdgcn_wave_barrier();
            }
            if (hh < heads && in) VecIO<ET, V>::store(s ? ok + (hh - heads0) * p.o_sh[1] : oq + hh * p.o_sh[0], y);
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
