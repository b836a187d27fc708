// QK_NORM: the per-head norm of queries and keys and the rotation of their positions, in one pass.
//
// A row is one (token, head) vector of D channels, held by the smallest power of two of lanes that
// covers it at V channels a lane: the sum of squares is a butterfly over those lanes, in fp32.
// The bound is HBM (read and write every element once).  A workgroup takes a few tokens with all
// their heads, because a token's angles are the same for every head: cos and sin of
// position * inv_freq are formed once per workgroup, in 64 bits up to the reduction to one turn
// (a 32-bit product would be off by 0.03 rad at position 2^20), and kept in LDS.
// Rotated pairs sit in one lane (interleaved) or rot / 2 channels apart (half): the latter
// exchange through a row of LDS that only the row's own lanes touch.
#include "kda_layer.hpp"

namespace kda {

constexpr int QK_PAIRS = 512;   // LDS room for cos and sin: tile * rot / 2 pairs

template <typename ET, int V, bool INTER>
__global__ __launch_bounds__(256) void qk_norm_kernel(const QkNormParams p, int lanes_log2)
{
    __shared__ float2 sCS[QK_PAIRS];
    __shared__ float sRow[INTER ? 1 : 256 * V];
    const int split = blockIdx.x % p.splits;
    const int64_t tok0 = (int64_t)(blockIdx.x / p.splits) * p.tile;
    const int ntok = (int)min((int64_t)p.tile, p.tokens - tok0);
    const int half = p.rot >> 1;
    for (int e = threadIdx.x; e < ntok * half; e += 256) {
        const int64_t tok = tok0 + e / half;
        const int64_t b = tok / p.T, t = tok % p.T;
        const double turns = (double)p.pos[b * p.pos_sb + t * p.pos_st] *
                             ((double)p.freq[e % half] * 0.15915494309189533577);   // 1 / (2 pi)
        const float r = (float)(turns - __builtin_rint(turns));
        float s, c;
        sincospif(2.f * r, &s, &c);
        sCS[e] = make_float2(c * p.scale, s * p.scale);
    }
    __syncthreads();
    const int lanes = 1 << lanes_log2, lane = threadIdx.x & (lanes - 1), slot = threadIdx.x >> lanes_log2;
    const int c0 = lane * V;
    const bool in = c0 < p.D;
    const int hq = p.heads[0], heads = hq + p.heads[1];
    const int rows = ntok * heads, per = 256 >> lanes_log2;
    float wt[2][V];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) wt[s][v] = (p.w[s] && in) ? p.w[s][c0 + v] : 1.f;
    // every lane of a wave runs the same number of rounds (the exchanges need them all)
    for (int r0 = split * per; r0 < rows; r0 += per * p.splits) {
        const int row = r0 + slot;
        const bool ok = row < rows && in;
        const int tl = min(row, rows - 1) / heads, hh = min(row, rows - 1) % heads;
        const int s = hh >= hq, h = s ? hh - hq : hh;
        const int64_t tok = tok0 + tl, b = tok / p.T, t = tok % p.T;
        float y[V];
        if (ok) VecIO<ET, V>::load((const ET *)p.x[s] + b * p.x_sb[s] + t * p.x_st[s] + h * p.x_sh[s] + c0, y);
        else
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = 0.f;
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) ss = __builtin_fmaf(y[v], y[v], ss);
            for (int off = 1; off < lanes; off <<= 1) ss += __shfl_xor(ss, off);
            const float rn = 1.f / sqrtf(__builtin_fmaf(ss, p.inv_d, p.eps));
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = y[v] * rn * (s ? wt[1][v] : wt[0][v]);
        }
        if (p.rot) {
            if constexpr (INTER) {
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    const int i = c0 + v - p.offset;        // even: the part starts at an even channel
                    if (i >= 0 && i < p.rot) {
                        const float2 cs = sCS[tl * half + (i >> 1)];
                        const float a = y[v], bb = y[v + 1];
                        y[v] = a * cs.x - bb * cs.y;
                        y[v + 1] = bb * cs.x + a * cs.y;
                    }
                }
            } else {
                float *row_l = sRow + slot * (lanes * V);
#pragma unroll
                for (int v = 0; v < V; v += 4) *(float4 *)(row_l + c0 + v) = make_float4(y[v], y[v + 1], y[v + 2], y[v + 3]);
                __builtin_amdgcn_wave_barrier();    // the row's lanes are one wave's: LDS keeps its order
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = c0 + v - p.offset;
                    if (i >= 0 && i < p.rot) {
                        const bool first = i < half;
                        const float2 cs = sCS[tl * half + (first ? i : i - half)];
                        const float other = row_l[c0 + v + (first ? half : -half)];
                        y[v] = first ? y[v] * cs.x - other * cs.y : y[v] * cs.x + other * cs.y;
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        if (ok) VecIO<ET, V>::store((ET *)p.o[s] + b * p.o_sb[s] + t * p.o_st[s] + h * p.o_sh[s] + c0, y);
    }
}

template <typename ET, int V>
static hipError_t launch_qk_t(const QkNormParams &p, bool interleaved, hipStream_t st)
{
    int lg = 0;
    while ((V << lg) < p.D) ++lg;
    const int64_t blocks = (p.tokens + p.tile - 1) / p.tile * p.splits;
    if (blocks <= 0) return hipSuccess;
    if (interleaved) hipLaunchKernelGGL((qk_norm_kernel<ET, V, true>), dim3((unsigned)blocks), dim3(256), 0, st, p, lg);
    else hipLaunchKernelGGL((qk_norm_kernel<ET, V, false>), dim3((unsigned)blocks), dim3(256), 0, st, p, lg);
    return hipGetLastError();
}

hipError_t launch_qk_norm(const QkNormParams &p, bool io_f32, int vec, bool interleaved, hipStream_t st)
{
    if (io_f32) return launch_qk_t<float, 4>(p, interleaved, st);
    return vec == 8 ? launch_qk_t<bf16, 8>(p, interleaved, st) : launch_qk_t<bf16, 4>(p, interleaved, st);
}

}  // namespace kda
