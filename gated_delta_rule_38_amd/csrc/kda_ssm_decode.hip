// SSM_DECODE: the state space scan token by token against a pool of states, 1..8 tokens per
// request (the formulas of kda_ssm.hip; the slot and token-count rules of kda_decode.hip).
//
// One 256-thread workgroup owns one (request, head): a lane group of P / 4 lanes covers 4 value
// columns each, the row groups split the N state rows, and every thread keeps its rows x 4 columns
// in registers, so each state row moves through HBM once in each direction as whole 16-byte (fp32)
// or 8-byte (bf16) lanes.  The bound is that traffic.  Decays and updates of a column need no
// other column, and the read-out's sum over rows is only joined after the last token: two barriers
// a call, whatever the token count.  256 requests of one token, 32 heads of 64, 128 state channels, fp32
// pool: 104 us, 5.2 TB/s of its 0.54 GB.
#include "kda_layer.hpp"

namespace kda {

typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));

// State rows are read once and written once by the launch: both bypass the caches (256 requests x 32
// heads, fp32: 112 us with plain loads, 104 with these).
__device__ __forceinline__ void ld4_nt(const float *p, float (&x)[4])
{
    const f32x4 v = __builtin_nontemporal_load((const f32x4 *)p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void ld4_nt(const bf16 *p, float (&x)[4])
{
    const u32x2_t v = __builtin_nontemporal_load((const u32x2_t *)p);
    Vec4<bf16>::unpack(make_uint2(v.x, v.y), x);
}
__device__ __forceinline__ void st4_nt(float *p, const float (&x)[4])
{
    const f32x4 v = {x[0], x[1], x[2], x[3]};
    __builtin_nontemporal_store(v, (f32x4 *)p);
}
__device__ __forceinline__ void st4_nt(bf16 *p, const float (&x)[4])
{
    const uint2 u = Vec4<bf16>::pack(x);
    const u32x2_t w = {u.x, u.y};
    __builtin_nontemporal_store(w, (u32x2_t *)p);
}

template <int P, int N, typename ET, typename ST>
__global__ __launch_bounds__(256) void ssm_decode_kernel(const SsmDecodeParams p)
{
    constexpr int NCQ = P / 4;          // column quads = lanes of a row group
    constexpr int NRG = 256 / NCQ;      // row groups
    constexpr int RPG = N / NRG;        // rows per thread
    constexpr int TM = DECODE_MAX_TOKENS;
    __shared__ __attribute__((aligned(16))) float sB[TM][N], sC[TM][N], sX[TM][P];
    __shared__ float sStep[TM], sDec[TM];
    __shared__ __attribute__((aligned(16))) float sRed[TM][4][P];
    const int h = blockIdx.x % p.H, r = blockIdx.x / p.H;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cq = tid % NCQ, rg = tid / NCQ;
    const int slot = p.idx[r];
    if (slot < 0 || slot >= p.P) return;
    const int n = p.ntok ? min(max(p.ntok[r], 0), p.T) : p.T;
    if (n == 0) return;
    const int grp = h / (p.H / p.G);
    ST *ps = (ST *)p.pool + slot * p.p_sn + h * p.p_sh + (int64_t)(rg * RPG) * p.p_sr + 4 * cq;
    float s[RPG][4];
#pragma unroll
    for (int j = 0; j < RPG; ++j) ld4_nt(ps + j * p.p_sr, s[j]);
    const ET *x = (const ET *)p.x + r * p.x_sr + h * p.x_sh;
    const ET *Bp = (const ET *)p.B + r * p.B_sr + grp * p.B_sg, *Cp = (const ET *)p.C + r * p.C_sr + grp * p.C_sg;
    for (int e = tid; e < n * N; e += 256) {
        const int t = e / N, c = e % N;
        sB[t][c] = (float)Bp[t * p.B_st + c];
        sC[t][c] = (float)Cp[t * p.C_st + c];
    }
    for (int e = tid; e < n * P; e += 256) sX[e / P][e % P] = (float)x[(e / P) * p.x_st + e % P];
    if (tid < n) {
        const float v = ld_any(p.dt, r * p.dt_sr + tid * p.dt_st + h * p.dt_sh, p.dt_bf16) + (p.dt_bias ? p.dt_bias[h] : 0.f);
        const float step = p.softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
        sStep[tid] = step;
        sDec[tid] = expf(p.A[h] * step);
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
        const float e = sDec[t], d = sStep[t];
        const float4 x4 = *(const float4 *)&sX[t][4 * cq];
        const float u[4] = {d * x4.x, d * x4.y, d * x4.z, d * x4.w};
        float po[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < RPG; ++j) {
            const float b = sB[t][rg * RPG + j], c = sC[t][rg * RPG + j];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[j][k] = __builtin_fmaf(s[j][k], e, b * u[k]);
                po[k] = __builtin_fmaf(c, s[j][k], po[k]);
            }
        }
#pragma unroll
        for (int off = NCQ; off < 64; off <<= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) po[k] += __shfl_xor(po[k], off);
        if (lane < NCQ) *(float4 *)&sRed[t][wave][4 * cq] = make_float4(po[0], po[1], po[2], po[3]);
    }
    if (p.update) {
#pragma unroll
        for (int j = 0; j < RPG; ++j) st4_nt(ps + j * p.p_sr, s[j]);
    }
    if (!p.o) return;
    __syncthreads();
    const float skip = p.Dv ? p.Dv[h] : 0.f;
    for (int e = tid; e < n * NCQ; e += 256) {
        const int t = e / NCQ, c4 = 4 * (e % NCQ);
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            y[k] = (sRed[t][0][c4 + k] + sRed[t][1][c4 + k]) + (sRed[t][2][c4 + k] + sRed[t][3][c4 + k]) + skip * sX[t][c4 + k];
        if (p.z) {
            float z4[4];
            Vec4<ET>::unpack(Vec4<ET>::load((const ET *)p.z + r * p.z_sr + t * p.z_st + h * p.z_sh + c4), z4);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] *= silu_act(z4[k]);
        }
        Vec4<ET>::store((ET *)p.o + r * p.o_sr + t * p.o_st + h * p.o_sh + c4, Vec4<ET>::pack(y));
    }
}

template <int P, int N>
static hipError_t launch_ssm_decode_t(const SsmDecodeParams &p, bool io_f32, bool pool_bf16, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)p.R * p.H)), thr(256);
    if (io_f32 && pool_bf16) hipLaunchKernelGGL((ssm_decode_kernel<P, N, float, bf16>), grid, thr, 0, st, p);
    else if (io_f32) hipLaunchKernelGGL((ssm_decode_kernel<P, N, float, float>), grid, thr, 0, st, p);
    else if (pool_bf16) hipLaunchKernelGGL((ssm_decode_kernel<P, N, bf16, bf16>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((ssm_decode_kernel<P, N, bf16, float>), grid, thr, 0, st, p);
    return hipGetLastError();
}

hipError_t launch_ssm_decode(const SsmDecodeParams &p, int P, int N, bool io_f32, bool pool_bf16, hipStream_t st)
{
    if ((int64_t)p.R * p.H <= 0) return hipSuccess;
    if (P == 64 && N == 64) return launch_ssm_decode_t<64, 64>(p, io_f32, pool_bf16, st);
    if (P == 64 && N == 128) return launch_ssm_decode_t<64, 128>(p, io_f32, pool_bf16, st);
    if (P == 128 && N == 64) return launch_ssm_decode_t<128, 64>(p, io_f32, pool_bf16, st);
    if (P == 128 && N == 128) return launch_ssm_decode_t<128, 128>(p, io_f32, pool_bf16, st);
    return hipErrorInvalidValue;
}

}  // namespace kda
