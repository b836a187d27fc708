// Parameter blocks, launchers and device helpers of the operators around the recurrence
// (kda_conv.hip, kda_qk_norm.hip, kda_ssm.hip, kda_ssm_decode.hip).
#pragma once
#include <hip/hip_runtime.h>

#include "kda_device.hpp"

namespace kda {

// ------------------------------------------------------------------ device helpers
// Element types of one operand, chosen at run time where a kernel touches it rarely.
__device__ __forceinline__ float ld_any(const void *p, int64_t i, int is_bf16)
{
    return is_bf16 ? (float)((const bf16 *)p)[i] : ((const float *)p)[i];
}

// V consecutive elements as one access of up to 16 bytes (V = 1, 4 or 8; fp32 takes two for 8).
template <typename ET, int V> struct VecIO {
    static __device__ __forceinline__ void load(const ET *p, float (&f)[V])
    {
        if constexpr (V == 1) {
            f[0] = (float)*p;
        } else if constexpr (sizeof(ET) == 2 && V == 8) {
            const uint4 u = *(const uint4 *)p;
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) Vec4<ET>::unpack(Vec4<ET>::load(p + i), f + i);
        }
    }
    static __device__ __forceinline__ void store(ET *p, const float (&f)[V])
    {
        if constexpr (V == 1) {
            *p = (ET)f[0];
        } else if constexpr (sizeof(ET) == 2 && V == 8) {
            *(uint4 *)p = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) Vec4<ET>::store(p + i, Vec4<ET>::pack(f + i));
        }
    }
};

// The same for rows the launch reads once, or does not read back: non-temporal where a lane moves 16
// bytes.
template <typename ET, int V>
__device__ __forceinline__ void load_once(const ET *p, float (&f)[V])
{
    typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(ET) == 2 && V == 8) {
        const u32v4 w = __builtin_nontemporal_load((const u32v4 *)p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        }
    } else if constexpr (sizeof(ET) == 4 && V == 4) {
        const f32x4 w = __builtin_nontemporal_load((const f32x4 *)p);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = w[i];
    } else {
        VecIO<ET, V>::load(p, f);
    }
}
template <typename ET, int V>
__device__ __forceinline__ void store_once(ET *p, const float (&f)[V])
{
    typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(ET) == 2 && V == 8) {
        const u32v4 w = {pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
        __builtin_nontemporal_store(w, (u32v4 *)p);
    } else if constexpr (sizeof(ET) == 4 && V == 4) {
        const f32x4 w = {f[0], f[1], f[2], f[3]};
        __builtin_nontemporal_store(w, (f32x4 *)p);
    } else {
        VecIO<ET, V>::store(p, f);
    }
}

// y sigmoid(y); large negative y gives -0 (the reciprocal of an overflowed exponential).
__device__ __forceinline__ float silu_act(float y) { return y * sigmoid_act(y); }

// The sequence of flat token f in a packed batch: the largest n with cu[n] <= f (0 <= f < cu[N]);
// empty sequences are never it.  16-way search: the probes of one round are independent loads.
__device__ __forceinline__ int find_seq(const int32_t *cu, int N, int f)
{
    int lo = 0, hi = N;     // cu[lo] <= f < cu[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 15) / 16;
        int c = 0;
#pragma unroll
        for (int k = 1; k < 16; ++k) {
            const int i = min(lo + k * step, hi);
            c += (i < hi && cu[i] <= f) ? 1 : 0;
        }
        lo += c * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// ------------------------------------------------------------------ convolution
constexpr int CONV_MAX_WIDTH = 4;

struct ConvParams {
    const void *x;             // [.., C]
    void *o;
    const void *w, *bias;      // [C, W] contiguous, [C] or NULL
    const void *s0;            // initial states [N, W - 1, C] or NULL
    void *sT;                  // final states or NULL
    const int32_t *cu;         // NULL: dense, N sequences of T tokens
    int64_t x_sb, x_st, o_sb, o_st, s0_sn, s0_sr, sT_sn, sT_sr;
    int64_t tokens;            // all sequences' tokens
    int32_t N, T, C;
    int32_t w_bf16, bias_bf16, s0_bf16, sT_bf16, silu;
    int32_t run;               // tokens per thread
    int32_t nrun;              // runs: ceil(tokens / run)
    int32_t ncb, cgl;          // channel blocks; log2 of the channel groups (threads) of one
    int32_t out_blocks;        // workgroups of outputs; the ones after them write final states
};
hipError_t launch_conv(const ConvParams &p, int W, bool io_f32, int vec, int state_blocks, hipStream_t st);

struct ConvDecodeParams {
    const void *x;             // [R, T, C]
    void *o;                   // or NULL
    const void *w, *bias;
    void *pool;                // [P, W - 1, C]
    const int32_t *idx, *ntok;
    int64_t x_sr, x_st, o_sr, o_st, p_sn, p_sr;
    int32_t R, T, C, P;
    int32_t w_bf16, bias_bf16, silu, update;
    int32_t ncb;               // workgroups across the channels of a request
};
hipError_t launch_conv_decode(const ConvDecodeParams &p, int W, bool io_f32, bool pool_bf16, int vec, hipStream_t st);

// ------------------------------------------------------------------ norm and rotation
struct QkNormParams {
    const void *x[2];          // q, k
    void *o[2];
    const float *w[2];         // norm weights [D] or NULL
    const int32_t *pos;        // [B, T] or NULL
    const float *freq;         // [rot / 2]
    int64_t x_sb[2], x_st[2], x_sh[2], o_sb[2], o_st[2], o_sh[2], pos_sb, pos_st;
    int64_t tokens;            // B T
    int32_t T, D;
    int32_t heads[2];
    int32_t norm;              // KDA_NORM_*
    float eps, inv_d;          // inv_d: 1 / D (rms) or 1 (l2)
    int32_t rot, offset;
    float scale;
    int32_t batched;           // tokens are [B, T]: the batch strides matter
    int32_t splits;            // waves that share a token's rows
};
hipError_t launch_qk_norm(const QkNormParams &p, bool io_f32, int vec, bool interleaved, hipStream_t st);

// ------------------------------------------------------------------ state space scan
constexpr int SSM_CHUNK = 32;  // tokens per chunk

struct SsmParams {
    const void *x, *B, *C, *dt, *z;
    void *o;
    const float *A, *Dv, *dt_bias;
    const void *s0;
    void *sT;
    const int32_t *cu;
    int64_t x_sb, x_st, x_sh, z_sb, z_st, z_sh, o_sb, o_st, o_sh;
    int64_t B_sb, B_st, B_sg, C_sb, C_st, C_sg, dt_sb, dt_st, dt_sh;
    int64_t s0_sn, s0_sh, s0_sr, sT_sn, sT_sh, sT_sr;
    int32_t N, T, H, G;        // sequences, tokens of each (dense), heads, groups
    int32_t dt_bf16, softplus, s0_bf16, sT_bf16;
    int32_t seg;               // tokens per segment (a multiple of SSM_CHUNK); 0: whole sequences
    int32_t slots;             // segment slots (seg > 0) or sequences: the last N for last segments
    int32_t fine;              // 16 bits in what only feeds the output (bf16 data)
    int32_t own_start;         // workgroups form their own start states (else the scan did)
    int32_t wg_per_slot;       // workgroups of one slot
    int32_t heads_per_wg;
    int32_t wide;              // x, z, B, C rows are 16-byte aligned (else 8-byte, bf16)
    float *ws_state;           // [slots][H][N x P]
    float *ws_decay;           // [slots][H]: e to the sum of A step over the segment
};
// states_only: the end state of every segment from a zero start, and its decay (pass 1);
// otherwise the outputs.
hipError_t launch_ssm(const SsmParams &p, int P, int N, bool io_f32, bool states_only, hipStream_t st);
// Between the passes: end states of the segments into their start states.
hipError_t launch_ssm_scan(const SsmParams &p, int P, int N, hipStream_t st);

struct SsmDecodeParams {
    const void *x, *B, *C, *dt, *z;
    void *o;
    void *pool;
    const float *A, *Dv, *dt_bias;
    const int32_t *idx, *ntok;
    int64_t x_sr, x_st, x_sh, z_sr, z_st, z_sh, o_sr, o_st, o_sh;
    int64_t B_sr, B_st, B_sg, C_sr, C_st, C_sg, dt_sr, dt_st, dt_sh, p_sn, p_sh, p_sr;
    int32_t R, T, H, G, P;     // P: pool slots
    int32_t dt_bf16, softplus, update;
};
hipError_t launch_ssm_decode(const SsmDecodeParams &p, int P, int N, bool io_f32, bool pool_bf16, hipStream_t st);

}  // namespace kda
