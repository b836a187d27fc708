// CONV: the short causal depthwise convolution in front of the recurrence,
//     out[t, c] = act(sum_{w < W} weight[c, w] x[t - (W - 1) + w, c] + bias[c]),
// over packed or dense sequences (kda_conv) and over a few tokens per request against a pool of
// states (kda_conv_decode).
//
// Every input feeds W outputs of its own channel only, so a thread keeps its channels' last W
// inputs in registers and walks a run of consecutive tokens: each input is read once (W - 1 more
// at the start of a run), and 64 lanes move 1 KB of consecutive channels at a time.  The bound is
// HBM: read x, write out; the arithmetic (W FMAs an element, an exponential and a reciprocal with the
// activation) is about half of that time.  32,733 tokens x 12,288 channels, width 4, silu, bf16: 284 us,
// 5.7 TB/s of its 1.61 GB, and 5% more is read at the starts of runs.  256 requests of one token:
// 9.6 us, 5.3 TB/s.
#include <type_traits>

#include "kda_layer.hpp"

namespace kda {

template <int W, int V>
__device__ __forceinline__ void load_weights(const void *w, const void *bias, int w_bf16, int bias_bf16, int c0,
                                             float (&wt)[W][V], float (&b)[V])
{
    // the V channels' weights are V W consecutive elements: whole 4-element loads where V > 1
    float f[V * W];
    if constexpr (V == 1) {
#pragma unroll
        for (int k = 0; k < W; ++k) f[k] = ld_any(w, (int64_t)c0 * W + k, w_bf16);
    } else if (w_bf16) {
#pragma unroll
        for (int e = 0; e < V * W; e += 4) Vec4<bf16>::unpack(Vec4<bf16>::load((const bf16 *)w + (int64_t)c0 * W + e), f + e);
    } else {
#pragma unroll
        for (int e = 0; e < V * W; e += 4) Vec4<float>::unpack(Vec4<float>::load((const float *)w + (int64_t)c0 * W + e), f + e);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) wt[k][v] = f[v * W + k];
        b[v] = bias ? ld_any(bias, c0 + v, bias_bf16) : 0.f;
    }
}

template <int V>
__device__ __forceinline__ void load_state(const void *s, int64_t i, int is_bf16, float (&f)[V])
{
    if (is_bf16) VecIO<bf16, V>::load((const bf16 *)s + i, f);
    else VecIO<float, V>::load((const float *)s + i, f);
}
template <int V>
__device__ __forceinline__ void store_state(void *s, int64_t i, int is_bf16, const float (&f)[V])
{
    if (is_bf16) VecIO<bf16, V>::store((bf16 *)s + i, f);
    else VecIO<float, V>::store((float *)s + i, f);
}

// One output from the window (win: the W - 1 inputs before x, oldest first), then the window moves.
template <int W, int V>
__device__ __forceinline__ void conv_step(float (&win)[W - 1][V], const float (&x)[V], const float (&wt)[W][V],
                                          const float (&b)[V], int silu, float (&y)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a = b[v];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) a = __builtin_fmaf(wt[k][v], win[k][v], a);
        a = __builtin_fmaf(wt[W - 1][v], x[v], a);
        y[v] = silu ? silu_act(a) : a;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][v] = win[k + 1][v];
        win[W - 2][v] = x[v];
    }
}

// Workgroups 0 .. out_blocks - 1: 2^cgl threads across a block of channels, the rest of the 256
// across runs of `run` consecutive tokens of the flat token order.  A run may cross sequence
// starts: the window is then reloaded from that sequence's initial state.  The workgroups after
// them write final states (one thread per sequence and channel group), from x and the initial
// states alone; when the states are updated in place they run as a launch of their own, after
// every reader.
// WHOLE: a wave's threads walk one run (cgl >= 6), and its tokens and sequence are kept in scalar
// registers.
template <int W, typename ET, int V, bool WHOLE>
__global__ __launch_bounds__(256) void conv_kernel(const ConvParams p)
{
    const int cg = threadIdx.x & ((1 << p.cgl) - 1);
    const ET *x = (const ET *)p.x;
    if ((int)blockIdx.x >= p.out_blocks) {
        const int64_t item = (int64_t)(blockIdx.x - p.out_blocks) * 256 + threadIdx.x;
        const int ngr = (p.C + V - 1) / V;
        const int n = (int)(item / ngr), c0 = (int)(item % ngr) * V;
        if (n >= p.N) return;
        const int64_t s = p.cu ? p.cu[n] : 0;
        const int len = p.cu ? p.cu[n + 1] - p.cu[n] : p.T;
        const ET *xs = x + (p.cu ? 0 : n * p.x_sb) + s * p.x_st + c0;
        float f[W - 1][V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int pos = len - (W - 1) + k;      // state row k: position of the input it holds
            if (pos >= 0) VecIO<ET, V>::load(xs + pos * p.x_st, f[k]);
            else if (p.s0) load_state<V>(p.s0, n * p.s0_sn + (W - 1 + pos) * p.s0_sr + c0, p.s0_bf16, f[k]);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) f[k][v] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store_state<V>(p.sT, n * p.sT_sn + k * p.sT_sr + c0, p.sT_bf16, f[k]);
        return;
    }
    const int cb = blockIdx.x % p.ncb;
    const int lane_run = threadIdx.x >> p.cgl;
    const int64_t r = (int64_t)(blockIdx.x / p.ncb) * (256 >> p.cgl) + (WHOLE ? __builtin_amdgcn_readfirstlane(lane_run) : lane_run);
    const int c0 = ((cb << p.cgl) + cg) * V;
    if (c0 >= p.C || r >= p.nrun) return;
    ET *o = (ET *)p.o;
    float wt[W][V], b[V];
    load_weights<W, V>(p.w, p.bias, p.w_bf16, p.bias_bf16, c0, wt, b);

    int64_t f = r * p.run;
    // rows behind the last sequence are left as they were
    const int64_t f1 = min(f + (int64_t)p.run, p.cu ? min((int64_t)p.cu[p.N], p.tokens) : p.tokens);
    if (f >= f1) return;
    int n = p.cu ? find_seq(p.cu, p.N, (int)f) : (int)(f / p.T);
    float win[W - 1][V];
    while (true) {
        // the part of the run inside sequence n, from position pos on
        const int64_t start = p.cu ? p.cu[n] : (int64_t)n * p.T;
        const int64_t end = p.cu ? p.cu[n + 1] : start + p.T;
        const int64_t stop = min(f1, end);
        int pos = (int)(f - start);
        const ET *xp = x + (p.cu ? f * p.x_st : n * p.x_sb + pos * p.x_st) + c0;
        ET *op = o + (p.cu ? f * p.o_st : n * p.o_sb + pos * p.o_st) + c0;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int q = pos - (W - 1) + k;
            if (q >= 0) VecIO<ET, V>::load(xp + (int64_t)(k - (W - 1)) * p.x_st, win[k]);
            else if (p.s0) load_state<V>(p.s0, n * p.s0_sn + (W - 1 + q) * p.s0_sr + c0, p.s0_bf16, win[k]);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = 0.f;
        }
        int m = (int)(stop - f);
        // inputs in flight: packed prefill batch, 12,288 channels: 4 at a time 332 us, 8 at a time 313,
        // 309 with stores that bypass the caches, 16 at a time 295, 291 with a wave's run in scalar
        // registers, 286 with loads that bypass them too (runs of 64 tokens: 303, of 128: 309)
        auto steps = [&](auto count) {
            constexpr int K = decltype(count)::value;
            float in[K][V], y[V];
#pragma unroll
            for (int u = 0; u < K; ++u) load_once<ET, V>(xp + u * p.x_st, in[u]);
#pragma unroll
            for (int u = 0; u < K; ++u) {
                conv_step<W, V>(win, in[u], wt, b, p.silu, y);
                store_once<ET, V>(op + u * p.o_st, y);
            }
            xp += K * p.x_st;
            op += K * p.o_st;
            m -= K;
        };
        while (m >= 16) steps(std::integral_constant<int, 16>{});
        if (m >= 8) steps(std::integral_constant<int, 8>{});
        if (m >= 4) steps(std::integral_constant<int, 4>{});
        while (m > 0) steps(std::integral_constant<int, 1>{});
        f = stop;
        if (f >= f1) return;
        ++n;
        if (p.cu)
            while (p.cu[n + 1] <= f) ++n;       // past empty sequences: f < cu[N]
    }
}

template <int W, typename ET>
static hipError_t launch_conv_t(const ConvParams &p, int vec, int state_blocks, hipStream_t st)
{
    const int64_t blocks = (int64_t)p.out_blocks + state_blocks;
    if (blocks <= 0) return hipSuccess;
    constexpr int VMAX = sizeof(ET) == 2 ? 8 : 4;
    const dim3 grid((unsigned)blocks), thr(256);
    if (vec == VMAX && p.cgl >= 6) hipLaunchKernelGGL((conv_kernel<W, ET, VMAX, true>), grid, thr, 0, st, p);
    else if (vec == VMAX) hipLaunchKernelGGL((conv_kernel<W, ET, VMAX, false>), grid, thr, 0, st, p);
    else if (p.cgl >= 6) hipLaunchKernelGGL((conv_kernel<W, ET, 1, true>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((conv_kernel<W, ET, 1, false>), grid, thr, 0, st, p);
    return hipGetLastError();
}

hipError_t launch_conv(const ConvParams &p, int W, bool io_f32, int vec, int state_blocks, hipStream_t st)
{
    switch (W) {
    case 2: return io_f32 ? launch_conv_t<2, float>(p, vec, state_blocks, st) : launch_conv_t<2, bf16>(p, vec, state_blocks, st);
    case 3: return io_f32 ? launch_conv_t<3, float>(p, vec, state_blocks, st) : launch_conv_t<3, bf16>(p, vec, state_blocks, st);
    case 4: return io_f32 ? launch_conv_t<4, float>(p, vec, state_blocks, st) : launch_conv_t<4, bf16>(p, vec, state_blocks, st);
    }
    return hipErrorInvalidValue;
}

// One thread per (request, channel group): the slot's W - 1 rows and the request's tokens go
// through registers once; the window left after the last token is the new state.
template <int W, typename ET, typename ST, int V>
__global__ __launch_bounds__(256) void conv_decode_kernel(const ConvDecodeParams p)
{
    const int r = blockIdx.x / p.ncb;
    const int c0 = ((int)(blockIdx.x % p.ncb) * 256 + (int)threadIdx.x) * V;
    if (c0 >= p.C) return;
    const int slot = p.idx[r];
    if (slot < 0 || slot >= p.P) return;
    const int n = p.ntok ? min(max(p.ntok[r], 0), p.T) : p.T;
    ST *ps = (ST *)p.pool + slot * p.p_sn + c0;
    const ET *x = (const ET *)p.x + r * p.x_sr + c0;
    float win[W - 1][V], wt[W][V], b[V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) VecIO<ST, V>::load(ps + k * p.p_sr, win[k]);
    load_weights<W, V>(p.w, p.bias, p.w_bf16, p.bias_bf16, c0, wt, b);
    ET *o = p.o ? (ET *)p.o + r * p.o_sr + c0 : nullptr;
    for (int t = 0; t < n; ++t) {
        float in[V], y[V];
        VecIO<ET, V>::load(x + t * p.x_st, in);
        conv_step<W, V>(win, in, wt, b, p.silu, y);
        if (o) store_once<ET, V>(o + t * p.o_st, y);
    }
    if (p.update && n > 0) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store_once<ST, V>(ps + k * p.p_sr, win[k]);
    }
}

template <int W, typename ET, typename ST>
static hipError_t launch_conv_decode_t(const ConvDecodeParams &p, int vec, hipStream_t st)
{
    const int64_t blocks = (int64_t)p.R * p.ncb;
    if (blocks <= 0) return hipSuccess;
    constexpr int VMAX = sizeof(ET) == 2 ? 8 : 4;
    if (vec == VMAX) hipLaunchKernelGGL((conv_decode_kernel<W, ET, ST, VMAX>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    else hipLaunchKernelGGL((conv_decode_kernel<W, ET, ST, 1>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_conv_decode(const ConvDecodeParams &p, int W, bool io_f32, bool pool_bf16, int vec, hipStream_t st)
{
#define KDA_CONV(WW)                                                                                    \
    case WW:                                                                                            \
        if (io_f32) return pool_bf16 ? launch_conv_decode_t<WW, float, bf16>(p, vec, st)                \
                                     : launch_conv_decode_t<WW, float, float>(p, vec, st);              \
        return pool_bf16 ? launch_conv_decode_t<WW, bf16, bf16>(p, vec, st)                             \
                         : launch_conv_decode_t<WW, bf16, float>(p, vec, st);
    switch (W) {
        KDA_CONV(2)
        KDA_CONV(3)
        KDA_CONV(4)
    }
#undef KDA_CONV
    return hipErrorInvalidValue;
}

}  // namespace kda
