// Host side of the C ABI of include/kda_layer.h: descriptor checks, launch shapes and enqueueing
// of the convolution, the query/key norm with rotation and the state space scan.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../include/kda_layer.h"
#include "kda_host.hpp"
#include "kda_layer.hpp"

using namespace kda_host;

namespace {

// No C++ exception leaves a C entry point (an error message that cannot be allocated, say).
template <typename F>
kda_status_t guarded(F &&f) noexcept
{
    try {
        return f();
    } catch (...) {
        return KDA_ERR_HIP;
    }
}

#define KDA_TRY(expr)                        \
    do {                                     \
        const kda_status_t st_ = (expr);     \
        if (st_) return st_;                 \
    } while (0)

bool is_float(const kda_tensor_t *t) { return t->dtype == KDA_BF16 || t->dtype == KDA_F32; }

// Base address and strides in multiples of `elems` elements.
bool aligned_to(const kda_tensor_t *t, int elems)
{
    if (!t || !t->data) return true;
    const uint64_t vec = (uint64_t)elems * elem_size(t->dtype);
    if ((uintptr_t)t->data % vec) return false;
    for (int d = 0; d + 1 < t->ndim; ++d)
        if (t->shape[d] > 1 && ((uint64_t)t->stride[d] * elem_size(t->dtype)) % vec) return false;
    return true;
}

// Whether two views share no element.  Spans that do not meet are enough; so are two views of one
// row-major buffer that take different columns of the same rows (the q and k parts of a fused
// projection): equal outer strides, and inner extents that stay apart within a row.
bool disjoint(const kda_tensor_t *a, const kda_tensor_t *b)
{
    if (!overlaps(span_of(a), span_of(b))) return true;
    if (a->dtype != b->dtype || a->ndim != b->ndim || a->ndim < 3) return false;
    const int lead = a->ndim - 2;      // token dimensions; then heads and channels
    const int64_t row = a->stride[lead - 1], es = (int64_t)elem_size(a->dtype);
    for (int d = 0; d < lead; ++d)
        if (a->stride[d] != b->stride[d] || row <= 0 || a->stride[d] % row) return false;
    auto inner = [&](const kda_tensor_t *t) {
        return (t->shape[lead] - 1) * t->stride[lead] + (t->shape[lead + 1] - 1) * t->stride[lead + 1] + 1;
    };
    const int64_t bytes = (int64_t)((intptr_t)b->data - (intptr_t)a->data);
    if (bytes % es) return false;
    const int64_t d = ((bytes / es) % row + row) % row;      // b's column relative to a's
    return inner(a) <= d && d + inner(b) <= row;
}

struct Named {
    const kda_tensor_t *t;
    const char *name;
};

// `out` may overlap none of `ins`, except that it may be exactly `same`.
template <size_t K>
kda_status_t no_overlap(const kda_tensor_t *out, const char *out_name, const Named (&ins)[K],
                        const kda_tensor_t *same = nullptr)
{
    if (!out) return KDA_OK;
    const Span so = span_of(out);
    for (const Named &in : ins) {
        if (!in.t || (same && in.t == same && same_view(out, same))) continue;
        if (overlaps(so, span_of(in.t)) && !disjoint(out, in.t)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", out_name, in.name);
    }
    return KDA_OK;
}

// An output's rows may not share memory with each other: every extent above 1 steps over the whole
// inner extent.  (Inputs may be broadcast by zero strides.)
kda_status_t distinct_rows(const kda_tensor_t *t, const char *name)
{
    if (!t || numel(t) == 0) return KDA_OK;
    // sort the dimensions by stride, smallest first
    int order[4], n = 0;
    for (int d = 0; d < t->ndim; ++d)
        if (t->shape[d] > 1) order[n++] = d;
    std::sort(order, order + n, [&](int a, int b) { return t->stride[a] < t->stride[b]; });
    int64_t span = 1;
    for (int i = 0; i < n; ++i) {
        const int d = order[i];
        if (t->stride[d] < span) return fail(KDA_ERR_LAYOUT, "%s: elements share memory", name);
        span += (t->shape[d] - 1) * t->stride[d];
    }
    return KDA_OK;
}

// Token layout shared by the prompt operators: dense [B, T, ...] or packed [Ttot, ...] (also
// [1, Ttot, ...]) with cu_seqlens.
struct Tokens {
    bool dense = true;
    int64_t B = 1, T = 0, N = 0, tokens = 0;
    const int32_t *cu = nullptr;
};

kda_status_t token_layout(const kda_tensor_t *x, const char *name, int inner, const kda_tensor_t *cu, Tokens &L)
{
    L.dense = cu == nullptr;
    if (L.dense) {
        if (x->ndim != inner + 2) return fail(KDA_ERR_SHAPE, "dense %s must have %d dimensions, got %d", name, inner + 2, x->ndim);
        L.B = x->shape[0];
        L.T = x->shape[1];
        L.N = L.B;
        if (L.B > 0 && L.T > ((int64_t)1 << 31) / L.B) return fail(KDA_ERR_SHAPE, "too many tokens");
        L.tokens = L.B * L.T;
    } else {
        if (cu->dtype != KDA_I32) return fail(KDA_ERR_DTYPE, "cu_seqlens must be int32");
        if (cu->ndim != 1 || cu->shape[0] < 1) return fail(KDA_ERR_SHAPE, "cu_seqlens must be [N + 1]");
        if (x->ndim == inner + 2 && x->shape[0] == 1) L.tokens = x->shape[1];
        else if (x->ndim == inner + 1) L.tokens = x->shape[0];
        else return fail(KDA_ERR_SHAPE, "packed %s must be [T, ...] or [1, T, ...]", name);
        L.N = cu->shape[0] - 1;
        L.cu = (const int32_t *)cu->data;
    }
    if (L.tokens >= (int64_t)1 << 31 || L.N >= (int64_t)1 << 31) return fail(KDA_ERR_SHAPE, "too many tokens or sequences");
    return KDA_OK;
}

// Strides of a token-major tensor whose dimensions after the tokens are inner[0 .. n): batch,
// token, and the first inner dimension's.
struct TokStride {
    int64_t sb = 0, st = 0, s1 = 0;
};
kda_status_t token_view(const kda_tensor_t *t, const char *name, const Tokens &L, const int64_t *inner, int n, TokStride &o)
{
    int d = 0;
    if (L.dense) {
        if (t->ndim != n + 2) return fail(KDA_ERR_SHAPE, "%s: expected %d dimensions, got %d", name, n + 2, t->ndim);
        if (t->shape[0] != L.B || t->shape[1] != L.T) return fail(KDA_ERR_SHAPE, "%s: batch or token extent mismatch", name);
        o.sb = t->stride[0];
        o.st = t->stride[1];
        d = 2;
    } else {
        if (t->ndim == n + 2 && t->shape[0] == 1) d = 1;
        else if (t->ndim != n + 1) return fail(KDA_ERR_SHAPE, "%s: expected %d dimensions, got %d", name, n + 1, t->ndim);
        if (t->shape[d] != L.tokens) return fail(KDA_ERR_SHAPE, "%s: token extent mismatch", name);
        o.st = t->stride[d];
        ++d;
    }
    for (int i = 0; i < n; ++i)
        if (t->shape[d + i] != inner[i])
            return fail(KDA_ERR_SHAPE, "%s: extent %lld must be %lld", name, (long long)t->shape[d + i], (long long)inner[i]);
    o.s1 = t->stride[d];
    return KDA_OK;
}

kda_status_t check_cu(const Tokens &L, hipStream_t st)
{
    if (!L.cu || !env_on("KDA_CHECK")) return KDA_OK;
    DeviceChecks dc;
    dc.cu = L.cu;
    dc.N = L.N;
    dc.Ttot = L.tokens;
    return run_device_checks(dc, st, nullptr);
}

kda_status_t check_slots(const int32_t *idx, int64_t R, int64_t P, hipStream_t st)
{
    if (!env_on("KDA_CHECK")) return KDA_OK;
    DeviceChecks dc;
    dc.slots = idx;
    dc.R = R;
    dc.P = P;
    return run_device_checks(dc, st, nullptr);
}

// -------------------------------------------------------------------------- convolution
kda_status_t conv_weights(const kda_tensor_t *w, const kda_tensor_t *bias, int64_t C, int32_t act, int &W)
{
    if (!is_float(w) || (bias && !is_float(bias))) return fail(KDA_ERR_DTYPE, "weight and bias must be bf16 or fp32");
    if (w->ndim != 2 || w->shape[0] != C) return fail(KDA_ERR_SHAPE, "weight must be [C, W]");
    if (w->shape[1] < 2 || w->shape[1] > kda::CONV_MAX_WIDTH)
        return fail(KDA_ERR_UNSUPPORTED, "convolution width %lld not in 2..%d", (long long)w->shape[1], kda::CONV_MAX_WIDTH);
    W = (int)w->shape[1];
    if (C > 1 && w->stride[0] != W) return fail(KDA_ERR_LAYOUT, "weight must be contiguous");
    if (bias && (bias->ndim != 1 || bias->shape[0] != C)) return fail(KDA_ERR_SHAPE, "bias must be [C]");
    if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return fail(KDA_ERR_UNSUPPORTED, "activation %d", act);
    return KDA_OK;
}

// Channels a thread moves at once: 16 bytes of x where everything it touches is aligned for that
// (32,733 tokens x 12,288 channels, bf16: 297 us; one at a time 605), else one.
int conv_vec(int64_t C, std::initializer_list<const kda_tensor_t *> rows, const kda_tensor_t *w, bool io_f32)
{
    const int v = io_f32 ? 4 : 8;
    if (C % v || !w->data || (uintptr_t)w->data % (4 * elem_size(w->dtype))) return 1;
    for (const kda_tensor_t *t : rows) {
        // an 8-element fp32 state row moves as two 16-byte accesses
        if (t && !aligned_to(t, t->dtype == KDA_BF16 ? v : 4)) return 1;
    }
    return v;
}

kda_status_t conv_state(const kda_tensor_t *s, const char *name, int64_t n, int W, int64_t C)
{
    if (!is_float(s)) return fail(KDA_ERR_DTYPE, "%s must be bf16 or fp32", name);
    if (s->ndim != 3 || (n >= 0 && s->shape[0] != n) || s->shape[1] != W - 1 || s->shape[2] != C)
        return fail(KDA_ERR_SHAPE, "%s must be [%s, %d, %lld]", name, n < 0 ? "P" : "N", W - 1, (long long)C);
    return KDA_OK;
}

kda_status_t conv(const kda_tensor_t *x, const kda_tensor_t *w, const kda_tensor_t *bias, const kda_tensor_t *s0,
                  const kda_tensor_t *cu, kda_tensor_t *out, kda_tensor_t *sT, int32_t act, hipStream_t st)
{
    KDA_TRY(check_basic(x, "x", false));
    KDA_TRY(check_basic(w, "weight", false));
    KDA_TRY(check_basic(bias, "bias", true));
    KDA_TRY(check_basic(s0, "initial_state", true));
    KDA_TRY(check_basic(cu, "cu_seqlens", true));
    KDA_TRY(check_basic(out, "out", false));
    KDA_TRY(check_basic(sT, "final_state", true));
    if (!is_float(x)) return fail(KDA_ERR_DTYPE, "x must be bf16 or fp32");
    if (out->dtype != x->dtype) return fail(KDA_ERR_DTYPE, "x and out must share one dtype");
    Tokens L;
    KDA_TRY(token_layout(x, "x", 1, cu, L));
    const int64_t C = x->shape[x->ndim - 1];
    if (C < 1 || C > (int64_t)1 << 24) return fail(KDA_ERR_SHAPE, "channels not in 1..2^24");
    int W = 0;
    KDA_TRY(conv_weights(w, bias, C, act, W));
    TokStride xs, os;
    KDA_TRY(token_view(x, "x", L, &C, 1, xs));
    KDA_TRY(token_view(out, "out", L, &C, 1, os));
    if (s0) KDA_TRY(conv_state(s0, "initial_state", L.N, W, C));
    if (sT) KDA_TRY(conv_state(sT, "final_state", L.N, W, C));
    const Named ins[] = {{x, "x"}, {w, "weight"}, {bias, "bias"}, {s0, "initial_state"}, {cu, "cu_seqlens"}};
    KDA_TRY(no_overlap(out, "out", ins));
    KDA_TRY(no_overlap(sT, "final_state", ins, s0));
    if (sT && overlaps(span_of(sT), span_of(out))) return fail(KDA_ERR_ALIAS, "final_state overlaps out");
    KDA_TRY(distinct_rows(out, "out"));
    KDA_TRY(distinct_rows(sT, "final_state"));

    const bool f32 = x->dtype == KDA_F32;
    const int vec = conv_vec(C, {x, out, s0, sT}, w, f32);
    kda::ConvParams p{};
    p.x = x->data; p.o = out->data; p.w = w->data; p.bias = bias ? bias->data : nullptr;
    p.s0 = s0 ? s0->data : nullptr; p.sT = sT ? sT->data : nullptr; p.cu = L.cu;
    p.x_sb = xs.sb; p.x_st = xs.st; p.o_sb = os.sb; p.o_st = os.st;
    if (s0) { p.s0_sn = s0->stride[0]; p.s0_sr = s0->stride[1]; }
    if (sT) { p.sT_sn = sT->stride[0]; p.sT_sr = sT->stride[1]; }
    p.tokens = L.tokens; p.N = (int32_t)L.N; p.T = (int32_t)L.T; p.C = (int32_t)C;
    p.w_bf16 = w->dtype == KDA_BF16; p.bias_bf16 = bias && bias->dtype == KDA_BF16;
    p.s0_bf16 = s0 && s0->dtype == KDA_BF16; p.sT_bf16 = sT && sT->dtype == KDA_BF16;
    p.silu = act == KDA_ACT_SILU;
    const int64_t groups = (C + vec - 1) / vec;
    while (p.cgl < 8 && ((int64_t)1 << p.cgl) < groups) ++p.cgl;
    p.ncb = (int32_t)((groups + (1 << p.cgl) - 1) >> p.cgl);
    // Runs long enough that the W - 1 inputs read again at their starts are few, short enough that
    // the launch still fills the chip.
    p.run = 32;
    while (p.run > 4 && L.tokens / p.run * groups < 256 * 1024) p.run /= 2;
    const int64_t nrun = (L.tokens + p.run - 1) / p.run, per = 256 >> p.cgl;
    const int64_t out_blocks = (nrun + per - 1) / per * p.ncb;
    const int64_t state_blocks = sT ? (L.N * groups + 255) / 256 : 0;
    if (out_blocks + state_blocks > (int64_t)INT32_MAX) return fail(KDA_ERR_UNSUPPORTED, "too many workgroups for one launch");
    p.nrun = (int32_t)nrun;
    KDA_TRY(check_cu(L, st));
    const bool in_place = s0 && sT && s0->data == sT->data;
    hipError_t e = timed("kda_conv", st, [&] {
        p.out_blocks = (int32_t)out_blocks;
        hipError_t r = kda::launch_conv(p, W, f32, vec, in_place ? 0 : (int)state_blocks, st);
        if (r == hipSuccess && in_place) {
            p.out_blocks = 0;
            r = kda::launch_conv(p, W, f32, vec, (int)state_blocks, st);
        }
        return r;
    });
    return e == hipSuccess ? KDA_OK : hip_fail(e, "convolution launch");
}

kda_status_t decode_common(const kda_tensor_t *idx, const kda_tensor_t *ntok, int64_t R, int64_t T, int64_t P)
{
    if (T < 1 || T > kda::DECODE_MAX_TOKENS)
        return fail(KDA_ERR_UNSUPPORTED, "%lld tokens per request: decode takes 1..%d", (long long)T, kda::DECODE_MAX_TOKENS);
    if (idx->dtype != KDA_I32 || (ntok && ntok->dtype != KDA_I32))
        return fail(KDA_ERR_DTYPE, "state_indices and num_tokens must be int32");
    if (idx->ndim != 1 || idx->shape[0] != R) return fail(KDA_ERR_SHAPE, "state_indices must be [R]");
    if (ntok && (ntok->ndim != 1 || ntok->shape[0] != R)) return fail(KDA_ERR_SHAPE, "num_tokens must be [R]");
    if (P >= (int64_t)1 << 31 || R >= (int64_t)1 << 31) return fail(KDA_ERR_SHAPE, "too many requests or pool slots");
    return KDA_OK;
}

kda_status_t conv_decode(const kda_tensor_t *x, const kda_tensor_t *w, const kda_tensor_t *bias, kda_tensor_t *pool,
                         const kda_tensor_t *idx, const kda_tensor_t *ntok, kda_tensor_t *out, int32_t update,
                         int32_t act, hipStream_t st)
{
    KDA_TRY(check_basic(x, "x", false));
    KDA_TRY(check_basic(w, "weight", false));
    KDA_TRY(check_basic(bias, "bias", true));
    KDA_TRY(check_basic(pool, "state_pool", false));
    KDA_TRY(check_basic(idx, "state_indices", false));
    KDA_TRY(check_basic(ntok, "num_tokens", true));
    KDA_TRY(check_basic(out, "out", true));
    if (!is_float(x)) return fail(KDA_ERR_DTYPE, "x must be bf16 or fp32");
    if (out && out->dtype != x->dtype) return fail(KDA_ERR_DTYPE, "x and out must share one dtype");
    if (x->ndim != 3) return fail(KDA_ERR_SHAPE, "x must be [R, T, C]");
    const int64_t R = x->shape[0], T = x->shape[1], C = x->shape[2];
    if (C < 1 || C > (int64_t)1 << 24) return fail(KDA_ERR_SHAPE, "channels not in 1..2^24");
    int W = 0;
    KDA_TRY(conv_weights(w, bias, C, act, W));
    KDA_TRY(conv_state(pool, "state_pool", -1, W, C));
    const int64_t P = pool->shape[0];
    KDA_TRY(decode_common(idx, ntok, R, T, P));
    if (out && (out->ndim != 3 || out->shape[0] != R || out->shape[1] != T || out->shape[2] != C))
        return fail(KDA_ERR_SHAPE, "out must have x's shape");
    const Named ins[] = {{x, "x"}, {w, "weight"}, {bias, "bias"}, {idx, "state_indices"}, {ntok, "num_tokens"}};
    KDA_TRY(no_overlap(out, "out", ins));
    KDA_TRY(no_overlap(pool, "state_pool", ins));
    if (out && overlaps(span_of(pool), span_of(out))) return fail(KDA_ERR_ALIAS, "out overlaps state_pool");
    KDA_TRY(distinct_rows(out, "out"));
    KDA_TRY(distinct_rows(pool, "state_pool"));
    const bool f32 = x->dtype == KDA_F32;
    const int vec = conv_vec(C, {x, out, pool}, w, f32);
    kda::ConvDecodeParams p{};
    p.x = x->data; p.o = out ? out->data : nullptr; p.w = w->data; p.bias = bias ? bias->data : nullptr;
    p.pool = pool->data; p.idx = (const int32_t *)idx->data; p.ntok = ntok ? (const int32_t *)ntok->data : nullptr;
    p.x_sr = x->stride[0]; p.x_st = x->stride[1];
    if (out) { p.o_sr = out->stride[0]; p.o_st = out->stride[1]; }
    p.p_sn = pool->stride[0]; p.p_sr = pool->stride[1];
    p.R = (int32_t)R; p.T = (int32_t)T; p.C = (int32_t)C; p.P = (int32_t)P;
    p.w_bf16 = w->dtype == KDA_BF16; p.bias_bf16 = bias && bias->dtype == KDA_BF16;
    p.silu = act == KDA_ACT_SILU; p.update = update != 0;
    const int64_t ncb = ((C + vec - 1) / vec + 255) / 256;
    if (R * ncb > (int64_t)INT32_MAX) return fail(KDA_ERR_UNSUPPORTED, "too many workgroups for one launch");
    p.ncb = (int32_t)ncb;
    if (R == 0 || (!out && !update)) return KDA_OK;
    if (update) KDA_TRY(check_slots(p.idx, R, P, st));
    hipError_t e = timed("kda_conv_decode", st, [&] {
        return kda::launch_conv_decode(p, W, f32, pool->dtype == KDA_BF16, vec, st);
    });
    return e == hipSuccess ? KDA_OK : hip_fail(e, "convolution decode launch");
}

// ------------------------------------------------------------------- norm and rotation
kda_status_t qk_norm(const kda_tensor_t *q, const kda_tensor_t *k, const kda_tensor_t *qw, const kda_tensor_t *kw,
                     const kda_tensor_t *pos, const kda_tensor_t *freq, kda_tensor_t *qo, kda_tensor_t *ko,
                     const kda_qk_norm_options_t *o, hipStream_t st)
{
    KDA_TRY(check_basic(q, "q", false));
    KDA_TRY(check_basic(k, "k", true));
    KDA_TRY(check_basic(qw, "q_weight", true));
    KDA_TRY(check_basic(kw, "k_weight", true));
    KDA_TRY(check_basic(pos, "positions", true));
    KDA_TRY(check_basic(freq, "inv_freq", true));
    KDA_TRY(check_basic(qo, "q_out", false));
    KDA_TRY(check_basic(ko, "k_out", true));
    if (!o) return fail(KDA_ERR_NULL, "options are NULL");
    if (!k != !ko) return fail(KDA_ERR_NULL, "k and k_out go together");
    if (!k && kw) return fail(KDA_ERR_NULL, "k_weight without k");
    if (!is_float(q)) return fail(KDA_ERR_DTYPE, "q must be bf16 or fp32");
    if (qo->dtype != q->dtype || (k && (k->dtype != q->dtype || ko->dtype != q->dtype)))
        return fail(KDA_ERR_DTYPE, "q, k and the outputs must share one dtype");
    if (o->norm < KDA_NORM_NONE || o->norm > KDA_NORM_L2) return fail(KDA_ERR_UNSUPPORTED, "norm %d", o->norm);
    if (o->norm == KDA_NORM_NONE && (qw || kw)) return fail(KDA_ERR_UNSUPPORTED, "weights without a norm");
    if (o->norm != KDA_NORM_NONE && !(o->norm_eps >= 0.f && o->norm_eps < 1e30f))
        return fail(KDA_ERR_UNSUPPORTED, "norm_eps must be finite and >= 0");
    if (q->ndim != 3 && q->ndim != 4) return fail(KDA_ERR_SHAPE, "q must be [T, H, D] or [B, T, H, D]");
    const int nd = q->ndim, lead = nd - 2;
    const int64_t D = q->shape[nd - 1];
    if (D < 4 || D > 256 || D % 4) return fail(KDA_ERR_UNSUPPORTED, "head size %lld not a multiple of 4 in 4..256", (long long)D);
    int64_t tokens = 1;
    for (int d = 0; d < lead; ++d) {
        if (q->shape[d] > 0 && tokens > ((int64_t)1 << 31) / q->shape[d]) return fail(KDA_ERR_SHAPE, "too many tokens");
        tokens *= q->shape[d];
    }
    const kda_tensor_t *ts[] = {k, qo, ko};
    const char *names[] = {"k", "q_out", "k_out"};
    for (int i = 0; i < 3; ++i) {
        const kda_tensor_t *t = ts[i];
        if (!t) continue;
        const int64_t heads = i == 1 ? q->shape[nd - 2] : k->shape[std::max(0, k->ndim - 2)];
        if (t->ndim != nd || t->shape[nd - 1] != D || t->shape[nd - 2] != heads)
            return fail(KDA_ERR_SHAPE, "%s: dimensions, heads or head size mismatch", names[i]);
        for (int d = 0; d < lead; ++d)
            if (t->shape[d] != q->shape[d]) return fail(KDA_ERR_SHAPE, "%s: token extent mismatch", names[i]);
    }
    for (const kda_tensor_t *w : {qw, kw}) {
        if (!w) continue;
        if (w->dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "weights must be fp32");
        if (w->ndim != 1 || w->shape[0] != D) return fail(KDA_ERR_SHAPE, "weights must be [%lld]", (long long)D);
    }
    int64_t rot = 0;
    if (freq && numel(freq) > 0) {
        if (freq->dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "inv_freq must be fp32");
        if (freq->ndim != 1) return fail(KDA_ERR_SHAPE, "inv_freq must be [rot / 2]");
        rot = 2 * freq->shape[0];
        if (rot > D || o->rotary_offset < 0 || o->rotary_offset > D - rot)
            return fail(KDA_ERR_SHAPE, "the rotated part [%d, %lld) leaves the head of %lld", o->rotary_offset,
                        (long long)(o->rotary_offset + rot), (long long)D);
        if (o->rotary_layout != KDA_ROTARY_HALF && o->rotary_layout != KDA_ROTARY_INTERLEAVED)
            return fail(KDA_ERR_UNSUPPORTED, "rotary layout %d", o->rotary_layout);
        if (o->rotary_layout == KDA_ROTARY_INTERLEAVED && o->rotary_offset % 2)
            return fail(KDA_ERR_UNSUPPORTED, "the interleaved layout needs an even offset");
        if (!std::isfinite(o->rotary_scale)) return fail(KDA_ERR_UNSUPPORTED, "rotary_scale must be finite");
        if (!pos) return fail(KDA_ERR_NULL, "a rotation needs positions");
        if (pos->dtype != KDA_I32) return fail(KDA_ERR_DTYPE, "positions must be int32");
        if (pos->ndim != lead) return fail(KDA_ERR_SHAPE, "positions must be one per token");
        for (int d = 0; d < lead; ++d)
            if (pos->shape[d] != q->shape[d]) return fail(KDA_ERR_SHAPE, "positions must be one per token");
    }
    if (o->norm == KDA_NORM_NONE && rot == 0) return fail(KDA_ERR_UNSUPPORTED, "neither a norm nor a rotation");
    for (const kda_tensor_t *t : {q, k, (const kda_tensor_t *)qo, (const kda_tensor_t *)ko})
        if (!aligned_to(t, 4)) return fail(KDA_ERR_LAYOUT, "q, k and the outputs need 4-element-aligned base addresses and strides");
    const Named ins[] = {{q, "q"}, {k, "k"}, {qw, "q_weight"}, {kw, "k_weight"}, {pos, "positions"}, {freq, "inv_freq"}};
    KDA_TRY(no_overlap(qo, "q_out", ins, q));
    KDA_TRY(no_overlap(ko, "k_out", ins, k));
    if (ko && !disjoint(qo, ko)) return fail(KDA_ERR_ALIAS, "k_out overlaps q_out");
    KDA_TRY(distinct_rows(qo, "q_out"));
    KDA_TRY(distinct_rows(ko, "k_out"));

    kda::QkNormParams p{};
    const kda_tensor_t *xi[2] = {q, k}, *oi[2] = {qo, ko}, *wi[2] = {qw, kw};
    for (int s = 0; s < 2; ++s) {
        if (!xi[s]) continue;
        p.x[s] = xi[s]->data; p.o[s] = oi[s]->data;
        p.w[s] = wi[s] ? (const float *)wi[s]->data : nullptr;
        p.x_sb[s] = nd == 4 ? xi[s]->stride[0] : 0; p.o_sb[s] = nd == 4 ? oi[s]->stride[0] : 0;
        p.x_st[s] = xi[s]->stride[nd - 3]; p.o_st[s] = oi[s]->stride[nd - 3];
        p.x_sh[s] = xi[s]->stride[nd - 2]; p.o_sh[s] = oi[s]->stride[nd - 2];
        p.heads[s] = (int32_t)xi[s]->shape[nd - 2];
    }
    if (rot) {
        p.pos = (const int32_t *)pos->data;
        p.pos_sb = lead == 2 ? pos->stride[0] : 0;
        p.pos_st = pos->stride[lead - 1];
        p.freq = (const float *)freq->data;
    }
    p.tokens = tokens; p.T = (int32_t)q->shape[nd - 3]; p.D = (int32_t)D;
    p.norm = o->norm; p.eps = o->norm_eps; p.inv_d = o->norm == KDA_NORM_RMS ? 1.f / (float)D : 1.f;
    p.rot = (int32_t)rot; p.offset = o->rotary_offset; p.scale = o->rotary_scale;
    const int64_t heads = (int64_t)p.heads[0] + p.heads[1];
    if (tokens == 0 || heads == 0) return KDA_OK;
    if (heads > (int64_t)1 << 20) return fail(KDA_ERR_SHAPE, "too many heads");
    const bool f32 = q->dtype == KDA_F32;
    const int vec = !f32 && D % 8 == 0 && aligned_to(q, 8) && aligned_to(k, 8) && aligned_to(qo, 8) && aligned_to(ko, 8) ? 8 : 4;
    int lanes = 1;
    while (lanes * vec < D) lanes *= 2;
    const int64_t rounds = (heads + 64 / lanes - 1) / (64 / lanes);
    // one wave a token; with fewer tokens than fill the chip, several share a token's heads
    p.splits = 1;
    while (tokens * p.splits < 4096 && p.splits < rounds) p.splits *= 2;
    if (tokens * p.splits / 4 > (int64_t)INT32_MAX - 1) return fail(KDA_ERR_UNSUPPORTED, "too many workgroups for one launch");
    p.batched = lead == 2;
    hipError_t e = timed("kda_qk_norm", st, [&] {
        return kda::launch_qk_norm(p, f32, vec, o->rotary_layout == KDA_ROTARY_INTERLEAVED, st);
    });
    return e == hipSuccess ? KDA_OK : hip_fail(e, "norm and rotation launch");
}

// ------------------------------------------------------------------ state space scan
struct Ssm {
    Tokens L;
    int64_t H = 0, P = 0, G = 0, N = 0;
    TokStride x, dt, B, C, z, out;
    const kda_tensor_t *tD = nullptr, *tbias = nullptr, *tz = nullptr;
    int32_t softplus = 0;
    int64_t seg = 0, slots = 0;
    bool own_start = false;
    int hpw = 1;
    int64_t wps = 0;
    size_t off_decay = 0, bytes = 0;
};

kda_status_t ssm_vectors(const kda_tensor_t *A, const kda_ssm_options_t *o, int64_t H)
{
    const Named hs[] = {{A, "A"}, {o ? o->D : nullptr, "D"}, {o ? o->dt_bias : nullptr, "dt_bias"}};
    for (const Named &v : hs) {
        if (!v.t) continue;
        KDA_TRY(check_basic(v.t, v.name, false));
        if (v.t->dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "%s must be fp32", v.name);
        if (v.t->ndim != 1 || v.t->shape[0] != H) return fail(KDA_ERR_SHAPE, "%s must be [%lld]", v.name, (long long)H);
    }
    if (o && (o->dt_softplus < 0 || o->dt_softplus > 1)) return fail(KDA_ERR_UNSUPPORTED, "dt_softplus %d (0 or 1)", o->dt_softplus);
    return KDA_OK;
}

kda_status_t ssm_sizes(int64_t H, int64_t P, int64_t G, int64_t N)
{
    if (H < 1 || H > (int64_t)1 << 20) return fail(KDA_ERR_SHAPE, "H must be in 1..2^20");
    if ((P != 64 && P != 128) || (N != 64 && N != 128))
        return fail(KDA_ERR_UNSUPPORTED, "head size %lld and state size %lld must each be 64 or 128", (long long)P, (long long)N);
    if (G < 1 || H % G) return fail(KDA_ERR_SHAPE, "G must divide H");
    return KDA_OK;
}

kda_status_t ssm_state(const kda_tensor_t *t, const char *name, int64_t n, int64_t H, int64_t N, int64_t P)
{
    if (!is_float(t)) return fail(KDA_ERR_DTYPE, "%s must be fp32 or bf16", name);
    if (t->ndim != 4 || (n >= 0 && t->shape[0] != n) || t->shape[1] != H || t->shape[2] != N || t->shape[3] != P)
        return fail(KDA_ERR_SHAPE, "%s must be [.., %lld, %lld, %lld]", name, (long long)H, (long long)N, (long long)P);
    return KDA_OK;
}

// Up to this many workgroups every one has a CU to itself, and keeps 16 bits in what only feeds the
// output (FINE in kda_ssm.hip).
constexpr int64_t SSM_CUS = 256;

// Microseconds of one pass over `chunks` chunks by `workgroups` workgroups: `alone` a chunk while every
// workgroup has its CU to itself, towards `shared` as two sit on some CUs (the pass ends with those)
// and on all (512 at once), rounds beyond that; one is the most a CU holds of the fp32 kernel.
double ssm_pass(double workgroups, double chunks, double alone, double shared, bool f32)
{
    if (workgroups <= 256) return chunks * alone;
    if (f32) return chunks * alone * workgroups / 256;
    if (workgroups <= 512) return chunks * (alone + (shared - alone) * (0.5 + 0.5 * (workgroups - 256) / 256));
    return chunks * shared * workgroups / 512;
}

// Segment length of a batch (0: whole sequences), by a cost in microseconds fitted to MI355X.  Whole
// sequences: one pass.  Segments: the states' pass (1.4 us a chunk, shared or not), the outputs' pass
// (2.3 alone, 4.3 shared, 3.7 with 64 state channels), and the way from end states to start states; 2.4
// times as much a chunk in fp32.  That way is the shorter of two.  The scan, a launch: end states
// written, turned into start states, read again (2.35 TB/s), and its walk.  Or every workgroup of the
// outputs' pass reads the end states before its own (16 TB/s, mostly from caches): no launch and no
// second trip, but bytes that grow with the segments of a sequence (8 prompts, 32,733 tokens, segments
// of 1,536: 420 us with the scan, 400 without; one of 65,536 in segments of 1,024: 180 and 212).
// The lengths of a packed batch are on the device: the longest is taken for what the longest of n parts
// of a randomly cut line comes to (ln n + 0.58 times the mean), whose end a whole run is charged for
// alone, and segments are charged half a segment of waste a sequence.
// Against 8 to 15 forced lengths each: within 10% of the best on 8 batches of 203 to 65,536 tokens and
// 4 to 64 heads; on 9 random packed batches 7% over it on average and 24% at most (where a length
// happens to fill whole rounds of workgroups, which the host cannot see).
// in_place: the final states replace the initial ones, which other workgroups would still read.
void ssm_plan(Ssm &s, const kda_ssm_options_t *o, bool f32, bool in_place)
{
    const int64_t hg = s.H / s.G;
    s.hpw = s.P == 64 && hg > 1 ? 2 : 1;
    s.wps = s.G * ((hg + s.hpw - 1) / s.hpw);
    const int64_t N = s.L.N, longest = s.L.dense ? s.L.T : s.L.tokens;    // the longest a sequence can be
    const int asked = o ? o->segment : 0;
    s.seg = std::max(0, asked);
    const double T = (double)s.L.tokens, n = (double)N, cl = kda::SSM_CHUNK;
    const double likely = s.L.dense || N == 1 ? (double)longest : std::min((double)longest, T / n * (std::log(n) + 0.58));
    // segments of a length, and the cost of their start states
    auto count = [&](int64_t seg) { return s.L.dense || N == 1 ? n * std::ceil((double)longest / (double)seg) : T / (double)seg + 0.5 * n; };
    auto starts = [&](int64_t seg, bool &own) {
        const double bytes = std::max(0., count(seg) - n) * (double)s.H * (double)(s.N * s.P) * 4., each = likely / (double)seg;
        const double scan = 2. * bytes / 2.35e6 + 0.03 * each + 10., walk = bytes / 5e6 + 0.5 * each * bytes / 16e6;
        own = !in_place && walk < scan;
        return own ? walk : scan;
    };
    if (asked == 0 && N > 0 && longest > kda::SSM_CHUNK) {
        const double per = f32 ? 2.4 : 1., shared = s.N == 64 ? 3.7 : 4.3;
        const double half = s.P == 64 && s.hpw == 1 ? 0.5 : 1.;     // (workgroups of half the size)
        const double wgs = (double)s.wps * half, mean = std::ceil(T / n / cl);
        double best = per * (ssm_pass(n * wgs, mean, 2.3, shared, f32) + (std::ceil(likely / cl) - mean) * 2.3);
        for (int64_t seg = 32; seg < longest && seg <= 8192; seg += seg < 256 ? 32 : seg < 1024 ? 128 : 256) {
            const double segs = count(seg), chunks = (double)seg / cl;
            bool own;
            const double cost = per * (ssm_pass((segs - n) * wgs, chunks, 1.4, 1.4, f32) + ssm_pass(segs * wgs, chunks, 2.3, shared, f32)) +
                                starts(seg, own);
            if (cost < best) {
                best = cost;
                s.seg = seg;
            }
        }
    }
    if (s.seg >= longest || N == 0) s.seg = 0;
    if (s.seg == 0) {
        s.slots = N;
        return;
    }
    starts(s.seg, s.own_start);
    s.slots = s.L.dense ? N * std::max<int64_t>(1, (s.L.T + s.seg - 1) / s.seg) : s.L.tokens / s.seg + N;
    s.off_decay = align256((size_t)s.slots * s.H * s.N * s.P * 4);
    s.bytes = s.off_decay + align256((size_t)s.slots * s.H * 4);
}

kda_status_t ssm_check(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A, const kda_tensor_t *B,
                       const kda_tensor_t *C, const kda_tensor_t *s0, const kda_tensor_t *cu, const kda_tensor_t *out,
                       const kda_tensor_t *sT, const kda_ssm_options_t *o, Ssm &s)
{
    KDA_TRY(check_basic(x, "x", false));
    KDA_TRY(check_basic(dt, "dt", false));
    KDA_TRY(check_basic(A, "A", false));
    KDA_TRY(check_basic(B, "B", false));
    KDA_TRY(check_basic(C, "C", false));
    KDA_TRY(check_basic(s0, "initial_state", true));
    KDA_TRY(check_basic(cu, "cu_seqlens", true));
    KDA_TRY(check_basic(out, "out", false));
    KDA_TRY(check_basic(sT, "final_state", true));
    if (o) {
        s.tD = o->D; s.tbias = o->dt_bias; s.tz = o->z; s.softplus = o->dt_softplus;
        KDA_TRY(check_basic(s.tz, "z", true));
        if (o->segment < -1 || (o->segment > 0 && o->segment % kda::SSM_CHUNK))
            return fail(KDA_ERR_UNSUPPORTED, "segment %d: -1, 0 or a multiple of %d", o->segment, kda::SSM_CHUNK);
    }
    if (!is_float(x)) return fail(KDA_ERR_DTYPE, "x must be bf16 or fp32");
    if (B->dtype != x->dtype || C->dtype != x->dtype || out->dtype != x->dtype || (s.tz && s.tz->dtype != x->dtype))
        return fail(KDA_ERR_DTYPE, "x, B, C, z and out must share one dtype");
    if (dt->dtype != x->dtype && dt->dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "dt must have x's dtype or be fp32");
    KDA_TRY(token_layout(x, "x", 2, cu, s.L));
    s.H = x->shape[x->ndim - 2];
    s.P = x->shape[x->ndim - 1];
    if (B->ndim < 2) return fail(KDA_ERR_SHAPE, "B must be [.., G, N]");
    s.G = B->shape[B->ndim - 2];
    s.N = B->shape[B->ndim - 1];
    KDA_TRY(ssm_sizes(s.H, s.P, s.G, s.N));
    KDA_TRY(ssm_vectors(A, o, s.H));
    const int64_t hp[] = {s.H, s.P}, gn[] = {s.G, s.N}, hd[] = {s.H};
    KDA_TRY(token_view(x, "x", s.L, hp, 2, s.x));
    KDA_TRY(token_view(out, "out", s.L, hp, 2, s.out));
    if (s.tz) KDA_TRY(token_view(s.tz, "z", s.L, hp, 2, s.z));
    KDA_TRY(token_view(B, "B", s.L, gn, 2, s.B));
    KDA_TRY(token_view(C, "C", s.L, gn, 2, s.C));
    KDA_TRY(token_view(dt, "dt", s.L, hd, 1, s.dt));
    if (s0) KDA_TRY(ssm_state(s0, "initial_state", s.L.N, s.H, s.N, s.P));
    if (sT) KDA_TRY(ssm_state(sT, "final_state", s.L.N, s.H, s.N, s.P));
    for (const kda_tensor_t *t : {x, B, C, (const kda_tensor_t *)out, s.tz})
        if (!aligned_to(t, 4)) return fail(KDA_ERR_LAYOUT, "x, B, C, z and out need 4-element-aligned base addresses and strides");
    // the kernel addresses a chunk of each with 32-bit byte offsets from its first row
    for (int64_t stride : {s.x.st, s.B.st, s.C.st, s.z.st, s.out.st})
        if ((s.L.dense ? s.L.T : s.L.tokens) > 1 && stride > ((int64_t)1 << 31) / (kda::SSM_CHUNK * 4) - 256)
            return fail(KDA_ERR_UNSUPPORTED, "token strides must stay below 2^24 - 256 elements");
    if (s.H > 1 && (s.x.s1 > (int64_t)1 << 28 || s.z.s1 > (int64_t)1 << 28))
        return fail(KDA_ERR_UNSUPPORTED, "head strides of x and z must stay within 2^28 elements");
    const Named ins[] = {{x, "x"}, {dt, "dt"}, {A, "A"}, {B, "B"}, {C, "C"}, {s0, "initial_state"}, {cu, "cu_seqlens"},
                         {s.tD, "D"}, {s.tbias, "dt_bias"}, {s.tz, "z"}};
    KDA_TRY(no_overlap(out, "out", ins));
    KDA_TRY(no_overlap(sT, "final_state", ins, s0));
    if (sT && overlaps(span_of(sT), span_of(out))) return fail(KDA_ERR_ALIAS, "final_state overlaps out");
    KDA_TRY(distinct_rows(out, "out"));
    KDA_TRY(distinct_rows(sT, "final_state"));
    ssm_plan(s, o, x->dtype == KDA_F32, s0 && sT && s0->data == sT->data);
    if (s.slots * s.wps > (int64_t)INT32_MAX || s.L.N * s.H * (s.N * s.P / 1024) > (int64_t)INT32_MAX)
        return fail(KDA_ERR_UNSUPPORTED, "too many workgroups for one launch");
    if (env_on("KDA_LOG"))
        fprintf(stderr, "kda: ssm plan N=%lld tokens=%lld H=%lld G=%lld P=%lld N=%lld segment=%lld slots=%lld workgroups=%lld workspace=%zu B%s\n",
                (long long)s.L.N, (long long)s.L.tokens, (long long)s.H, (long long)s.G, (long long)s.P, (long long)s.N,
                (long long)s.seg, (long long)s.slots, (long long)(s.slots * s.wps), s.bytes, s.own_start ? ", own start states" : "");
    return KDA_OK;
}

kda_status_t ssm_run(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A, const kda_tensor_t *B,
                     const kda_tensor_t *C, const kda_tensor_t *s0, kda_tensor_t *out, kda_tensor_t *sT, const Ssm &s,
                     void *ws, hipStream_t st)
{
    KDA_TRY(check_cu(s.L, st));
    kda::SsmParams p{};
    p.x = x->data; p.B = B->data; p.C = C->data; p.dt = dt->data; p.z = s.tz ? s.tz->data : nullptr; p.o = out->data;
    p.A = (const float *)A->data;
    p.Dv = s.tD ? (const float *)s.tD->data : nullptr;
    p.dt_bias = s.tbias ? (const float *)s.tbias->data : nullptr;
    p.s0 = s0 ? s0->data : nullptr; p.sT = sT ? sT->data : nullptr; p.cu = s.L.cu;
    p.x_sb = s.x.sb; p.x_st = s.x.st; p.x_sh = s.x.s1;
    p.z_sb = s.z.sb; p.z_st = s.z.st; p.z_sh = s.z.s1;
    p.o_sb = s.out.sb; p.o_st = s.out.st; p.o_sh = s.out.s1;
    p.B_sb = s.B.sb; p.B_st = s.B.st; p.B_sg = s.B.s1;
    p.C_sb = s.C.sb; p.C_st = s.C.st; p.C_sg = s.C.s1;
    p.dt_sb = s.dt.sb; p.dt_st = s.dt.st; p.dt_sh = s.dt.s1;
    if (s0) { p.s0_sn = s0->stride[0]; p.s0_sh = s0->stride[1]; p.s0_sr = s0->stride[2]; }
    if (sT) { p.sT_sn = sT->stride[0]; p.sT_sh = sT->stride[1]; p.sT_sr = sT->stride[2]; }
    p.N = (int32_t)s.L.N; p.T = (int32_t)s.L.T; p.H = (int32_t)s.H; p.G = (int32_t)s.G;
    p.dt_bf16 = dt->dtype == KDA_BF16; p.softplus = s.softplus;
    p.s0_bf16 = s0 && s0->dtype == KDA_BF16; p.sT_bf16 = sT && sT->dtype == KDA_BF16;
    p.seg = (int32_t)s.seg; p.own_start = s.own_start;
    p.fine = s.slots * s.wps <= SSM_CUS; p.slots = (int32_t)s.slots; p.wg_per_slot = (int32_t)s.wps; p.heads_per_wg = s.hpw;
    p.wide = aligned_to(x, 8) && aligned_to(B, 8) && aligned_to(C, 8) && aligned_to(s.tz, 8) && aligned_to(out, 8);
    p.ws_state = (float *)ws;
    p.ws_decay = ws ? (float *)((char *)ws + s.off_decay) : nullptr;
    const bool f32 = x->dtype == KDA_F32;
    hipError_t e;
    if (s.seg) {
        if ((e = timed("kda_ssm_states", st, [&] { return kda::launch_ssm(p, (int)s.P, (int)s.N, f32, true, st); })) != hipSuccess)
            return hip_fail(e, "segment state launch");
        if (!p.own_start && (e = timed("kda_ssm_scan", st, [&] { return kda::launch_ssm_scan(p, (int)s.P, (int)s.N, st); })) != hipSuccess)
            return hip_fail(e, "segment scan launch");
    }
    if ((e = timed("kda_ssm", st, [&] { return kda::launch_ssm(p, (int)s.P, (int)s.N, f32, false, st); })) != hipSuccess)
        return hip_fail(e, "scan launch");
    return KDA_OK;
}

kda_status_t ssm_decode(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A, const kda_tensor_t *B,
                        const kda_tensor_t *C, kda_tensor_t *pool, const kda_tensor_t *idx, const kda_tensor_t *ntok,
                        kda_tensor_t *out, int32_t update, const kda_ssm_options_t *o, hipStream_t st)
{
    const kda_tensor_t *tz = o ? o->z : nullptr;
    KDA_TRY(check_basic(x, "x", false));
    KDA_TRY(check_basic(dt, "dt", false));
    KDA_TRY(check_basic(A, "A", false));
    KDA_TRY(check_basic(B, "B", false));
    KDA_TRY(check_basic(C, "C", false));
    KDA_TRY(check_basic(pool, "state_pool", false));
    KDA_TRY(check_basic(idx, "state_indices", false));
    KDA_TRY(check_basic(ntok, "num_tokens", true));
    KDA_TRY(check_basic(out, "out", true));
    KDA_TRY(check_basic(tz, "z", true));
    if (!is_float(x)) return fail(KDA_ERR_DTYPE, "x must be bf16 or fp32");
    if (B->dtype != x->dtype || C->dtype != x->dtype || (out && out->dtype != x->dtype) || (tz && tz->dtype != x->dtype))
        return fail(KDA_ERR_DTYPE, "x, B, C, z and out must share one dtype");
    if (dt->dtype != x->dtype && dt->dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "dt must have x's dtype or be fp32");
    if (x->ndim != 4) return fail(KDA_ERR_SHAPE, "x must be [R, T, H, P]");
    const int64_t R = x->shape[0], T = x->shape[1], H = x->shape[2], P = x->shape[3];
    if (B->ndim != 4) return fail(KDA_ERR_SHAPE, "B must be [R, T, G, N]");
    const int64_t G = B->shape[2], N = B->shape[3];
    KDA_TRY(ssm_sizes(H, P, G, N));
    KDA_TRY(ssm_vectors(A, o, H));
    KDA_TRY(ssm_state(pool, "state_pool", -1, H, N, P));
    KDA_TRY(decode_common(idx, ntok, R, T, pool->shape[0]));
    auto like = [&](const kda_tensor_t *t, const char *name, int64_t a, int64_t b) -> kda_status_t {
        if (t->ndim != 4 || t->shape[0] != R || t->shape[1] != T || t->shape[2] != a || t->shape[3] != b)
            return fail(KDA_ERR_SHAPE, "%s must be [%lld, %lld, %lld, %lld]", name, (long long)R, (long long)T, (long long)a, (long long)b);
        return KDA_OK;
    };
    KDA_TRY(like(B, "B", G, N));
    KDA_TRY(like(C, "C", G, N));
    if (out) KDA_TRY(like(out, "out", H, P));
    if (tz) KDA_TRY(like(tz, "z", H, P));
    if (dt->ndim != 3 || dt->shape[0] != R || dt->shape[1] != T || dt->shape[2] != H)
        return fail(KDA_ERR_SHAPE, "dt must be [R, T, H]");
    if (R * H > (int64_t)INT32_MAX) return fail(KDA_ERR_UNSUPPORTED, "too many workgroups for one launch");
    for (const kda_tensor_t *t : {(const kda_tensor_t *)pool, (const kda_tensor_t *)out, tz})
        if (!aligned_to(t, 4)) return fail(KDA_ERR_LAYOUT, "state_pool, out and z need 4-element-aligned base addresses and strides");
    const Named ins[] = {{x, "x"}, {dt, "dt"}, {A, "A"}, {B, "B"}, {C, "C"}, {idx, "state_indices"}, {ntok, "num_tokens"},
                         {o ? o->D : nullptr, "D"}, {o ? o->dt_bias : nullptr, "dt_bias"}, {tz, "z"}};
    KDA_TRY(no_overlap(out, "out", ins));
    KDA_TRY(no_overlap(pool, "state_pool", ins));
    if (out && overlaps(span_of(pool), span_of(out))) return fail(KDA_ERR_ALIAS, "out overlaps state_pool");
    KDA_TRY(distinct_rows(out, "out"));
    KDA_TRY(distinct_rows(pool, "state_pool"));
    if (R == 0 || (!out && !update)) return KDA_OK;
    kda::SsmDecodeParams p{};
    p.x = x->data; p.B = B->data; p.C = C->data; p.dt = dt->data; p.z = tz ? tz->data : nullptr;
    p.o = out ? out->data : nullptr; p.pool = pool->data;
    p.A = (const float *)A->data;
    p.Dv = o && o->D ? (const float *)o->D->data : nullptr;
    p.dt_bias = o && o->dt_bias ? (const float *)o->dt_bias->data : nullptr;
    p.idx = (const int32_t *)idx->data; p.ntok = ntok ? (const int32_t *)ntok->data : nullptr;
    p.x_sr = x->stride[0]; p.x_st = x->stride[1]; p.x_sh = x->stride[2];
    if (tz) { p.z_sr = tz->stride[0]; p.z_st = tz->stride[1]; p.z_sh = tz->stride[2]; }
    if (out) { p.o_sr = out->stride[0]; p.o_st = out->stride[1]; p.o_sh = out->stride[2]; }
    p.B_sr = B->stride[0]; p.B_st = B->stride[1]; p.B_sg = B->stride[2];
    p.C_sr = C->stride[0]; p.C_st = C->stride[1]; p.C_sg = C->stride[2];
    p.dt_sr = dt->stride[0]; p.dt_st = dt->stride[1]; p.dt_sh = dt->stride[2];
    p.p_sn = pool->stride[0]; p.p_sh = pool->stride[1]; p.p_sr = pool->stride[2];
    p.R = (int32_t)R; p.T = (int32_t)T; p.H = (int32_t)H; p.G = (int32_t)G; p.P = (int32_t)pool->shape[0];
    p.dt_bf16 = dt->dtype == KDA_BF16; p.softplus = o ? o->dt_softplus : 0; p.update = update != 0;
    if (update) KDA_TRY(check_slots(p.idx, R, p.P, st));
    hipError_t e = timed("kda_ssm_decode", st, [&] {
        return kda::launch_ssm_decode(p, (int)P, (int)N, x->dtype == KDA_F32, pool->dtype == KDA_BF16, st);
    });
    return e == hipSuccess ? KDA_OK : hip_fail(e, "scan decode launch");
}

}  // namespace

extern "C" {

kda_status_t kda_conv(const kda_tensor_t *x, const kda_tensor_t *weight, const kda_tensor_t *bias,
                      const kda_tensor_t *initial_state, const kda_tensor_t *cu_seqlens, kda_tensor_t *out,
                      kda_tensor_t *final_state, int32_t activation, void *stream)
{
    return guarded([&] {
        return conv(x, weight, bias, initial_state, cu_seqlens, out, final_state, activation, (hipStream_t)stream);
    });
}

kda_status_t kda_conv_decode(const kda_tensor_t *x, const kda_tensor_t *weight, const kda_tensor_t *bias,
                             kda_tensor_t *state_pool, const kda_tensor_t *state_indices,
                             const kda_tensor_t *num_tokens, kda_tensor_t *out, int32_t update_state,
                             int32_t activation, void *stream)
{
    return guarded([&] {
        return conv_decode(x, weight, bias, state_pool, state_indices, num_tokens, out, update_state, activation,
                           (hipStream_t)stream);
    });
}

kda_status_t kda_qk_norm(const kda_tensor_t *q, const kda_tensor_t *k, const kda_tensor_t *q_weight,
                         const kda_tensor_t *k_weight, const kda_tensor_t *positions, const kda_tensor_t *inv_freq,
                         kda_tensor_t *q_out, kda_tensor_t *k_out, const kda_qk_norm_options_t *opts, void *stream)
{
    return guarded([&] {
        return qk_norm(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, opts, (hipStream_t)stream);
    });
}

kda_status_t kda_ssm_workspace_size(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                                    const kda_tensor_t *B, const kda_tensor_t *C, const kda_tensor_t *initial_state,
                                    const kda_tensor_t *cu_seqlens, const kda_tensor_t *out,
                                    const kda_tensor_t *final_state, const kda_ssm_options_t *opts, size_t *bytes)
{
    return guarded([&]() -> kda_status_t {
        if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
        Ssm s;
        KDA_TRY(ssm_check(x, dt, A, B, C, initial_state, cu_seqlens, out, final_state, opts, s));
        *bytes = s.bytes;
        return KDA_OK;
    });
}

kda_status_t kda_ssm_prefill_ws(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                                const kda_tensor_t *B, const kda_tensor_t *C, const kda_tensor_t *initial_state,
                                const kda_tensor_t *cu_seqlens, kda_tensor_t *out, kda_tensor_t *final_state,
                                const kda_ssm_options_t *opts, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> kda_status_t {
        Ssm s;
        KDA_TRY(ssm_check(x, dt, A, B, C, initial_state, cu_seqlens, out, final_state, opts, s));
        if (s.bytes) {
            if (workspace_bytes < s.bytes || !workspace)
                return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, s.bytes);
            if ((uintptr_t)workspace % 256) return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
            const Span w{(uintptr_t)workspace, (uintptr_t)workspace + s.bytes};
            for (const kda_tensor_t *t : {x, dt, A, B, C, initial_state, cu_seqlens, (const kda_tensor_t *)out,
                                          (const kda_tensor_t *)final_state, s.tD, s.tbias, s.tz})
                if (overlaps(w, span_of(t))) return fail(KDA_ERR_ALIAS, "the workspace overlaps a tensor");
        }
        return ssm_run(x, dt, A, B, C, initial_state, out, final_state, s, s.bytes ? workspace : nullptr, (hipStream_t)stream);
    });
}

kda_status_t kda_ssm_prefill(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                             const kda_tensor_t *B, const kda_tensor_t *C, const kda_tensor_t *initial_state,
                             const kda_tensor_t *cu_seqlens, kda_tensor_t *out, kda_tensor_t *final_state,
                             const kda_ssm_options_t *opts, void *stream)
{
    return guarded([&]() -> kda_status_t {
        Ssm s;
        KDA_TRY(ssm_check(x, dt, A, B, C, initial_state, cu_seqlens, out, final_state, opts, s));
        auto call = [&](void *ws) { return ssm_run(x, dt, A, B, C, initial_state, out, final_state, s, ws, (hipStream_t)stream); };
        if (s.bytes == 0) return call(nullptr);
        return with_cached_ws(s.bytes, stream, [](void *ws, void *arg) { return (*(decltype(call) *)arg)(ws); }, &call);
    });
}

kda_status_t kda_ssm_decode(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                            const kda_tensor_t *B, const kda_tensor_t *C, kda_tensor_t *state_pool,
                            const kda_tensor_t *state_indices, const kda_tensor_t *num_tokens, kda_tensor_t *out,
                            int32_t update_state, const kda_ssm_options_t *opts, void *stream)
{
    return guarded([&] {
        return ssm_decode(x, dt, A, B, C, state_pool, state_indices, num_tokens, out, update_state, opts, (hipStream_t)stream);
    });
}

}  // extern "C"
