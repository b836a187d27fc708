// SSM: the selective state space scan over prompts,
//     S_t = e^{a_t} S_{t-1} + step_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,   out = y silu(z),
// a_t = A step_t, one decay per head and token, S an N x P matrix per head.
//
// Chunks of L = 32 tokens, with c_i = a_1 + ... + a_i inside the chunk:
//     Y^T = X^T (B C^T o E) + (S^T C^T) diag(e^{c_i}),   E_ji = step_j e^{c_i - c_j} for j <= i, else 0
//     S  <- e^{c_L} S + B^T diag(step_j e^{c_L - c_j}) X
// every exponent a difference taken directly (no factor can overflow when a <= 0); the ones of
// the state use sums from the chunk's end, so that the weights near 1 keep full precision.
//
// One wave owns 32 value columns of one head's state, in MFMA 32x32 accumulators for the whole
// chain, and forms everything those columns need: B C^T (32 x 32, 16 FMAs' worth of matrix time a
// wave, cheaper than sharing it through LDS and a barrier), Y^T and the state update.  The
// accumulator layout (lane = column, registers = rows) is the next product's operand as it
// stands: B C^T becomes the B operand of X^T (..), and S the A operand S^T.  B and C rows are
// shared by the workgroup's waves (two heads of a group for P = 64) in LDS, double-buffered, one
// barrier a chunk; x and z tiles belong to one wave each and need none.
// LDS rows are permuted in units of 4 elements so that both the row reads (32 rows, 8 bytes) and
// the transposed reads (4 rows, 32 bytes a 16-lane group) touch every bank once.
//
// Precision on bf16 data: x, B, C enter exactly; weighted x is split into three bf16 parts (24
// bits) for the state update, so states carry fp32 precision; the decayed B C^T and the copy of S
// that only feed the bf16 output are rounded to bf16 once (2^-9 relative each).
//
// Sequences too few to fill the chip are cut into segments of equal length: pass 1 runs every
// segment but the last of its sequence from a zero state (state update only), a scan turns the end
// states into start states (a segment's map is its decay and its end state: the decay is one
// number per head), pass 2 runs all segments from their start states.
#include <type_traits>

#include "kda_layer.hpp"

namespace kda {
namespace ssm {

constexpr int L = SSM_CHUNK;

// Physical unit of logical unit u (4 elements) of row r in a tile of U units a row.  32 row reads
// at one u, and 4 rows x 8 units of a transposed read, each spread over all 64 banks (bf16).
template <int U>
__device__ __forceinline__ int unit(int r, int u)
{
    if constexpr (U == 32) return u ^ (((r & 3) << 3) | ((r >> 2) & 7));
    else if constexpr (U == 16) return u ^ ((((r >> 1) & 1) << 3) | ((r >> 2) & 7));
    else return u ^ ((r >> 2) & 7);
}

// 4 consecutive elements of row r, logical unit u
template <typename ET, int U>
__device__ __forceinline__ typename Vec4<ET>::raw lds_unit(const ET *tile, int r, int u)
{
    return Vec4<ET>::load(tile + (r * U + unit<U>(r, u)) * 4);
}

// operand fragment: row r, elements 16 ks + 4 g + 0..3 and 16 ks + 8 + 4 g + 0..3
template <typename ET, int U>
__device__ __forceinline__ void row_frag(Frag8<ET> &f, const ET *tile, int r, int ks, int g)
{
    f.load44(tile + (r * U + unit<U>(r, 4 * ks + g)) * 4, tile + (r * U + unit<U>(r, 4 * ks + 2 + g)) * 4);
}

// operand fragment of the transpose: element k of lane l is tile[row 16 ks + 4 g + k (k < 4) or
// 16 ks + 8 + 4 g + k - 4][32 m + l % 32]
template <typename ET, int U>
__device__ __forceinline__ void col_frag(Frag8<ET> &f, const ET *tile, int ks, int m, int lane)
{
    const int g = lane >> 5;
    if constexpr (sizeof(ET) == 2) {
        const int r = 16 * ks + 4 * g + ((lane & 15) >> 2), u = 8 * m + 4 * ((lane >> 4) & 1) + (lane & 3);
        f.load44_tr(tile + (r * U + unit<U>(r, u)) * 4, tile + ((r + 8) * U + unit<U>(r + 8, u)) * 4);
    } else {
        const int c = 32 * m + (lane & 31);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 16 * ks + 4 * g + (k & 3) + 8 * (k >> 2);
            f.v[k] = tile[(r * U + unit<U>(r, c >> 2)) * 4 + (c & 3)];
        }
    }
}

// A tile of 32 rows of `cols` elements on its way from HBM to LDS: `per` threads of index t move
// 8 elements (bf16) or 4 (fp32) each, K times.
template <typename ET, int COLS, int PER>
struct TileRegs {
    static constexpr int EPV = sizeof(ET) == 2 ? 8 : 4;      // elements of a 16-byte piece
    static constexpr int PIECES = L * COLS / EPV, K = PIECES / PER, PPR = COLS / EPV;
    static_assert(PIECES % PER == 0, "whole pieces");
    uint4 v[K];
    // rows past `rows` become zeros.  wide: every piece is 16-byte aligned; else 8-byte (bf16)
    __device__ __forceinline__ void load(const ET *p, int64_t stride, int rows, int t, bool wide)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int piece = t + k * PER, r = piece / PPR, c = piece % PPR;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
                const ET *s = p + r * stride + c * EPV;
                if (wide || sizeof(ET) == 4) {
                    x = *(const uint4 *)s;
                } else {
                    const uint2 a = *(const uint2 *)s, b = *(const uint2 *)(s + 4);
                    x = make_uint4(a.x, a.y, b.x, b.y);
                }
            }
            v[k] = x;
        }
    }
    __device__ __forceinline__ void store(ET *tile, int t) const
    {
        constexpr int U = COLS / 4;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int piece = t + k * PER, r = piece / PPR, c = piece % PPR;
            if constexpr (sizeof(ET) == 4) {
                *(uint4 *)(tile + (r * U + unit<U>(r, c)) * 4) = v[k];
            } else {
                // the two units of a piece stay neighbours, in one order or the other
                const int a = unit<U>(r, 2 * c);
                const bool odd = a & 1;
                const uint4 x = v[k];
                *(uint4 *)(tile + (r * U + (a & ~1)) * 4) =
                    make_uint4(odd ? x.z : x.x, odd ? x.w : x.y, odd ? x.x : x.z, odd ? x.y : x.w);
            }
        }
    }
};

// The three bf16 parts of 8 fp32 values: hi + mid + lo holds 24 bits.
__device__ __forceinline__ void split3(const float (&f)[8], Frag8<bf16> (&o)[3])
{
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = f[e];
#pragma unroll
    for (int part = 0; part < 3; ++part) {
        o[part].set(r);
        if (part < 2) {
            const uint4 u = __builtin_bit_cast(uint4, o[part].v);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r[2 * e] -= __builtin_bit_cast(float, w[e] << 16);
                r[2 * e + 1] -= __builtin_bit_cast(float, w[e] & 0xffff0000u);
            }
        }
    }
}

// softplus without cancellation for steps far below 1
__device__ __forceinline__ float step_of(float v, int softplus)
{
    return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

struct Place {
    int n;              // sequence
    int64_t tok;        // first token: flat (packed) or within the sequence (dense)
    int len;            // tokens of this workgroup
    bool first, last;   // first / last segment of its sequence
    bool ok;
};

// What slot runs: a whole sequence, or one segment.  Packed batches number their slots
// conservatively: sequence n owns slots cu[n] / seg + n onwards, enough for its segments whatever
// the other lengths are; the ones left over exit.
__device__ __forceinline__ Place place(const SsmParams &p, int slot)
{
    Place w{};
    if (p.seg == 0) {
        w.n = slot;
        w.tok = p.cu ? p.cu[slot] : 0;
        w.len = p.cu ? p.cu[slot + 1] - p.cu[slot] : p.T;
        w.first = w.last = w.ok = true;
        return w;
    }
    int idx, len;
    if (p.cu) {
        int lo = 0, hi = p.N;           // the largest n with cu[n] / seg + n <= slot
        while (hi - lo > 1) {
            const int step = (hi - lo + 15) / 16;
            int c = 0;
#pragma unroll
            for (int k = 1; k < 16; ++k) {
                const int i = min(lo + k * step, hi);
                c += (i < hi && p.cu[i] / p.seg + i <= slot) ? 1 : 0;
            }
            lo += c * step;
            hi = min(hi, lo + step);
        }
        w.n = lo;
        idx = slot - (p.cu[lo] / p.seg + lo);
        len = p.cu[lo + 1] - p.cu[lo];
        w.tok = p.cu[lo] + (int64_t)idx * p.seg;
    } else {
        const int per = max(1, (p.T + p.seg - 1) / p.seg);
        w.n = slot / per;
        idx = slot % per;
        len = p.T;
        w.tok = (int64_t)idx * p.seg;
    }
    const int64_t left = (int64_t)len - (int64_t)idx * p.seg;
    w.first = idx == 0;
    w.last = left <= p.seg;
    w.len = (int)max((int64_t)0, min(left, (int64_t)p.seg));
    w.ok = idx == 0 || left > 0;
    return w;
}

// Offset of accumulator registers 4 q .. 4 q + 3 of tile m of a state, in the workspace's order
// (the order a wave holds it in, 16 bytes a lane).
template <int P, int N>
__device__ __forceinline__ int ws_index(int slab, int m, int q, int lane)
{
    return ((slab * (N / 32) + m) * 4 + q) * 256 + lane * 4;
}

template <typename ET, int P, int N, int HPW, bool OUT>
__global__ __launch_bounds__(HPW * P * 2, 2) void ssm_kernel(const SsmParams p)
{
    constexpr int NW = HPW * P / 32, NT = NW * 64;      // waves, threads
    constexpr int SLABS = P / 32, NM = N / 32, U = N / 4;
    __shared__ __attribute__((aligned(16))) ET sB[2][L * N];
    __shared__ __attribute__((aligned(16))) ET sC[OUT ? 2 : 1][OUT ? L * N : 4];
    __shared__ __attribute__((aligned(16))) ET sX[NW][L * 32];
    __shared__ __attribute__((aligned(16))) ET sZ[OUT ? NW : 1][OUT ? L * 32 : 4];
    // c log2 e, step, state weight; on fp32 data also the low part of c: after a large decay the
    // differences c_i - c_j of two 32-bit sums would keep too few digits for an fp32 output
    constexpr bool FINE = sizeof(ET) == 4;
    __shared__ __attribute__((aligned(16))) float sAux[NW][FINE ? 4 : 3][L];

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / p.wg_per_slot, wgi = blockIdx.x % p.wg_per_slot;
    const Place w = place(p, slot);
    if (!w.ok || (!OUT && w.last)) return;
    // heads: this workgroup's HPW heads of one group (a wave past the group's last head repeats it
    // and stores nothing)
    const int hg = p.H / p.G, wpg = (hg + HPW - 1) / HPW, grp = wgi / wpg;
    const int hi = (wgi % wpg) * HPW + wave / SLABS, slab = wave % SLABS;
    const bool live = hi < hg;
    const int h = grp * hg + min(hi, hg - 1);

    const int64_t seq = p.cu ? 0 : w.n;
    const ET *x = (const ET *)p.x + seq * p.x_sb + w.tok * p.x_st + h * p.x_sh + slab * 32;
    const ET *Bp = (const ET *)p.B + seq * p.B_sb + w.tok * p.B_st + grp * p.B_sg;
    const ET *Cp = (const ET *)p.C + seq * p.C_sb + w.tok * p.C_st + grp * p.C_sg;
    const ET *z = p.z ? (const ET *)p.z + seq * p.z_sb + w.tok * p.z_st + h * p.z_sh + slab * 32 : nullptr;
    ET *o = (ET *)p.o + seq * p.o_sb + w.tok * p.o_st + h * p.o_sh + slab * 32;
    const int64_t dt0 = seq * p.dt_sb + w.tok * p.dt_st + h * p.dt_sh;
    const float a2 = p.A[h] * LOG2E, bias = p.dt_bias ? p.dt_bias[h] : 0.f, skip = p.Dv ? p.Dv[h] : 0.f;

    // start state
    f32x16 S[NM];
    float *ws = p.seg ? p.ws_state + ((int64_t)slot * p.H + h) * (N * P) : nullptr;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        if (OUT && p.seg) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = *(const float4 *)(ws + ws_index<P, N>(slab, m, q, lane));
                S[m][4 * q] = v.x; S[m][4 * q + 1] = v.y; S[m][4 * q + 2] = v.z; S[m][4 * q + 3] = v.w;
            }
        } else if (OUT && p.s0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = 32 * m + 8 * (e >> 2) + 4 * g + (e & 3);
                S[m][e] = ld_any(p.s0, w.n * p.s0_sn + h * p.s0_sh + row * p.s0_sr + slab * 32 + l32, p.s0_bf16);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) S[m][e] = 0.f;
        }
    }

    TileRegs<ET, N, NT> rB, rC;
    TileRegs<ET, 32, 64> rX, rZ;
    float rdt = 0.f;
    const int nck = (w.len + L - 1) / L;
    auto load = [&](int c) {
        const int rows = min(L, w.len - c * L);
        const int64_t t = (int64_t)c * L;
        rB.load(Bp + t * p.B_st, p.B_st, rows, tid, p.wide);
        if constexpr (OUT) rC.load(Cp + t * p.C_st, p.C_st, rows, tid, p.wide);
        rX.load(x + t * p.x_st, p.x_st, rows, lane, p.wide);
        if constexpr (OUT)
            if (z) rZ.load(z + t * p.z_st, p.z_st, rows, lane, p.wide);
        rdt = l32 < rows ? ld_any(p.dt, dt0 + (t + l32) * p.dt_st, p.dt_bf16) : 0.f;
    };
    if (nck > 0) load(0);
    float total2 = 0.f;         // sum of a over the segment, in powers of two
    for (int c = 0; c < nck; ++c) {
        const int rows = min(L, w.len - c * L);
        ET *tB = sB[c & 1], *tC = sC[OUT ? c & 1 : 0], *tX = sX[wave], *tZ = sZ[OUT ? wave : 0];
        rB.store(tB, tid);
        if constexpr (OUT) rC.store(tC, tid);
        rX.store(tX, lane);
        if constexpr (OUT)
            if (z) rZ.store(tZ, lane);
        // decays of the chunk: token i = lane % 32; tokens past the end have step 0
        const float step = l32 < rows ? step_of(rdt + bias, p.softplus) : 0.f;
        const float a = step * a2;
        typedef std::conditional_t<FINE, double, float> sum_t;
        sum_t cs = a;
        float ri = a;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const sum_t u = __shfl_up(cs, off, 32);
            const float d = __shfl_down(ri, off, 32);
            cs += l32 >= off ? u : (sum_t)0;
            ri += l32 + off < 32 ? d : 0.f;
        }
        const float ci = (float)cs, cl = (float)(cs - (sum_t)ci);       // cl: 0 unless FINE
        const float tot = __shfl(ci, 31, 32);
        float rev = __shfl_down(ri, 1, 32);
        rev = l32 == 31 ? 0.f : rev;                // sum over the tokens after i
        if (g == 0) {
            sAux[wave][0][l32] = ci;
            sAux[wave][1][l32] = step;
            sAux[wave][2][l32] = step * __builtin_amdgcn_exp2f(rev);
            if constexpr (FINE) sAux[wave][3][l32] = cl;
        }
        __syncthreads();
        if (c + 1 < nck) load(c + 1);

        // x^T fragments: lane = column, elements = tokens
        Frag8<ET> fx[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) col_frag<ET, 8>(fx[ks], tX, ks, 0, lane);

        if constexpr (OUT) {
            f32x16 G = {}, Y = {};
#pragma unroll
            for (int ks = 0; ks < N / 16; ++ks) {
                Frag8<ET> fb, fc, fs;
                row_frag<ET, U>(fc, tC, l32, ks, g);
                row_frag<ET, U>(fb, tB, l32, ks, g);
                float t8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t8[e] = S[ks >> 1][8 * (ks & 1) + e];
                fs.set(t8);
                mma32(G, fb, fc);           // (B C^T)[j][i]: column i = lane
                mma32(Y, fs, fc);           // (S^T C^T)[p][i]
            }
            const float ei = __builtin_amdgcn_exp2f(ci);
#pragma unroll
            for (int e = 0; e < 16; ++e) Y[e] *= ei;
            float M[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 cj = *(const float4 *)&sAux[wave][0][8 * q + 4 * g];
                const float4 sj = *(const float4 *)&sAux[wave][1][8 * q + 4 * g];
                const float c4[4] = {cj.x, cj.y, cj.z, cj.w}, s4[4] = {sj.x, sj.y, sj.z, sj.w};
                float d4[4] = {ci - c4[0], ci - c4[1], ci - c4[2], ci - c4[3]};
                if constexpr (FINE) {
                    const float4 lj = *(const float4 *)&sAux[wave][3][8 * q + 4 * g];
                    d4[0] += cl - lj.x; d4[1] += cl - lj.y; d4[2] += cl - lj.z; d4[3] += cl - lj.w;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = G[4 * q + r] * (__builtin_amdgcn_exp2f(d4[r]) * s4[r]);
                    M[4 * q + r] = 8 * q + 4 * g + r <= l32 ? v : 0.f;
                }
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag8<ET> fm;
                float t8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t8[e] = M[8 * ks + e];
                fm.set(t8);
                mma32(Y, fx[ks], fm);
            }
            // lane = token, registers = columns 8 q + 4 g + 0..3
            if (live && l32 < rows) {
                ET *dst = o + ((int64_t)c * L + l32) * p.o_st + 4 * g;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x4[4], y4[4];
                    Vec4<ET>::unpack(lds_unit<ET, 8>(tX, l32, 2 * q + g), x4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y4[r] = __builtin_fmaf(skip, x4[r], Y[4 * q + r]);
                    if (z) {
                        float z4[4];
                        Vec4<ET>::unpack(lds_unit<ET, 8>(tZ, l32, 2 * q + g), z4);
#pragma unroll
                        for (int r = 0; r < 4; ++r) y4[r] *= silu_act(z4[r]);
                    }
                    Vec4<ET>::store(dst + 8 * q, Vec4<ET>::pack(y4));
                }
            }
        }
        // state update
        const float et = __builtin_amdgcn_exp2f(tot);
        total2 += tot;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) S[m][e] *= et;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const float4 wa = *(const float4 *)&sAux[wave][2][16 * ks + 4 * g];
            const float4 wb = *(const float4 *)&sAux[wave][2][16 * ks + 8 + 4 * g];
            const float w8[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
            float xw[8];
            if constexpr (sizeof(ET) == 2) {
                const uint4 u = __builtin_bit_cast(uint4, fx[ks].v);
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xw[2 * e] = __builtin_bit_cast(float, uw[e] << 16) * w8[2 * e];
                    xw[2 * e + 1] = __builtin_bit_cast(float, uw[e] & 0xffff0000u) * w8[2 * e + 1];
                }
                Frag8<bf16> part[3];
                split3(xw, part);
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    Frag8<bf16> fb;
                    col_frag<bf16, U>(fb, tB, ks, m, lane);
#pragma unroll
                    for (int i = 0; i < 3; ++i) mma32(S[m], fb, part[i]);
                }
            } else {
                Frag8<float> fw;
#pragma unroll
                for (int e = 0; e < 8; ++e) fw.v[e] = fx[ks].v[e] * w8[e];
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    Frag8<float> fb;
                    col_frag<float, U>(fb, tB, ks, m, lane);
                    mma32(S[m], fb, fw);
                }
            }
        }
    }
    if constexpr (!OUT) {
        if (!live) return;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(float4 *)(ws + ws_index<P, N>(slab, m, q, lane)) =
                    make_float4(S[m][4 * q], S[m][4 * q + 1], S[m][4 * q + 2], S[m][4 * q + 3]);
        if (slab == 0 && lane == 0) p.ws_decay[(int64_t)slot * p.H + h] = total2;
    } else if (live && w.last && p.sT) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = 32 * m + 8 * (e >> 2) + 4 * g + (e & 3);
                const int64_t i = w.n * p.sT_sn + h * p.sT_sh + row * p.sT_sr + slab * 32 + l32;
                if (p.sT_bf16) ((bf16 *)p.sT)[i] = (bf16)S[m][e];
                else ((float *)p.sT)[i] = S[m][e];
            }
    }
}

// Start states from end states: one thread per 4 state elements of a (sequence, head), walking
// the sequence's segments.  The workspace slot of a segment holds its end state (from zero) on
// entry and its start state on return; the last segment's end state is never needed.
template <int P, int N>
__global__ __launch_bounds__(256) void ssm_scan_kernel(const SsmParams p)
{
    constexpr int BPS = N * P / 1024;       // workgroups per state
    const int part = blockIdx.x % BPS;
    const int64_t chain = blockIdx.x / BPS;
    const int n = (int)(chain / p.H), h = (int)(chain % p.H);
    const int i4 = part * 256 + threadIdx.x, lane = i4 & 63, g = lane >> 5;
    const int q = (i4 >> 6) & 3, m = (i4 >> 8) % (N / 32), slab = i4 / (64 * 4 * (N / 32));
    int slot, count;
    if (p.cu) {
        slot = p.cu[n] / p.seg + n;
        count = max(1, (p.cu[n + 1] - p.cu[n] + p.seg - 1) / p.seg);
    } else {
        count = max(1, (p.T + p.seg - 1) / p.seg);
        slot = n * count;
    }
    float s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        s[r] = p.s0 ? ld_any(p.s0, n * p.s0_sn + h * p.s0_sh + (32 * m + 8 * q + 4 * g + r) * p.s0_sr + slab * 32 + (lane & 31),
                             p.s0_bf16)
                    : 0.f;
    float *ws = p.ws_state + ((int64_t)slot * p.H + h) * (N * P) + i4 * 4;
    const float *dec = p.ws_decay + (int64_t)slot * p.H + h;
    const int64_t step = (int64_t)p.H * (N * P);
    for (int k = 0; k + 1 < count; ++k) {
        const float4 e = *(const float4 *)ws;
        const float d = __builtin_amdgcn_exp2f(*dec);
        *(float4 *)ws = make_float4(s[0], s[1], s[2], s[3]);
        s[0] = __builtin_fmaf(s[0], d, e.x);
        s[1] = __builtin_fmaf(s[1], d, e.y);
        s[2] = __builtin_fmaf(s[2], d, e.z);
        s[3] = __builtin_fmaf(s[3], d, e.w);
        ws += step;
        dec += p.H;
    }
    *(float4 *)ws = make_float4(s[0], s[1], s[2], s[3]);
}

template <typename ET, int P, int N, int HPW>
static hipError_t launch_t(const SsmParams &p, bool states_only, hipStream_t st)
{
    const int64_t blocks = (int64_t)p.slots * p.wg_per_slot;
    if (blocks <= 0) return hipSuccess;
    if (states_only)
        hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, false>), dim3((unsigned)blocks), dim3(HPW * P * 2), 0, st, p);
    else
        hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, true>), dim3((unsigned)blocks), dim3(HPW * P * 2), 0, st, p);
    return hipGetLastError();
}

}  // namespace ssm

hipError_t launch_ssm(const SsmParams &p, int P, int N, bool io_f32, bool states_only, hipStream_t st)
{
#define KDA_SSM(PP, NN, HH)                                                                     \
    if (P == PP && N == NN && p.heads_per_wg == HH)                                             \
        return io_f32 ? ssm::launch_t<float, PP, NN, HH>(p, states_only, st) : ssm::launch_t<bf16, PP, NN, HH>(p, states_only, st);
    KDA_SSM(64, 64, 1)
    KDA_SSM(64, 64, 2)
    KDA_SSM(64, 128, 1)
    KDA_SSM(64, 128, 2)
    KDA_SSM(128, 64, 1)
    KDA_SSM(128, 128, 1)
#undef KDA_SSM
    return hipErrorInvalidValue;
}

hipError_t launch_ssm_scan(const SsmParams &p, int P, int N, hipStream_t st)
{
    const int64_t blocks = (int64_t)p.N * p.H * (N * P / 1024);
    if (blocks <= 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), thr(256);
    if (P == 64 && N == 64) hipLaunchKernelGGL((ssm::ssm_scan_kernel<64, 64>), grid, thr, 0, st, p);
    else if (P == 64 && N == 128) hipLaunchKernelGGL((ssm::ssm_scan_kernel<64, 128>), grid, thr, 0, st, p);
    else if (P == 128 && N == 64) hipLaunchKernelGGL((ssm::ssm_scan_kernel<128, 64>), grid, thr, 0, st, p);
    else if (P == 128 && N == 128) hipLaunchKernelGGL((ssm::ssm_scan_kernel<128, 128>), grid, thr, 0, st, p);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace kda
