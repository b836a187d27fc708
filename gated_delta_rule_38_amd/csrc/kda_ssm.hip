// SSM: the selective state space scan over prompts,
//     S_t = e^{a_t} S_{t-1} + step_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,   out = y silu(z),
// a_t = A step_t, one decay per head and token, S an N x P matrix per head.
//
// Chunks of L = 32 tokens.  With c_i the sum of a up to token i since a reference token and the
// state kept in units of the reference, S = e^{c} Z, a chunk is
//     Y^T = [Z^T C^T + (X diag(g))^T (B C^T, j <= i)] diag(e^{c_i}),   g_j = step_j e^{-c_j}
//     Z  <- Z + B^T diag(g) X
// so one weighted copy of x serves both products, the decay matrix is never formed and the state
// is not touched by decays.  The reference moves (Z <- e^{c} Z) before e^{-c} could leave 2^LIMIT;
// a chunk that decays by more than that on its own takes the direct form, every exponent a
// difference: Y^T = (Z^T C^T) diag(e^{c_i}) + X^T (B C^T o step_j e^{c_i - c_j}, j <= i) and
// Z <- e^{c_L} Z + B^T diag(step_j e^{c_L - c_j}) X.  c is summed in 64 bits: weights and decays
// then carry full 32-bit precision however far the reference is.
//
// One wave owns 16 value columns of one head's state, in MFMA 16x16 accumulators for the whole
// chain (32 registers for N = 128), so that four waves share a SIMD and one wave's conversions and
// exponentials run under another's matrix products.  The accumulator layout (lane = column,
// registers = rows) is the next product's operand as it stands: Z feeds Z^T C^T, and B C^T, formed
// once a chunk and workgroup, feeds every wave's X^T (..) through 2 KB of LDS.  A workgroup is
// 8 waves (two heads of a group for P = 64, one for P = 128) over double-buffered tiles of B, C, x
// and z; two barriers a chunk.  Steps, sums, weights and decays of 8 (chunk, head) pairs are formed
// at a time, one pair in each half of four waves.
// State rows are numbered so that the 8 registers of a lane's two tiles are 8 consecutive channels
// (the transposed reads fetch columns in that order), which makes every row access 16 bytes.  In
// LDS the 8-element units of a row are permuted by the row number so that row reads (one unit of
// each row) touch every bank once, and transposed reads (4 rows, 4 neighbouring units) twice.
//
// Precision on bf16 data: x, B, C enter exactly; weighted x is split into three bf16 parts (24
// bits) for the state update, so states carry fp32 precision, and two of them (16 bits) feed the
// output; B C^T and the copy of the state that only feed the bf16 output are rounded to bf16 once, or
// where workgroups are few kept in two parts.
//
// Sequences too few to fill the chip are cut into segments of equal length: pass 1 runs every
// segment but the last of its sequence from a zero state (state update only), the end states are
// turned into start states (a segment's map is its decay and its end state: the decay is one
// number per head) by a scan, or where a sequence has few segments by the workgroups of pass 2
// themselves, which runs all segments from their start states.
//
// What bounds it: instruction issue.  16 x 2,048 tokens, 64 heads of 64, 128 state channels, gated,
// bf16 (one pass, 0.87 GB): 285 us, 3.0 TB/s; a chunk and wave is about 230 vector instructions, 16 of
// them transcendental, and 38 matrix instructions, which keep the vector units 60% and the matrix
// units 28% busy at four waves a SIMD (LDS 46%).  A chunk takes 2.3 us with one workgroup on a CU and
// 4.3 with two.  8 prompts of 32,733 tokens: 127 + 294 us in segments of 1,280.
#include <type_traits>

#include "kda_layer.hpp"

namespace kda {
namespace ssm {

constexpr int L = SSM_CHUNK;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Element offset of unit u (8 elements) of row r in a tile of COLS columns.
template <int COLS>
__device__ __forceinline__ int unit_at(int r, int u)
{
    const int f = COLS == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    return r * COLS + ((u ^ f) << 3);
}

// The offsets one lane needs in a tile of COLS columns (l16 = lane % 16, g = lane / 16).
template <typename ET, int COLS>
struct Rows {                   // row l16 (+ 16 t): units g + 4 a
    int base;
    __device__ __forceinline__ explicit Rows(int lane) : base(unit_at<COLS>(lane & 15, lane >> 4)) {}
    // (the permutation is an exclusive or, the same for rows 16 apart)
    __device__ __forceinline__ int at(int t, int a) const { return (base ^ (a << 5)) + t * 16 * COLS; }
};

// The transposed operand of 32 tokens: element k of lane l is token 4 g + k (k < 4) or 16 + 4 g + k - 4.
// SPREAD: lane l16 stands for channel 8 (l16 / 4) + l16 % 4 (+ 4 for the odd tile) of 32, else for
// column l16.
template <typename ET, int COLS, bool SPREAD>
struct Cols {
    int base;
    __device__ __forceinline__ explicit Cols(int lane, int first)
    {
        const int g = lane >> 4;
        if constexpr (sizeof(ET) == 2) {
            // the transposing read: this lane addresses word l16 % 4 of row l16 / 4
            const int r = 4 * g + ((lane & 15) >> 2), wd = lane & 3;
            base = SPREAD ? unit_at<COLS>(r, wd) : unit_at<COLS>(r, (first >> 3) + (wd >> 1)) + (wd & 1) * 4;
        } else {
            const int c = SPREAD ? 8 * ((lane & 15) >> 2) + (lane & 3) : first + (lane & 15);
            base = unit_at<COLS>(4 * g, c >> 3) + (c & 7);
        }
    }
    // SPREAD: channels 32 a ..; odd: their upper fours
    __device__ __forceinline__ void get(Frag8<ET> &f, const ET *tile, int a, int odd) const
    {
        const ET *t = tile + (base ^ (a << 5)) + 4 * odd;
        if constexpr (sizeof(ET) == 2) {
            f.load44_tr(t, t + 16 * COLS);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // rows 1 .. 3 of a group of four: their permutations differ in the bits of row % 4
                const int d = k & 3, x = COLS == 128 ? d << 2 : ((d >> 1) & 1) << 2;
                f.v[k] = tile[(((base ^ (a << 5)) ^ (x << 3)) + 4 * odd) + (d + 16 * (k >> 2)) * COLS];
            }
        }
    }
};

// A tile of 32 rows of COLS elements on its way from HBM to LDS: PER threads move 8 elements (bf16)
// or 4 (fp32) each, K times.  The columns belong to heads of PC columns that lie `head` elements
// apart.
template <typename ET, int COLS, int PER, int PC>
struct TileRegs {
    static constexpr int EPV = sizeof(ET) == 2 ? 8 : 4;      // elements of a 16-byte piece
    static constexpr int PIECES = L * COLS / EPV, USED = PER < PIECES ? PER : PIECES;     // threads that move any
    static constexpr int K = PIECES / USED, PPR = COLS / EPV, ROWS = USED / PPR;
    static_assert(PIECES % USED == 0 && USED % PPR == 0, "whole pieces, whole rows");
    u32x4 v[K];
    uint32_t off[K];            // byte offsets from the chunk's first row
    // rows past the last one repeat it: their step is 0, so they weigh nothing
    __device__ __forceinline__ void offsets(int64_t stride, int64_t head, int heads, int rows, int t)
    {
        const int c = t % PPR * EPV;
#pragma unroll
        for (int k = 0; k < K; ++k)
            off[k] = ((uint32_t)min(t / PPR + k * ROWS, rows - 1) * (uint32_t)stride + (uint32_t)min(c / PC, heads - 1) * (uint32_t)head +
                      (uint32_t)(c % PC)) * (uint32_t)sizeof(ET);
    }
    // WIDE: every piece is 16-byte aligned; else 8-byte (bf16)
    template <bool WIDE>
    __device__ __forceinline__ void load(const ET *p, int t)
    {
        if (USED < PER && t >= USED) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const char *s = (const char *)p + off[k];
            if constexpr (WIDE || sizeof(ET) == 4) {
                v[k] = *(const u32x4 *)s;
            } else {
                const uint2 a = *(const uint2 *)s, b = *(const uint2 *)(s + 8);
                v[k] = u32x4{a.x, a.y, b.x, b.y};
            }
        }
    }
    __device__ __forceinline__ void store(ET *tile, int t) const
    {
        if (USED < PER && t >= USED) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int r = t / PPR + k * ROWS, c = t % PPR;
            // a piece is a unit (bf16) or half of one (fp32)
            *(u32x4 *)(tile + (sizeof(ET) == 2 ? unit_at<COLS>(r, c) : unit_at<COLS>(r, c >> 1) + 4 * (c & 1))) = v[k];
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

// What rounding 8 fp32 values to bf16 leaves of them, rounded to bf16.
__device__ __forceinline__ void rest_of(const float (&f)[8], Frag8<bf16> &o)
{
    Frag8<bf16> hi;
    hi.set(f);
    const uint4 u = __builtin_bit_cast(uint4, hi.v);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float r[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r[2 * e] = f[2 * e] - __builtin_bit_cast(float, w[e] << 16);
        r[2 * e + 1] = f[2 * e + 1] - __builtin_bit_cast(float, w[e] & 0xffff0000u);
    }
    o.set(r);
}

// 2^x of a 64-bit exponent, to 32-bit precision: the whole part goes into the exponent bits.
__device__ __forceinline__ float exp2_of(double x)
{
    x = fmin(fmax(x, -4096.), 4096.);
    const double n = __builtin_rint(x);
    return __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp64(double x)      // lanes without a source read 0
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Inclusive sum over the lanes of each 32-lane half: shifts within 16-lane rows, then lane 15 of
// the row before.
__device__ __forceinline__ double prefix32(double x)
{
    x += dpp64<0x111, 0xf>(x);
    x += dpp64<0x112, 0xf>(x);
    x += dpp64<0x114, 0xf>(x);
    x += dpp64<0x118, 0xf>(x);
    x += dpp64<0x142, 0xa>(x);
    return x;
}

// The reference moves before a weight could pass 2^LIMIT (and a decay fall under 2^-LIMIT): products
// of x, B and C up to 2^31 still fit an fp32 number, and the direct form (a batch of nothing else takes
// 25% longer) is left to chunks that decay by more than 2^-96.
constexpr double LIMIT = 96.;

// softplus(v) = max(v, 0) + log(1 + e^{-|v|}) without cancellation for steps far below 1: log(1 + t) is
// 2 atanh(s), s = t / (2 + t) <= 1/3, by its odd power series (the first term left out is under
// 2^-27 of the sum).
__device__ __forceinline__ float step_of(float v, int softplus)
{
    if (!softplus) return v;
    const float t = __builtin_amdgcn_exp2f(-fabsf(v) * LOG2E), d = 2.f + t;
    float r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.f), r);
    const float s = t * r, q = s * s;
    float a = 1.f / 15.f;
    a = __builtin_fmaf(a, q, 1.f / 13.f);
    a = __builtin_fmaf(a, q, 1.f / 11.f);
    a = __builtin_fmaf(a, q, 1.f / 9.f);
    a = __builtin_fmaf(a, q, 1.f / 7.f);
    a = __builtin_fmaf(a, q, 1.f / 5.f);
    a = __builtin_fmaf(a, q, 1.f / 3.f);
    a = __builtin_fmaf(a * q, s, s);
    return fmaxf(v, 0.f) + 2.f * a;
}

// The same value, but not one the compiler can compute before a loop: what depends on it stays where
// it is used instead of holding registers through the loop.
__device__ __forceinline__ int here(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

struct Place {
    int n;              // sequence
    int64_t tok;        // first token: flat (packed) or within the sequence (dense)
    int len;            // tokens of this workgroup
    int before, first;  // segments of its sequence before it, and the first one's slot
    bool last;          // the last segment of its sequence
    bool ok;
};

// The slots of a sequence's segments.  Packed batches number the full ones from cu[n] / seg on, which
// leaves room for them whatever the other lengths are, and a last one that is shorter behind all of
// those: long segments start first (a packed batch of 8 prompts, 32,733 tokens, 64 heads: 318 us in
// the sequences' order, 296 in this).
struct Cut {
    int first, full, last, len;     // slot of the first segment, segments before the last, the last one's slot; tokens
};

__device__ __forceinline__ Cut cut_of(const SsmParams &p, int n)
{
    Cut c;
    const int room = p.slots - p.N;
    c.first = p.cu ? p.cu[n] / p.seg : n * (room / p.N);
    c.len = p.cu ? p.cu[n + 1] - p.cu[n] : p.T;
    c.full = max(0, c.len - 1) / p.seg;
    c.last = p.cu && c.len > 0 && c.len % p.seg == 0 ? c.first + c.full : room + n;
    return c;
}

// What slot runs: a whole sequence, or one segment.
__device__ __forceinline__ Place place(const SsmParams &p, int slot)
{
    Place w{};
    if (p.seg == 0) {
        w.n = slot;
        w.tok = p.cu ? p.cu[slot] : 0;
        w.len = p.cu ? p.cu[slot + 1] - p.cu[slot] : p.T;
        w.last = w.ok = true;
        return w;
    }
    const int room = p.slots - p.N;
    if (slot >= room) {
        w.n = slot - room;
    } else if (p.cu) {
        int lo = 0, hi = p.N;           // the largest n with cu[n] / seg <= slot
        while (hi - lo > 1) {
            const int step = (hi - lo + 15) / 16;
            int c = 0;
#pragma unroll
            for (int k = 1; k < 16; ++k) {
                const int i = min(lo + k * step, hi);
                c += (i < hi && p.cu[i] / p.seg <= slot) ? 1 : 0;
            }
            lo += c * step;
            hi = min(hi, lo + step);
        }
        w.n = lo;
    } else {
        w.n = slot / (room / p.N);
    }
    const Cut c = cut_of(p, w.n);
    w.last = slot == c.last;
    w.ok = w.last || (slot < room && slot - c.first < c.full);
    w.first = c.first;
    w.before = w.last ? c.full : slot - c.first;
    const int64_t from = (int64_t)w.before * p.seg;
    w.tok = (p.cu ? p.cu[w.n] : 0) + from;
    w.len = w.last ? (int)(c.len - from) : p.seg;
    return w;
}

// Offset of tile m of a state's 16-column slab, in the workspace's order (the order a wave holds it
// in, 16 bytes a lane).
template <int P, int N>
__device__ __forceinline__ int ws_index(int slab, int m, int lane) { return ((slab * (N / 16) + m) * 64 + lane) * 4; }

// Channel of register r of tile m (lane group g = lane / 16).
__device__ __forceinline__ int row_of(int m, int g, int r) { return 32 * (m >> 1) + 8 * g + 4 * (m & 1) + r; }

// GATED: z is given.  FINE (bf16, as many workgroups as CUs or fewer): what only feeds the output, B C^T
// and the state's copy, keeps 16 bits too, so that the output's own rounding is all that is left of it.
// In few outputs the roundings are not evened out (on 10 tokens an error of 2.2e-3 was met where the
// output's rounding alone makes 1.3e-3), and with one workgroup on a CU it costs nothing: 10 to 2,048
// tokens in up to 256 workgroups take the same time within 2%.  Its registers let one workgroup into a
// CU instead of two: 16 x 2,048 tokens of 64 heads take 405 us with it and 286 without.
template <typename ET, int P, int N, int HPW, bool OUT, bool GATED, bool FINE>
__global__ __launch_bounds__(HPW * P * 4, sizeof(ET) == 2 ? (FINE ? 2 : 4) : 1) void ssm_kernel(const SsmParams p)
{
    constexpr int NW = HPW * P / 16, NT = NW * 64;      // waves, threads
    constexpr int SLABS = P / 16, NM = N / 16, NA = N / 32, XC = HPW * P;
    constexpr bool BF = sizeof(ET) == 2;
    constexpr int PARTS = BF ? 3 : 1;                   // of weighted x
    constexpr int GC = 8 / HPW;                         // chunks of a group
    __shared__ __attribute__((aligned(16))) ET sB[2][L * N];
    __shared__ __attribute__((aligned(16))) ET sC[OUT ? 2 : 1][OUT ? L * N : 4];
    __shared__ __attribute__((aligned(16))) ET sX[2][L * XC];
    __shared__ __attribute__((aligned(16))) ET sZ[GATED ? 2 : 1][GATED ? L * XC : 4];
    __shared__ __attribute__((aligned(16))) ET sM[OUT ? L * L : 4];     // C B^T, j <= i: row i, units of 4 j
    __shared__ __attribute__((aligned(16))) ET sRest[FINE ? L * L : 4];  // what sM's rounding left
    // of a group's chunks and heads, for each token: step, sum of a, weight of x, decay of y
    __shared__ __attribute__((aligned(16))) float sStep[2][GC][HPW][L], sWt[2][GC][HPW][L], sEi[OUT ? 2 : 1][GC][HPW][L];
    __shared__ __attribute__((aligned(16))) float2 sSum[2][GC][HPW][L];
    // and for each chunk: the factor the state takes before it, c after it, whether it is direct
    __shared__ double sBase[2][GC][HPW];
    __shared__ float sScale[2][GC][HPW];
    __shared__ int sDirect[2][GC][HPW];
    __shared__ double sA[HPW];                          // A log2 e
    __shared__ float sBias[HPW];

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / p.wg_per_slot, wgi = blockIdx.x % p.wg_per_slot;
    const Place w = place(p, slot);
    if (!w.ok || (!OUT && w.last)) return;
    // heads: this workgroup's HPW heads of one group (a wave past the group's last head repeats it
    // and stores nothing)
    const int hg = p.H / p.G, wpg = (hg + HPW - 1) / HPW, grp = wgi / wpg;
    const int h0 = grp * hg + (wgi % wpg) * HPW, heads = min(HPW, (grp + 1) * hg - h0);
    const int wh = wave / SLABS, slab = wave % SLABS;
    const bool live = wh < heads;
    const int h = h0 + min(wh, heads - 1);

    const int64_t seq = p.cu ? 0 : w.n;
    const float skip = p.Dv ? p.Dv[h] : 0.f;
    const Rows<ET, N> rn(lane);
    const Cols<ET, N, true> cn(lane, 0);
    const Cols<ET, XC, false> cx(lane, wh * P + slab * 16);
    // row l16, columns 4 g .. 4 g + 3 of this wave's slab of x and z
    const int xrow = unit_at<XC>(l16, (wh * P + slab * 16 + 4 * g) >> 3) + 4 * (g & 1);
    // row l16 of M: units of 4 j, permuted by the row
    auto m_at = [&](int i, int u) { return i * L + ((u ^ ((i >> 2) & 7)) << 2); };

    // start state
    f32x4 S[NM];
    float *ws = p.seg ? p.ws_state + ((int64_t)slot * p.H + h) * (N * P) : nullptr;
    const bool formed = OUT && p.seg && !p.own_start;       // the scan's
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        if (formed) {
            S[m] = *(const f32x4 *)(ws + ws_index<P, N>(slab, m, lane));
        } else if (OUT && p.s0) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[m][r] = ld_any(p.s0, w.n * p.s0_sn + h * p.s0_sh + row_of(m, g, r) * p.s0_sr + slab * 16 + l16, p.s0_bf16);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = 0.f;
        }
    }
    if (OUT && p.seg && p.own_start && w.before > 0) {
        // the walk over the segments before this one, the next one's end state in flight
        const float *end = p.ws_state + ((int64_t)w.first * p.H + h) * (N * P) + ws_index<P, N>(slab, 0, lane);
        const float *dec = p.ws_decay + (int64_t)w.first * p.H + h;
        f32x4 e[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) e[m] = *(const f32x4 *)(end + m * 256);
        for (int k = 0; k < w.before; ++k) {
            f32x4 next[NM];
            end += k + 1 < w.before ? (int64_t)p.H * (N * P) : 0;
#pragma unroll
            for (int m = 0; m < NM; ++m) next[m] = *(const f32x4 *)(end + m * 256);
            const float d = dec[(int64_t)k * p.H];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][r] = __builtin_fmaf(S[m][r], d, e[m][r]);
                e[m] = next[m];
            }
        }
    }
    auto scale_state = [&](float f) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] *= f;
    };

    TileRegs<ET, N, NT, N> rB, rC;
    const int tc = tid ^ (NT / 2);      // (where half the threads move a tile, B and C take one half each)
    TileRegs<ET, XC, NT, P> rX, rZ;
    const int nck = (w.len + L - 1) / L;
    const ET *Bp = (const ET *)p.B + seq * p.B_sb + w.tok * p.B_st + grp * p.B_sg;
    const ET *Cp = (const ET *)p.C + seq * p.C_sb + w.tok * p.C_st + grp * p.C_sg;
    const ET *xp = (const ET *)p.x + seq * p.x_sb + w.tok * p.x_st + h0 * p.x_sh;
    const ET *zp = (const ET *)p.z + seq * p.z_sb + w.tok * p.z_st + h0 * p.z_sh;
    auto offsets = [&](int rows) {
        rB.offsets(p.B_st, 0, 1, rows, tid);
        rX.offsets(p.x_st, p.x_sh, heads, rows, tid);
        if constexpr (OUT) rC.offsets(p.C_st, 0, 1, rows, tc);
        if constexpr (GATED) rZ.offsets(p.z_st, p.z_sh, heads, rows, tid);
    };
    auto load_as = [&](int c, auto wide) {
        constexpr bool W = decltype(wide)::value;
        const int64_t t = (int64_t)c * L;
        rB.template load<W>(Bp + t * p.B_st, tid);
        rX.template load<W>(xp + t * p.x_st, tid);
        if constexpr (OUT) rC.template load<W>(Cp + t * p.C_st, tc);
        if constexpr (GATED) rZ.template load<W>(zp + t * p.z_st, tid);
    };
    auto load = [&](int c) {
        if (w.len - c * L < L) offsets(w.len - c * L);
        if (p.wide) load_as(c, std::true_type{});
        else load_as(c, std::false_type{});
    };

    // The decays of a group, in halves of waves 0 .. 3: half wave u forms chunk uc of the group for
    // head uh.  First steps and their sums (a barrier follows before the second part), then the
    // reference's walk over the group's chunks, the weights and the decays.
    struct Unit {
        int c, h, i;            // chunk of the group, head of the workgroup, token
    };
    auto unit = [&] {
        const int t = here(tid), u = t >> 5;
        return Unit{u / HPW, u % HPW, t & 31};
    };
    const bool forms = wave < 4;
    auto load_dt = [&](int k) {
        const Unit u = unit();
        const int t = min((k * GC + u.c) * L + u.i, w.len - 1);
        const int64_t at = seq * p.dt_sb + (w.tok + t) * p.dt_st + (h0 + min(u.h, heads - 1)) * p.dt_sh;
        return forms && k * GC < nck ? ld_any(p.dt, at, p.dt_bf16) : 0.f;
    };
    auto steps = [&](int k, float raw) {            // tokens past the end: step 0
        const Unit u = unit();
        const float step = (k * GC + u.c) * L + u.i < w.len ? step_of(raw + sBias[u.h], p.softplus) : 0.f;
        sStep[k & 1][u.c][u.h][u.i] = step;
        // decays in powers of two; sums in 64 bits, kept as two floats
        const double cs = prefix32((double)step * sA[u.h]);
        sSum[k & 1][u.c][u.h][u.i] = make_float2((float)cs, (float)(cs - (double)(float)cs));
    };
    auto sum_of = [&](float2 v) { return (double)v.x + (double)v.y; };
    auto weights = [&](int k) {
        const Unit u = unit();
        // c at the group's start: the state is 2^base times what S holds
        double base = k ? sBase[(k - 1) & 1][GC - 1][u.h] : 0.;
        double mine = 0., after = 0.;
        float scale = 1.f;
        bool direct = false;
        for (int c = 0; c < GC; ++c) {
            const double tot = sum_of(sSum[k & 1][c][u.h][L - 1]), old = base;
            const bool d = tot < -LIMIT, move = fabs(base + tot) > LIMIT && base != 0.;
            if (move) base = 0.;
            if (c == u.c) {
                mine = base;
                direct = d;
                scale = move ? exp2_of(old) : 1.f;
            }
            if (!d) base += tot;                    // (a direct chunk leaves S in its own units)
            if (c == u.c) after = base;
        }
        const double cs = sum_of(sSum[k & 1][u.c][u.h][u.i]);
        // e^{c_i}, and the weight: e^{-c_j} step_j, or e^{c_L - c_j} step_j
        const double ce = fmin(fmax(mine + cs, -4096.), 4096.), cr = __builtin_rint(ce);
        const float cf = (float)(ce - cr);
        const int ci = (int)cr;
        if constexpr (OUT) sEi[k & 1][u.c][u.h][u.i] = __builtin_ldexpf(__builtin_amdgcn_exp2f(cf), ci);
        float wt = __builtin_ldexpf(__builtin_amdgcn_exp2f(-cf), -ci);
        if (direct) wt = exp2_of(sum_of(sSum[k & 1][u.c][u.h][L - 1]) - cs);
        sWt[k & 1][u.c][u.h][u.i] = sStep[k & 1][u.c][u.h][u.i] * wt;
        if (u.i == 0) {
            sBase[k & 1][u.c][u.h] = after;
            sScale[k & 1][u.c][u.h] = scale;
            sDirect[k & 1][u.c][u.h] = direct;
        }
    };
    float dt_next = 0.f;
    if (nck > 0) {
        offsets(L);
        load(0);
        if constexpr (OUT) {
            if (tid < L * L / 8) *(f32x4 *)((char *)sM + tid * 8 * sizeof(ET)) = f32x4{0.f, 0.f, 0.f, 0.f};
            if (sizeof(ET) == 4 && tid < L * L / 8) *(f32x4 *)((char *)sM + tid * 32 + 16) = f32x4{0.f, 0.f, 0.f, 0.f};
            if (FINE && tid < L * L / 8) *(f32x4 *)((char *)sRest + tid * 16) = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        const float dt0 = load_dt(0);
        dt_next = load_dt(1);
        if (tid < HPW) {
            const int hu = h0 + min(tid, heads - 1);
            sA[tid] = (double)p.A[hu] * 1.4426950408889634;
            sBias[tid] = p.dt_bias ? p.dt_bias[hu] : 0.f;
        }
        __syncthreads();
        if (forms) steps(0, dt0);
        __syncthreads();
        if (forms) weights(0);
        __syncthreads();
    }
    double total = 0.;          // sum of a over the segment
    for (int c = 0; c < nck; ++c) {
        const int k = (c / GC) & 1, cg = c % GC, rows = min(L, w.len - c * L);
        ET *tB = sB[c & 1], *tC = sC[OUT ? c & 1 : 0], *tX = sX[c & 1], *tZ = sZ[GATED ? c & 1 : 0];
        rB.store(tB, tid);
        rX.store(tX, tid);
        if constexpr (OUT) rC.store(tC, tc);
        if constexpr (GATED) rZ.store(tZ, tid);
        const float scale = sScale[k][cg][wh];
        const bool direct = __builtin_amdgcn_readfirstlane(sDirect[k][cg][wh]);
        if constexpr (!OUT) total += sum_of(sSum[k][cg][wh][L - 1]);
        __syncthreads();
        if (c + 1 < nck) load(c + 1);
        if (forms && cg == 0) {
            steps(c / GC + 1, dt_next);
            dt_next = load_dt(c / GC + 2);
        }
        if (forms && cg == 1) weights(c / GC + 1);

        f32x4 Y[2] = {};
        if (__builtin_amdgcn_readfirstlane(__float_as_int(scale)) != __float_as_int(1.f)) scale_state(scale);
        if constexpr (OUT) {
            // the three 16 x 16 tiles of C B^T that hold j <= i, by three of the waves in turn
            const int job = (wave - 3 * c) & (NW - 1);
            if (job < 3) {
                const int jt = job >> 1, it = (job + 1) >> 1;
                f32x4 G = {};
#pragma unroll
                for (int a = 0; a < NA; ++a) {
                    Frag8<ET> fb, fc;
                    fb.load8(tB + rn.at(jt, a));
                    fc.load8(tC + rn.at(it, a));
                    mma16(G, fb, fc);               // row j = 4 g + r, column i = l16
                }
                float m4[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) m4[r] = (jt != it || 4 * g + r <= l16) ? G[r] : 0.f;
                Vec4<ET>::store(sM + m_at(16 * it + l16, 4 * jt + g), Vec4<ET>::pack(m4));
                if constexpr (FINE) {
                    float hi[4];
                    Vec4<ET>::unpack(Vec4<ET>::pack(m4), hi);
#pragma unroll
                    for (int r = 0; r < 4; ++r) m4[r] -= hi[r];
                    Vec4<ET>::store(sRest + m_at(16 * it + l16, 4 * jt + g), Vec4<ET>::pack(m4));
                }
            }
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                Frag8<ET> fs, fc;
                const float t8[8] = {S[2 * a][0], S[2 * a][1], S[2 * a][2], S[2 * a][3],
                                     S[2 * a + 1][0], S[2 * a + 1][1], S[2 * a + 1][2], S[2 * a + 1][3]};
                fs.set(t8);
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    fc.load8(tC + rn.at(it, a));
                    mma16(Y[it], fs, fc);           // (Z^T C^T)[p][i]
                }
                if constexpr (FINE) {
                    rest_of(t8, fs);
#pragma unroll
                    for (int it = 0; it < 2; ++it) {
                        fc.load8(tC + rn.at(it, a));
                        mma16(Y[it], fs, fc);
                    }
                }
            }
        }
        // weighted x^T (lane = column, elements = tokens 4 g .. + 3 and 16 + 4 g .. + 3)
        Frag8<ET> fx, fw[PARTS];
        cx.get(fx, tX, 0, 0);
        {
            const float4 wa = *(const float4 *)&sWt[k][cg][wh][4 * g], wb = *(const float4 *)&sWt[k][cg][wh][16 + 4 * g];
            const float w8[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
            if constexpr (BF) {
                float xw[8];
                const uint4 v = __builtin_bit_cast(uint4, fx.v);
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xw[2 * e] = __builtin_bit_cast(float, vw[e] << 16) * w8[2 * e];
                    xw[2 * e + 1] = __builtin_bit_cast(float, vw[e] & 0xffff0000u) * w8[2 * e + 1];
                }
                split3(xw, fw);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) fw[0].v[e] = fx.v[e] * w8[e];
            }
        }
        if (direct) scale_state(exp2_of(sum_of(sSum[k][cg][wh][L - 1])));
        // state update: neighbouring products belong to different tiles
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            Frag8<ET> fb[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) cn.get(fb[t], tB, a, t);
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                for (int t = 0; t < 2; ++t) mma16(S[2 * a + t], fb[t], fw[i]);
        }
        if constexpr (OUT) {
            __syncthreads();                        // sM
            float ei[2] = {sEi[k][cg][wh][l16], sEi[k][cg][wh][16 + l16]};
            if (!direct) {
                Frag8<ET> fm[2];
#pragma unroll
                for (int it = 0; it < 2; ++it) fm[it].load44(sM + m_at(16 * it + l16, g), sM + m_at(16 * it + l16, 4 + g));
#pragma unroll
                for (int i = 0; i < (BF ? 2 : 1); ++i)
#pragma unroll
                    for (int it = 0; it < 2; ++it) mma16(Y[it], fw[i], fm[it]);
                if constexpr (FINE) {
#pragma unroll
                    for (int it = 0; it < 2; ++it) {
                        fm[it].load44(sRest + m_at(16 * it + l16, g), sRest + m_at(16 * it + l16, 4 + g));
                        mma16(Y[it], fw[0], fm[it]);
                    }
                }
            } else {
                // every weight a difference of sums: step_j e^{c_i - c_j} on M, plain x.  (The
                // addresses are formed here: held through the loop they would cost its registers.)
                const int hl = here(lane), hi = hl & 15, hg = hl >> 4;
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const float2 ci = sSum[k][cg][wh][16 * it + hi];
                    float m8[8];
                    Frag8<ET> fd, fp;
                    fd.load44(sM + m_at(16 * it + hi, hg), sM + m_at(16 * it + hi, 4 + hg));
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (BF) {
                        const uint4 v = __builtin_bit_cast(uint4, fd.v);
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            m8[2 * e] = __builtin_bit_cast(float, vw[e] << 16);
                            m8[2 * e + 1] = __builtin_bit_cast(float, vw[e] & 0xffff0000u);
                        }
                        if constexpr (FINE) {
                            fd.load44(sRest + m_at(16 * it + hi, hg), sRest + m_at(16 * it + hi, 4 + hg));
                            const uint4 q = __builtin_bit_cast(uint4, fd.v);
                            const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                m8[2 * e] += __builtin_bit_cast(float, qw[e] << 16);
                                m8[2 * e + 1] += __builtin_bit_cast(float, qw[e] & 0xffff0000u);
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) m8[e] = fd.v[e];
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int j = 16 * (q >> 1) + 4 * hg + 2 * (q & 1);
                        const float2 sj = *(const float2 *)&sStep[k][cg][wh][j];
                        const float4 cj = *(const float4 *)&sSum[k][cg][wh][j];
                        m8[2 * q] *= sj.x * __builtin_amdgcn_exp2f(fminf((ci.x - cj.x) + (ci.y - cj.y), 0.f));
                        m8[2 * q + 1] *= sj.y * __builtin_amdgcn_exp2f(fminf((ci.x - cj.z) + (ci.y - cj.w), 0.f));
                        __builtin_amdgcn_sched_barrier(0);      // (few registers at a time)
                    }
                    fd.set(m8);
#pragma unroll
                    for (int r = 0; r < 4; ++r) Y[it][r] *= ei[it];
                    Cols<ET, XC, false>(hl, wh * P + slab * 16).get(fp, tX, 0, 0);
                    mma16(Y[it], fp, fd);
                    if constexpr (FINE) {
                        rest_of(m8, fd);
                        mma16(Y[it], fp, fd);
                    }
                    ei[it] = 1.f;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // lane = token, registers = columns 4 g .. + 3 of the slab
            ET *dst = (ET *)p.o + seq * p.o_sb + (w.tok + (int64_t)c * L) * p.o_st + h * p.o_sh + slab * 16 + 4 * g;
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                float x4[4], y4[4];
                Vec4<ET>::unpack(Vec4<ET>::load(tX + xrow + it * 16 * XC), x4);
#pragma unroll
                for (int r = 0; r < 4; ++r) y4[r] = __builtin_fmaf(Y[it][r], ei[it], skip * x4[r]);
                if constexpr (GATED) {
                    float z4[4];
                    Vec4<ET>::unpack(Vec4<ET>::load(tZ + xrow + it * 16 * XC), z4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y4[r] *= silu_act(z4[r]);
                }
                if (live && 16 * it + l16 < rows) Vec4<ET>::store(dst + (uint32_t)(16 * it + l16) * (uint32_t)p.o_st, Vec4<ET>::pack(y4));
            }
        }
    }
    if (nck > 0) {
        const double b = sBase[((nck - 1) / GC) & 1][(nck - 1) % GC][wh];
        if (b != 0.) scale_state(exp2_of(b));
    }
    if (!live) return;
    if constexpr (!OUT) {
#pragma unroll
        for (int m = 0; m < NM; ++m) *(f32x4 *)(ws + ws_index<P, N>(slab, m, lane)) = S[m];
        if (slab == 0 && lane == 0) p.ws_decay[(int64_t)slot * p.H + h] = exp2_of(total);
    } else if (w.last && p.sT) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t i = w.n * p.sT_sn + h * p.sT_sh + row_of(m, g, r) * p.sT_sr + slab * 16 + l16;
                if (p.sT_bf16) ((bf16 *)p.sT)[i] = (bf16)S[m][r];
                else ((float *)p.sT)[i] = S[m][r];
            }
    }
}

// Start states from end states: one thread per 4 state elements of a (sequence, head), walking
// the sequence's segments.  The workspace slot of a segment holds its end state (from zero) on
// entry and its start state on return; a last segment's holds nothing on entry.
template <int P, int N>
__global__ __launch_bounds__(256) void ssm_scan_kernel(const SsmParams p)
{
    constexpr int BPS = N * P / 1024;       // workgroups per state
    const int part = blockIdx.x % BPS;
    const int64_t chain = blockIdx.x / BPS;
    const int n = (int)(chain / p.H), h = (int)(chain % p.H);
    const int i4 = part * 256 + threadIdx.x, lane = i4 & 63;
    const int m = (i4 >> 6) % (N / 16), slab = i4 / (64 * (N / 16));
    const Cut cut = cut_of(p, n);
    const int count = cut.full;
    float s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        s[r] = p.s0 ? ld_any(p.s0, n * p.s0_sn + h * p.s0_sh + row_of(m, lane >> 4, r) * p.s0_sr + slab * 16 + (lane & 15),
                             p.s0_bf16)
                    : 0.f;
    float *ws = p.ws_state + ((int64_t)cut.first * p.H + h) * (N * P) + i4 * 4;
    const float *dec = p.ws_decay + (int64_t)cut.first * p.H + h;
    const int64_t step = (int64_t)p.H * (N * P);
    // the end states of AHEAD segments are requested before the first of them is needed: the walk
    // itself is four FMAs a segment
    constexpr int AHEAD = 16;
    for (int k = 0; k < count; k += AHEAD) {
        float4 e[AHEAD];
        float d[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t at = min(k + u, count - 1);
            e[u] = *(const float4 *)(ws + at * step);
            d[u] = dec[at * p.H];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (k + u >= count) break;
            *(float4 *)(ws + (k + u) * step) = make_float4(s[0], s[1], s[2], s[3]);
            s[0] = __builtin_fmaf(s[0], d[u], e[u].x);
            s[1] = __builtin_fmaf(s[1], d[u], e[u].y);
            s[2] = __builtin_fmaf(s[2], d[u], e[u].z);
            s[3] = __builtin_fmaf(s[3], d[u], e[u].w);
        }
    }
    *(float4 *)(p.ws_state + ((int64_t)cut.last * p.H + h) * (N * P) + i4 * 4) = make_float4(s[0], s[1], s[2], s[3]);
}

template <typename ET, int P, int N, int HPW>
static hipError_t launch_t(const SsmParams &p, bool states_only, hipStream_t st)
{
    const int64_t blocks = (int64_t)(states_only ? p.slots - p.N : p.slots) * p.wg_per_slot;
    if (blocks <= 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), thr(HPW * P * 4);
    constexpr bool BF = sizeof(ET) == 2;
    if (states_only) hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, false, false, false>), grid, thr, 0, st, p);
    else if (BF && p.fine && p.z) hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, true, true, BF>), grid, thr, 0, st, p);
    else if (BF && p.fine) hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, true, false, BF>), grid, thr, 0, st, p);
    else if (p.z) hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, true, true, false>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((ssm_kernel<ET, P, N, HPW, true, false, false>), grid, thr, 0, st, p);
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
