// Linear attention with one decay per head: the sweep over a sequence (prompt, and every
// gradient of the training pass) and the single-token update.
//
// Per batch row b and head h, with lambda = exp(log_decay[h]):
//     S_t = lambda S_{t-1} + k_t v_t^T,        y_t = scale * q_t^T S_t
// Over a chunk of m <= Q tokens that starts from the state H (i, j local to the chunk):
//     y_i = s_in sum_{j<=i} lambda^(i-j) (q_i . k_j) v_j + s_rd lambda^(i+1-sh) q_i^T H
//     H'  = lambda^m H + s_wr sum_j lambda^(m-1-j+sh) k_j v_j^T
// with s_in = s_rd = scale, s_wr = 1 and sh = 0.  The decay does not depend on the token, so
// every power of lambda a chunk needs comes from one table of Q + 1 values per workgroup.
//
// The gradients are the same sweep with other operands (dH = dLoss/dS after the last token):
//     dq = sweep(dy, v, k) from h0^T                        forward in time
//     dk = sweep(v, dy, q) from dH^T,  dv = sweep(k, q, dy) from dH    backward in time
// where a backward sweep reads the state before it decays (sh = 1; its end is dh0), and
// s_wr = scale, s_rd = 1, as dH is a gradient of the state itself.  The gradient of
// log_decay is sum_i dy_i . dy_i/da: with R = dS/da, R_t = lambda (R_{t-1} + S_{t-1}), the
// sweep of dq carries R beside S (AGE) and takes its product with q instead of y's with dy.
#include "ssm_device.h"

#include <type_traits>

namespace ssm {
namespace {

typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 512;   // 8 waves, two per SIMD
constexpr int kN = 64;          // value columns of one workgroup
constexpr int kYP = kN + 4;     // padded rows of the fp32 output shares

// Operands of a 16x16 product over K = 32, lane l: row (A) or column (B) l % 16, and eight
// k in two runs of four: 4 (l / 16) + e and 16 + 4 (l / 16) + e.  That is the order in
// which two 16x16 results (lane: rows 4 (l / 16) + j, column l % 16) stand side by side, so a
// result is the next product's operand without any exchange between lanes.
template <class T>
struct Op;

template <>
struct Op<uint16_t> {
    using V4 = s4;
    using Frag = s8;
    static constexpr int kPad = 8;    // LDS row padding (elements): rows 16 bytes apart modulo the banks
    static constexpr int kWide = 3;   // bf16 parts that carry an fp32 value whole
    static constexpr int kNarrow = 2; // and to about 16 bits
    static __device__ __forceinline__ Frag cat(V4 a, V4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
    static __device__ __forceinline__ f4 mma(Frag a, Frag b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ V4 ld4(const uint16_t *p) { return *reinterpret_cast<const s4 *>(p); }
    static __device__ __forceinline__ Frag ld8(const uint16_t *p) { return *reinterpret_cast<const s8 *>(p); }
    // column c0 + lr of rows r0 + 4 lg .. + 3, by the LDS transpose read: the sixteen lanes of
    // group lg address those four rows, four lanes of 8 bytes to a row
    static __device__ __forceinline__ V4 column4(const uint16_t *base, int row, int r0, int c0, int lr, int lg) {
        const uint16_t *p = base + (r0 + 4 * lg + (lr >> 2)) * row + c0 + 4 * (lr & 3);
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4 *)(const_cast<uint16_t *>(p)));
    }
    static __device__ __forceinline__ f4 widen4(V4 v) {
        const u2 r = __builtin_bit_cast(u2, v);
        return f4{bf_lo(r.x), bf_hi(r.x), bf_lo(r.y), bf_hi(r.y)};
    }
    // bits that are set where a piece of eight values holds an infinity or NaN (exponent all ones)
    static __device__ __forceinline__ uint32_t odd_bits(uint4 u) {
        auto two = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };
        return (two(u.x) | two(u.y) | two(u.z) | two(u.w)) & 0x80008000u;
    }
    // v with zeros in place of infinities and NaN
    static __device__ __forceinline__ V4 only_finite4(V4 v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (v[e] & 0x7f80) == 0x7f80 ? 0 : v[e];
        return v;
    }
    // v as a sum of N bf16 values, each the rounding of what the ones before it leave
    template <int N>
    static __device__ __forceinline__ void split(f4 v, V4 (&part)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const u2 r = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            part[n] = __builtin_bit_cast(s4, r);
            if (n + 1 < N) v = f4{v[0] - bf_lo(r.x), v[1] - bf_hi(r.x), v[2] - bf_lo(r.y), v[3] - bf_hi(r.y)};
        }
    }
};

template <>
struct Op<float> {
    using V4 = f4;
    struct Frag { f4 a, b; };
    static constexpr int kPad = 4;
    static constexpr int kWide = 1;
    static constexpr int kNarrow = 1;
    static __device__ __forceinline__ Frag cat(V4 a, V4 b) { return Frag{a, b}; }
    // K = 32 as eight products over K = 4 (v_mfma_f32_16x16x4_f32): product e takes element e of
    // every lane, the same k in both operands
    static __device__ __forceinline__ f4 mma(const Frag &a, const Frag &b, f4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[e], b.a[e], c, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[e], b.b[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ V4 ld4(const float *p) { return *reinterpret_cast<const f4 *>(p); }
    static __device__ __forceinline__ Frag ld8(const float *p) { return Frag{ld4(p), ld4(p + 4)}; }
    static __device__ __forceinline__ V4 column4(const float *base, int row, int r0, int c0, int lr, int lg) {
        const float *p = base + (r0 + 4 * lg) * row + c0 + lr;
        return f4{p[0], p[row], p[2 * row], p[3 * row]};
    }
    static __device__ __forceinline__ f4 widen4(V4 v) { return v; }
    static __device__ __forceinline__ bool finite1(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
    static __device__ __forceinline__ uint32_t odd_bits(uint4 u) {
        auto one = [](uint32_t x) { return (x & 0x7f800000u) + 0x00800000u; };
        return (one(u.x) | one(u.y) | one(u.z) | one(u.w)) & 0x80000000u;
    }
    static __device__ __forceinline__ V4 only_finite4(V4 v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = finite1(v[e]) ? v[e] : 0.0f;
        return v;
    }
    template <int N>
    static __device__ __forceinline__ void split(f4 v, V4 (&part)[N]) { part[0] = v; }
};

// lambda^n = hi + lo to more than 32 bits: near 1 the rounding of lambda^n alone would be
// the same at every chunk and add up over a long memory
struct Decay { float hi, lo; };
__device__ __forceinline__ Decay decay_of(float a, float n) {
    const float x = a * n;
    if (n == 0.0f) return Decay{1.0f, 0.0f};
    if (x > -0.5f && x < 0.5f) return Decay{1.0f, expm1f(x)};
    return Decay{expf(x), 0.0f};
}

template <class T, int DK>
struct Tile {
    // fp32 at 256 contraction columns: 32 rows to a chunk, so that q and k fit
    static constexpr int kQ = (sizeof(T) == 4 && DK == 256) ? 32 : 64;
    static constexpr int kBufs = (sizeof(T) == 2 && DK <= 128) ? 2 : 1;
    static constexpr int kRow = DK + Op<T>::kPad, kVRow = kN + Op<T>::kPad;
    static constexpr int kBlocks = kQ / 16;
    static constexpr int kTiles = kBlocks * (kBlocks + 1) / 2;   // 16x16 tiles on and below the diagonal
};

template <class T, int DK, bool AGE, bool STATE>
struct __align__(16) Smem {
    using G = Tile<T, DK>;
    using V4 = typename Op<T>::V4;
    T q[STATE ? 1 : G::kBufs][STATE ? 1 : G::kQ][G::kRow];
    T k[G::kBufs][G::kQ][G::kRow];
    T v[G::kBufs][G::kQ][G::kVRow];
    V4 p[Op<T>::kNarrow][STATE ? 1 : G::kTiles][64];                           // decayed (q k^T)^T, operand-ready
    V4 pa[AGE && !STATE ? Op<T>::kWide : 1][AGE && !STATE ? G::kTiles : 1][64];  // the same times i - j (AGE)
    float y[STATE ? 1 : 2][STATE ? 1 : G::kQ][kYP];                             // output shares of the two state halves
    // powers of the decay with the sweep's factors: in-chunk s_in lambda^d (0 for d < 0, offset 16),
    // readout s_rd lambda^(t + 1 - sh), update s_wr lambda^(m - 1 - j + sh) of a whole chunk and
    // of the segment's last one (0 past its m rows); AGE: the last two times m - 1 - j
    float w_in[16 + G::kQ], w_rd[G::kQ], w_up[2][G::kQ], w_age[AGE ? 2 : 1][AGE ? G::kQ : 4];
    uint32_t odd[2][8];                                         // waves that staged an infinity or NaN of v
};

__host__ __device__ constexpr int tile_of(int k, int i) { return i * (i + 1) / 2 + k; }

// One workgroup: the value columns [64 nt, 64 nt + 64) of one (b, h), one segment of the
// sequence.  Wave w owns value columns 16 (w % 4) .. + 15 and half w / 4 of the contraction
// columns: its part of the state stays in registers from chunk to chunk.  Per chunk: the
// tiles of q k^T (shared out over the waves) and each wave's share of the carried state's
// readout, a barrier, the in-chunk product (output blocks shared out between the halves),
// the state update and the next chunk's rows into LDS, a barrier, and the sum of the halves'
// shares to memory.  The rows after those are loaded into registers meanwhile.
//
// STATE: only the segment's own contribution to the state (from zero), into the workspace.
template <class T, int DK, bool AGE, bool STATE, bool VEC, int PF>
__global__ void __launch_bounds__(kThreads) linattn_kernel(LinAttnArgs a) {
    using G = Tile<T, DK>;
    using O = Op<T>;
    using V4 = typename O::V4;
    using Frag = typename O::Frag;
    constexpr int Q = G::kQ, KH = DK / 2, NT = KH / 16, NB = G::kBlocks, NJ = Q / 32;
    constexpr int NS = AGE ? O::kWide : O::kNarrow;   // parts of the state in its readout
    constexpr int VE = 16 / sizeof(T);
    constexpr int NQ = Q * DK / VE / kThreads, NV = Q * kN / VE / kThreads;
    static_assert(NQ >= 1 && NV >= 1, "a thread loads whole 16-byte pieces");
    __shared__ Smem<T, DK, AGE, STATE> sm;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nb = w & 3, hf = w >> 2, lr = lane & 15, lg = lane >> 4;

    // workgroup -> (b, h, segment, column tile): the hardware deals workgroups to the 8 XCDs
    // in turn; the column tiles of one segment read the same q and k and go to one XCD
    const int64_t per = (a.work + 7) / 8;
    int64_t id = static_cast<int64_t>(blockIdx.x) % 8 * per + blockIdx.x / 8;
    if (id >= a.work) return;
    const int nt = static_cast<int>(id % a.ntiles);
    id /= a.ntiles;
    const int64_t segs = STATE ? a.nseg - 1 : a.nseg;
    const int64_t seg = id % segs;
    id /= segs;
    const int64_t h = id % a.H, b = id / a.H;
    const int n0 = nt * kN;

    // (rows are counted in 32 bits, and in scalar registers: the planner's bound on seqlen)
    const int L = static_cast<int>(a.L), seg_len = static_cast<int>(a.seg_len);
    const int Lb = a.lengths ? __builtin_amdgcn_readfirstlane(min(max(a.lengths[b], 0), L)) : L;
    const int first = static_cast<int>(seg) * seg_len, end = min(first + seg_len, Lb);
    if (STATE && first + seg_len >= Lb) return;   // no later segment starts from this one's state
    const int sh = a.reverse ? 1 : 0;
    const float la = a.log_decay[h];

    // rows are counted in the sweep's direction: row t is token t, or token Lb - 1 - t
    const int64_t origin = a.reverse ? Lb - 1 : 0;
    const int64_t dir = a.reverse ? -1 : 1;
    const T *qg = static_cast<const T *>(a.q) + (b * a.L + origin) * a.q_row + (h / (a.H / a.q_heads)) * a.dk;
    const T *kg = static_cast<const T *>(a.k) + (b * a.L + origin) * a.k_row + (h / (a.H / a.k_heads)) * a.dk;
    const T *vg = static_cast<const T *>(a.v) + (b * a.L + origin) * a.v_row + (h / (a.H / a.v_heads)) * a.dn + n0;
    const int ncols = min(static_cast<int>(a.dn) - n0, kN);

    // rows past the sequence's end: zeros (a padded batch)
    if (!STATE && Lb < L) {
        const int from = max(first, Lb), to = min(first + seg_len, L);
        for (int64_t e = tid; e < static_cast<int64_t>(to - from) * ncols; e += kThreads) {
            const int64_t at = ((b * a.L + from + e / ncols) * a.H + h) * a.dn + n0 + e % ncols;
            if (a.out_f32) static_cast<float *>(a.y)[at] = 0.0f;
            else put(static_cast<T *>(a.y), at, 0.0f);
        }
    }
    if (!STATE && first >= Lb && !(Lb == 0 && seg == 0)) {
        if (AGE && tid == 0) a.age_part[((b * a.H + h) * a.nseg + seg) * a.ntiles + nt] = 0.0f;
        return;
    }

    const float s_in = a.s_in, s_rd = a.s_rd, s_wr = a.s_wr;
    const int tail = max(end - first, 0) % Q;   // rows of the last chunk, if it is not whole
    if (tid < 4 * Q) {
        auto power = [&](int n) { const Decay d = decay_of(la, static_cast<float>(n)); return d.hi + d.lo; };
        const int t = tid % Q, which = tid / Q;
        if (which == 0) {
            sm.w_in[16 + t] = s_in * power(t);
            if (t < 16) sm.w_in[t] = 0.0f;
        } else if (which == 1) {
            sm.w_rd[t] = s_rd * power(t + 1 - sh);
        } else {
            const int left = (which == 2 ? Q : tail) - 1 - t;
            const float x = left >= 0 ? s_wr * power(left + sh) : 0.0f;
            sm.w_up[which - 2][t] = x;
            if constexpr (AGE) sm.w_age[which - 2][t] = left >= 0 ? x * static_cast<float>(left) : 0.0f;
        }
    }

    // ---- the wave's part of the state: contraction row 16 t + 4 lg + j of its half, column lr
    f4 S[NT], R[AGE ? NT : 1];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int kk = hf * KH + 16 * t + 4 * lg + j, n = n0 + 16 * nb + lr;
            const bool in = kk < a.dk && n < a.dn;
            float s0 = 0.0f, r0 = 0.0f;
            if (!STATE && in) {
                if (seg > 0) {
                    const int64_t at = (((b * a.H + h) * (a.nseg - 1) + seg - 1) * a.dk + kk) * a.dn + n;
                    s0 = a.ws_S[at];
                    if constexpr (AGE) r0 = a.ws_R[at];
                } else if (a.h0) {
                    s0 = a.h0[(b * a.H + h) * a.dk * a.dn + kk * a.h_sr + n * a.h_sc];
                }
            }
            S[t][j] = s0;
            if constexpr (AGE) R[t][j] = r0;
        }
    }

    // ---- rows to registers (16 bytes each), registers to LDS (zeros outside the operand).
    // VEC: a chunk's loads are the same instructions whatever the chunk, with no branch around
    // them, so that waiting for one set leaves the later ones in flight.  The last chunk loads
    // the segment's last Q rows (rows before it among them) and sorts them on the way to LDS; a
    // sequence shorter than Q rows repeats its last row.  Addresses: a scalar base and a 32-bit
    // offset per lane; backward in time the base is the last row, the lowest address.
    uint4 rq[STATE ? 1 : PF][NQ], rk[PF][NQ], rv[PF][NV];
    const int dk = static_cast<int>(a.dk);
    const bool whole_cols = dk == DK && ncols == kN;
    const int top = min(Q, Lb) - 1, latest = max(end - Q, 0);   // last row of a load, last start of one
    uint32_t oq[NQ], ok[NQ], ov[NV];
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
        const int s = tid + r * kThreads, row = min(s / (DK / VE), top), c = s % (DK / VE) * VE;
        const uint32_t at = a.reverse ? top - row : row, col = c < dk ? c : 0;
        oq[r] = at * static_cast<uint32_t>(a.q_row) + col;
        ok[r] = at * static_cast<uint32_t>(a.k_row) + col;
    }
#pragma unroll
    for (int r = 0; r < NV; ++r) {
        const int s = tid + r * kThreads, row = min(s / (kN / VE), top), c = s % (kN / VE) * VE;
        ov[r] = (a.reverse ? top - row : row) * static_cast<uint32_t>(a.v_row) + (c < ncols ? c : 0);
    }
    auto piece = [&](const T *base, uint32_t off) __attribute__((always_inline)) {
        return *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + static_cast<uint64_t>(off) * sizeof(T));
    };
    // (single elements where rows or heads do not start on 16 bytes)
    auto piece_of_elements = [&](const T *g, int64_t stride, int t, int col, int cols) __attribute__((always_inline)) {
        const T *p = g + dir * t * stride + col;
        struct { T e[VE]; } x;
#pragma unroll
        for (int i = 0; i < VE; ++i) x.e[i] = t < end && col + i < cols ? p[i] : T(0);
        return __builtin_bit_cast(uint4, x);
    };
    auto load = [&](int t0, int set) __attribute__((always_inline)) {
        const int64_t at = a.reverse ? -static_cast<int64_t>(min(t0, latest) + top) : min(t0, latest);
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            const int s = tid + r * kThreads, row = s / (DK / VE), col = s % (DK / VE) * VE;
            if constexpr (!STATE) rq[set][r] = VEC ? piece(qg + at * a.q_row, oq[r]) : piece_of_elements(qg, a.q_row, t0 + row, col, dk);
            rk[set][r] = VEC ? piece(kg + at * a.k_row, ok[r]) : piece_of_elements(kg, a.k_row, t0 + row, col, dk);
        }
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int s = tid + r * kThreads, row = s / (kN / VE), col = s % (kN / VE) * VE;
            rv[set][r] = VEC ? piece(vg + at * a.v_row, ov[r]) : piece_of_elements(vg, a.v_row, t0 + row, col, ncols);
        }
        __builtin_amdgcn_sched_barrier(0);   // sets are waited for in the order of their loads
    };
    auto stage_rows = [&](int t0, int buf, int set, auto inside) __attribute__((always_inline)) {
        constexpr bool IN = decltype(inside)::value || !VEC;
        // m: the chunk's rows (none past the end: the turn of the last chunk stages zeros); shift: the
        // loaded rows that come before it, 0 .. Q, whose places the rows behind its end take
        const int m = max(end - t0, 0), shift = IN || Lb < Q ? 0 : Q - min(m, Q);
        auto place = [&](int row) { return IN ? row : row >= shift ? row - shift : row - shift + Q; };
        auto within = [&](uint4 u, int row, int col, int cols) __attribute__((always_inline)) {
            return IN || (row < m && col < cols) ? u : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            const int s = tid + r * kThreads, row = place(s / (DK / VE)), col = s % (DK / VE) * VE;
            if constexpr (!STATE) *reinterpret_cast<uint4 *>(&sm.q[buf][row][col]) = within(rq[set][r], row, col, dk);
            *reinterpret_cast<uint4 *>(&sm.k[buf][row][col]) = within(rk[set][r], row, col, dk);
        }
        uint32_t odd = 0;
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int s = tid + r * kThreads, row = place(s / (kN / VE)), col = s % (kN / VE) * VE;
            const uint4 u = within(rv[set][r], row, col, ncols);
            *reinterpret_cast<uint4 *>(&sm.v[buf][row][col]) = u;
            odd |= O::odd_bits(u);
        }
        if constexpr (!STATE) {
            const bool any = __ballot(odd != 0) != 0;
            if (lane == 0) sm.odd[buf][w] = any;
        }
    };
    auto stage = [&](int t0, int buf, int set) __attribute__((always_inline)) {
        if (t0 + Q <= end && whole_cols) stage_rows(t0, buf, set, std::true_type{});
        else stage_rows(t0, buf, set, std::false_type{});
    };

    const Decay full = decay_of(la, static_cast<float>(Q)), part = decay_of(la, static_cast<float>(tail));
    float age = 0.0f;
    if (first < end) {
#pragma unroll
    for (int p = 0; p < PF; ++p) load(first + p * Q, p);
    stage(first, 0, 0);
    load(first + PF * Q, 0);
    __syncthreads();
    // the chunk at row t0, staged in LDS; its successor's rows are in register set (set + 1) % PF
    auto chunk = [&](int t0, auto which, auto further) __attribute__((always_inline)) {
        constexpr int set = decltype(which)::value;
        constexpr bool MORE = decltype(further)::value;   // in the loop: rows are loaded ahead
        constexpr int kB = G::kBufs;
        static_assert(PF == 1 || PF == 2, "one or two sets");
        static_assert(kB == 1 || PF == 2, "a chunk's LDS buffer is known at compile time");
        const int buf = kB == 1 ? 0 : set & 1, nbuf = kB == 1 ? 0 : buf ^ 1;
        const int m = min(Q, end - t0);
        f4 acc[STATE ? 1 : NB], acca[AGE ? NB : 1];
        if constexpr (!STATE) {
            // ---- tiles of (q k^T)^T with their decay: lane s = 16 k + 4 lg + j, t = 16 i + lr
            for (int idx = w; idx < G::kTiles; idx += 8) {
                const int i = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, k = idx - i * (i + 1) / 2;
                f4 g = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < DK / 32; ++c)
                    g = O::mma(O::ld8(&sm.k[buf][16 * k + lr][32 * c + 8 * lg]), O::ld8(&sm.q[buf][16 * i + lr][32 * c + 8 * lg]), g);
                f4 x;
                const int d0 = 16 * (i - k) + lr - 4 * lg;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = g[j] * sm.w_in[16 + d0 - j];
                if (i == k)   // rows after the output's: zero whatever q and k hold
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = d0 - j >= 0 ? x[j] : 0.0f;
                V4 part[O::kNarrow];
                O::template split<O::kNarrow>(x, part);
#pragma unroll
                for (int n = 0; n < O::kNarrow; ++n) sm.p[n][idx][lane] = part[n];
                if constexpr (AGE) {
                    f4 xa;
#pragma unroll
                    for (int j = 0; j < 4; ++j) xa[j] = x[j] * static_cast<float>(max(d0 - j, 0));
                    V4 wide[O::kWide];
                    O::template split<O::kWide>(xa, wide);
#pragma unroll
                    for (int n = 0; n < O::kWide; ++n) sm.pa[n][idx][lane] = wide[n];
                }
            }
            // ---- this half's share of the carried state's readout, y^T: lane n = 4 lg + j, t = lr
            V4 sp[NT][NS], rp[AGE ? NT : 1][NS];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                O::template split<NS>(S[t], sp[t]);
                if constexpr (AGE) O::template split<NS>(R[t], rp[t]);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                f4 off = {0.0f, 0.0f, 0.0f, 0.0f}, offa = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < NT / 2; ++c) {
                    const T *qr = &sm.q[buf][16 * i + lr][hf * KH + 32 * c + 4 * lg];
                    const Frag qf = O::cat(O::ld4(qr), O::ld4(qr + 16));
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        off = O::mma(O::cat(sp[2 * c][n], sp[2 * c + 1][n]), qf, off);
                        if constexpr (AGE) offa = O::mma(O::cat(rp[2 * c][n], rp[2 * c + 1][n]), qf, offa);
                    }
                }
                const int t = 16 * i + lr;
                const float e = sm.w_rd[t];
                acc[i] = off * e;
                if constexpr (AGE) acca[i] = offa * e + off * (e * static_cast<float>(t + 1));
            }
            __syncthreads();   // tiles built
        }

        // ---- the value rows as an operand: column 16 nb + lr, rows in the operand order
        V4 vp[2 * NJ];
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j) vp[j] = O::column4(&sm.v[buf][0][0], G::kVRow, 16 * j, 16 * nb, lr, lg);
        if constexpr (!STATE) {
            const uint4 o0 = *reinterpret_cast<const uint4 *>(&sm.odd[buf][0]), o1 = *reinterpret_cast<const uint4 *>(&sm.odd[buf][4]);
            const bool odd = __builtin_amdgcn_readfirstlane(o0.x | o0.y | o0.z | o0.w | o1.x | o1.y | o1.z | o1.w) != 0;
            // ---- in-chunk product; half 0 takes output blocks 0 and 3, half 1 blocks 1 and 2
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const bool mine = NB == 2 ? i == hf : hf == 0 ? (i == 0 || i == 3) : (i == 1 || i == 2);
                if (mine) {
                    // the diagonal tile's zeros (rows after the output's) must not meet an infinity
                    // or NaN: such values are taken out of the product and added to their own and
                    // later rows only
                    V4 vd = vp[i];
                    if (odd) {
                        asm volatile("");   // (a branch, not selects: next to no chunk goes here)
                        vd = O::only_finite4(vd);
                    }
#pragma unroll
                    for (int k = 0; k <= i; k += 2) {
                        const bool two = k + 1 <= i;
                        const V4 zero = {};
                        const Frag vf = O::cat(k == i ? vd : vp[k], two ? (k + 1 == i ? vd : vp[k + 1]) : zero);
#pragma unroll
                        for (int n = 0; n < O::kNarrow; ++n)
                            acc[i] = O::mma(vf, O::cat(sm.p[n][tile_of(k, i)][lane], two ? sm.p[n][tile_of(k + 1, i)][lane] : zero), acc[i]);
                        if constexpr (AGE) {
#pragma unroll
                            for (int n = 0; n < O::kWide; ++n)
                                acca[i] = O::mma(vf, O::cat(sm.pa[n][tile_of(k, i)][lane], two ? sm.pa[n][tile_of(k + 1, i)][lane] : zero), acca[i]);
                        }
                    }
                    if (odd) {
                        for (int r = 0; r <= lr; ++r) {
                            const int from = (r >> 2) * 16 + lr;   // the lane that holds row r, column lr of the tile
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float x = widen_v(sm.v[buf][16 * i + r][16 * nb + 4 * lg + j]);
                                if ((__float_as_uint(x) & 0x7f800000u) != 0x7f800000u) continue;
                                float p = 0.0f;
                                for (int n = 0; n < O::kNarrow; ++n) p += O::widen4(sm.p[n][tile_of(i, i)][from])[r & 3];
                                acc[i][j] = __builtin_fmaf(p, x, acc[i][j]);
                                if constexpr (AGE) acca[i][j] = __builtin_fmaf(p * static_cast<float>(lr - r), x, acca[i][j]);
                            }
                        }
                    }
                }
                *reinterpret_cast<f4 *>(&sm.y[hf][16 * i + lr][16 * nb + 4 * lg]) = acc[i];
                if constexpr (AGE) {
                    const int t = 16 * i + lr;
                    if (t < m) {
                        const T *wr = static_cast<const T *>(a.age_w) + (b * a.L + t0 + t) * a.age_row + (h / (a.H / a.age_heads)) * a.dn + n0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int n = 16 * nb + 4 * lg + j;
                            if (n < ncols) age = __builtin_fmaf(acca[i][j], widen_v(wr[n]), age);
                        }
                    }
                }
            }
        }

        // ---- state update with the weighted value rows
        {
            const Decay d = m == Q ? full : part;
            V4 wp[2 * NJ][O::kWide], ap[AGE ? 2 * NJ : 1][O::kWide];
#pragma unroll
            for (int j = 0; j < 2 * NJ; ++j) {
                const f4 x = O::widen4(vp[j]);
                O::template split<O::kWide>(x * *reinterpret_cast<const f4 *>(&sm.w_up[m == Q ? 0 : 1][16 * j + 4 * lg]), wp[j]);
                if constexpr (AGE)
                    O::template split<O::kWide>(x * *reinterpret_cast<const f4 *>(&sm.w_age[m == Q ? 0 : 1][16 * j + 4 * lg]), ap[j]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f4 s = S[t];
                if constexpr (AGE) {
                    f4 r = R[t] + s * static_cast<float>(m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[j] = __builtin_fmaf(r[j], d.lo, r[j] * d.hi);
                    R[t] = r;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = __builtin_fmaf(s[j], d.lo, s[j] * d.hi);
#pragma unroll
                for (int c = 0; c < NJ; ++c) {
                    const Frag kf = O::cat(O::column4(&sm.k[buf][0][0], G::kRow, 32 * c, hf * KH + 16 * t, lr, lg),
                                           O::column4(&sm.k[buf][0][0], G::kRow, 32 * c + 16, hf * KH + 16 * t, lr, lg));
#pragma unroll
                    for (int n = 0; n < O::kWide; ++n) {
                        s = O::mma(kf, O::cat(wp[2 * c][n], wp[2 * c + 1][n]), s);
                        if constexpr (AGE) R[t] = O::mma(kf, O::cat(ap[2 * c][n], ap[2 * c + 1][n]), R[t]);
                    }
                }
                S[t] = s;
            }
        }
        // ---- the next chunk's rows into LDS, the ones after it into registers
        if constexpr (G::kBufs == 1) __syncthreads();   // this chunk's rows read
        stage(t0 + Q, nbuf, (set + 1) % PF);
        if constexpr (MORE) load(t0 + (PF + 1) * Q, (set + 1) % PF);
        __syncthreads();   // output shares written, the next chunk staged
        if constexpr (!STATE) {
            // ---- the halves' shares added, eight columns of one row per thread
            const int row = tid >> 3, col = (tid & 7) * 8;
            if (row < m) {
                float o[8];
                const f4 *p0 = reinterpret_cast<const f4 *>(&sm.y[0][row][col]), *p1 = reinterpret_cast<const f4 *>(&sm.y[1][row][col]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[4 * e + j] = p0[e][j] + p1[e][j];
                const int64_t at = ((b * a.L + origin + dir * (t0 + row)) * a.H + h) * a.dn + n0 + col;
                if (a.out_f32 || sizeof(T) == 4) {
                    float *y = static_cast<float *>(a.y) + at;
                    if (a.y_vec && col + 8 <= ncols) {
                        *reinterpret_cast<f4 *>(y) = f4{o[0], o[1], o[2], o[3]};
                        *reinterpret_cast<f4 *>(y + 4) = f4{o[4], o[5], o[6], o[7]};
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (col + j < ncols) y[j] = o[j];
                    }
                } else {
                    uint16_t *y = static_cast<uint16_t *>(a.y) + at;
                    if (a.y_vec && col + 8 <= ncols) {
                        *reinterpret_cast<uint4 *>(y) = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                                                   pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (col + j < ncols) y[j] = to_bf16(o[j]);
                    }
                }
            }
        }
    };
    // whole turns of PF chunks, then the rest (a way out in the middle of a turn would make the
    // compiler's waits at the top of the loop cover all loads)
    int t0 = first;
    for (; t0 + (PF - 1) * Q < end; t0 += PF * Q) {
        chunk(t0, std::integral_constant<int, 0>{}, std::true_type{});
        if constexpr (PF > 1) chunk(t0 + Q, std::integral_constant<int, 1 % PF>{}, std::true_type{});
    }
    if constexpr (PF > 1)
        if (t0 < end) chunk(t0, std::integral_constant<int, 0>{}, std::false_type{});
    }

    // ---- the state passed on
    const bool last = !STATE && end == Lb;
    float *out = STATE ? a.ws_S + ((b * a.H + h) * (a.nseg - 1) + seg) * a.dk * a.dn
                       : last && a.h_last ? a.h_last + (b * a.H + h) * a.dk * a.dn : nullptr;
    const int64_t sr = STATE ? a.dn : a.h_sr, sc = STATE ? 1 : a.h_sc;
    float *outR = STATE && AGE ? a.ws_R + ((b * a.H + h) * (a.nseg - 1) + seg) * a.dk * a.dn : nullptr;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int kk = hf * KH + 16 * t + 4 * lg + j, n = n0 + 16 * nb + lr;
            if (kk < a.dk && n < a.dn) {
                if (out) out[kk * sr + n * sc] = S[t][j];
                if constexpr (AGE) {
                    if (outR) outR[kk * sr + n * sc] = R[t][j];
                    // the last state's own gradient sees its age too
                    if (last && a.age_dh) age = __builtin_fmaf(R[t][j], a.age_dh[(b * a.H + h) * a.dk * a.dn + kk * a.h_sr + n * a.h_sc], age);
                }
            }
        }
    if constexpr (AGE && !STATE) {
        // the workgroup's share of dlog_decay, summed in a fixed order
        __syncthreads();
        float *red = &sm.y[0][0][0];
        red[tid] = age;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o) red[tid] += red[tid + o];
            __syncthreads();
        }
        if (tid == 0) a.age_part[((b * a.H + h) * a.nseg + seg) * a.ntiles + nt] = red[0];
    }
}

// Own contributions of the segments -> the states that segments 1, 2, ... start from, one
// thread per state element: H_{s+1} = lambda^T H_s + own_s (T rows to a segment), and with R
// its derivative by log_decay.
__global__ void __launch_bounds__(256) linattn_combine_kernel(LinAttnArgs a) {
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t sz = a.dk * a.dn;
    if (gid >= a.B * a.H * sz) return;
    const int64_t bh = gid / sz, e = gid % sz, kk = e / a.dn, n = e % a.dn;
    int64_t Lb = a.L;
    if (a.lengths) Lb = min(max(static_cast<int64_t>(a.lengths[bh / a.H]), int64_t(0)), a.L);
    const double x = static_cast<double>(a.log_decay[bh % a.H]) * static_cast<double>(a.seg_len);
    const float d = static_cast<float>(exp(x)), T = static_cast<float>(a.seg_len);
    float S = a.h0 ? a.h0[bh * sz + kk * a.h_sr + n * a.h_sc] : 0.0f, R = 0.0f;
    for (int64_t s = 0; s + 1 < a.nseg && (s + 1) * a.seg_len < Lb; ++s) {
        const int64_t at = (bh * (a.nseg - 1) + s) * sz + e;
        if (a.ws_R) {
            R = __builtin_fmaf(d, __builtin_fmaf(T, S, R), a.ws_R[at]);
            a.ws_R[at] = R;
        }
        S = __builtin_fmaf(d, S, a.ws_S[at]);
        a.ws_S[at] = S;
    }
}

// dlog_decay[h] = sum of the workgroups' shares over (b, segment, tile), in a fixed order
__global__ void __launch_bounds__(64) linattn_age_sum_kernel(const float *part, float *out, int64_t B, int64_t H, int64_t per) {
    const int64_t h = blockIdx.x;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < B * per; i += 64) s += part[((i / per) * H + h) * per + i % per];
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if (threadIdx.x == 0) out[h] = static_cast<float>(s);
}

// per-head gradients [rows][H][D] fp32 -> [rows][G][D], summed over the heads of a group in order
template <class T>
__global__ void __launch_bounds__(256) linattn_share_kernel(const float *part, T *out, int64_t n, int64_t G, int64_t D, int64_t per) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t d = i % D, g = i / D % G, row = i / (D * G);
    const float *p = part + (row * G + g) * per * D + d;
    float s = 0.0f;
    for (int64_t j = 0; j < per; ++j) s += p[j * D];
    put(out, i, s);
}

// One token: every state element is read and written once, so the launch is bound by the
// state's traffic.  A workgroup takes CW value columns of one (b, h); thread: four columns
// (16 bytes) of every (1024 / CW)-th contraction row.
template <class T, int CW>
__global__ void __launch_bounds__(256) linattn_update_kernel(LinAttnArgs a) {
    constexpr int C4 = CW / 4, RG = 256 / C4;
    __shared__ float red[4][CW];
    __shared__ float qs[256], ks[256];
    const int tid = threadIdx.x, c4 = tid % C4, rg = tid / C4;
    const int64_t tiles = (a.dn + CW - 1) / CW;
    const int64_t bh = blockIdx.x / tiles, h = bh % a.H, b = bh / a.H;
    const int n = static_cast<int>(blockIdx.x % tiles) * CW + 4 * c4, dk = static_cast<int>(a.dk), dn = static_cast<int>(a.dn);
    const T *q = static_cast<const T *>(a.q) + b * a.q_row + (h / (a.H / a.q_heads)) * dk;
    const T *k = static_cast<const T *>(a.k) + b * a.k_row + (h / (a.H / a.k_heads)) * dk;
    const T *v = static_cast<const T *>(a.v) + b * a.v_row + (h / (a.H / a.v_heads)) * dn;
    for (int i = tid; i < dk; i += 256) {
        qs[i] = a.s_rd * widen(q, i);
        ks[i] = widen(k, i);
    }
    f4 vv;
#pragma unroll
    for (int j = 0; j < 4; ++j) vv[j] = n + j < dn ? widen(v, n + j) : 0.0f;
    const Decay d = decay_of(a.log_decay[h], 1.0f);
    float *S = a.h_last + bh * dk * dn;
    f4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    if (a.y_vec && n < dn) {
#pragma unroll 8
        for (int kk = rg; kk < dk; kk += RG) {
            f4 *p = reinterpret_cast<f4 *>(S + static_cast<int64_t>(kk) * dn + n);
            f4 s = *p;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = __builtin_fmaf(s[j], d.hi, __builtin_fmaf(s[j], d.lo, ks[kk] * vv[j]));
                y[j] = __builtin_fmaf(qs[kk], s[j], y[j]);
            }
            *p = s;
        }
    } else {
        for (int kk = rg; kk < dk; kk += RG)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < dn) {
                    float *p = S + static_cast<int64_t>(kk) * dn + n + j;
                    const float s = __builtin_fmaf(*p, d.hi, __builtin_fmaf(*p, d.lo, ks[kk] * vv[j]));
                    y[j] = __builtin_fmaf(qs[kk], s, y[j]);
                    *p = s;
                }
    }
    // rows of the wave, then of the four waves, in a fixed order
#pragma unroll
    for (int o = C4; o < 64; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] += __shfl_xor(y[j], o, 64);
    if ((tid & 63) < C4)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[tid >> 6][4 * c4 + j] = y[j];
    __syncthreads();
    const int nn = static_cast<int>(blockIdx.x % tiles) * CW + tid;
    if (tid < CW && nn < dn) put(static_cast<T *>(a.y), bh * dn + nn, red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid]);
}

template <class T, int DK, bool AGE, bool STATE>
hipError_t launch_one(const LinAttnArgs &a0, hipStream_t s) {
    LinAttnArgs a = a0;
    a.work = a.B * a.H * (STATE ? a.nseg - 1 : a.nseg) * a.ntiles;
    static_assert(sizeof(Smem<T, DK, AGE, STATE>) <= kLdsPerCU, "LDS of one CU");
    // chunks whose rows are on their way in registers (as many as LDS buffers at least)
    constexpr int PF = Tile<T, DK>::kBufs == 2 || (STATE && sizeof(T) == 2) ? 2 : 1;
    const dim3 grid(static_cast<unsigned>((a.work + 7) / 8 * 8));
    if (a.vec) hipLaunchKernelGGL((linattn_kernel<T, DK, AGE, STATE, true, PF>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((linattn_kernel<T, DK, AGE, STATE, false, Tile<T, DK>::kBufs>), grid, dim3(kThreads), 0, s, a);
    return launch_status(s);
}

template <class T, int DK, bool AGE>
hipError_t launch_sweep(const LinAttnArgs &a, hipStream_t s) {
    if (a.nseg > 1) {
        hipError_t e = launch_one<T, DK, AGE, true>(a, s);
        if (e != hipSuccess) return e;
        const int64_t n = a.B * a.H * a.dk * a.dn;
        hipLaunchKernelGGL(linattn_combine_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, a);
        e = launch_status(s);
        if (e != hipSuccess) return e;
    }
    return launch_one<T, DK, AGE, false>(a, s);
}

template <class T>
hipError_t launch_typed(const LinAttnArgs &a, hipStream_t s) {
    const bool age = a.age_part != nullptr;
    if (a.dk <= 64) return age ? launch_sweep<T, 64, true>(a, s) : launch_sweep<T, 64, false>(a, s);
    if (a.dk <= 128) return age ? launch_sweep<T, 128, true>(a, s) : launch_sweep<T, 128, false>(a, s);
    return age ? launch_sweep<T, 256, true>(a, s) : launch_sweep<T, 256, false>(a, s);
}

}  // namespace

hipError_t launch_linattn(const LinAttnArgs &a0, bool bf16, hipStream_t s) {
    LinAttnArgs a = a0;
    const int64_t ve = bf16 ? 8 : 4;
    // 16-byte loads where every row and head starts on 16 bytes (the pointers do)
    a.vec = a.q_row % ve == 0 && a.k_row % ve == 0 && a.v_row % ve == 0 && a.dk % ve == 0 && a.dn % ve == 0;
    a.y_vec = a.dn % 8 == 0;
    return bf16 ? launch_typed<uint16_t>(a, s) : launch_typed<float>(a, s);
}

hipError_t launch_linattn_age_sum(const LinAttnArgs &a, float *dlog_decay, hipStream_t s) {
    hipLaunchKernelGGL(linattn_age_sum_kernel, dim3(static_cast<unsigned>(a.H)), dim3(64), 0, s, a.age_part, dlog_decay, a.B,
                       a.H, a.nseg * a.ntiles);
    return launch_status(s);
}

hipError_t launch_linattn_share(const float *part, void *out, int64_t rows, int64_t H, int64_t G, int64_t D, bool bf16, hipStream_t s) {
    const int64_t n = rows * G * D;
    const dim3 grid(static_cast<unsigned>((n + 255) / 256));
    if (bf16) hipLaunchKernelGGL((linattn_share_kernel<uint16_t>), grid, dim3(256), 0, s, part, static_cast<uint16_t *>(out), n, G, D, H / G);
    else hipLaunchKernelGGL((linattn_share_kernel<float>), grid, dim3(256), 0, s, part, static_cast<float *>(out), n, G, D, H / G);
    return launch_status(s);
}

hipError_t launch_linattn_update(const LinAttnArgs &a0, bool bf16, hipStream_t s) {
    LinAttnArgs a = a0;
    a.y_vec = a.dn % 4 == 0;
    // 16 columns to a workgroup while that leaves CUs without one at 64
    const bool narrow = a.B * a.H * ((a.dn + 63) / 64) < kCUs;
    const int64_t cw = narrow ? 16 : 64;
    const dim3 grid(static_cast<unsigned>(a.B * a.H * ((a.dn + cw - 1) / cw)));
    if (narrow) {
        if (bf16) hipLaunchKernelGGL((linattn_update_kernel<uint16_t, 16>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((linattn_update_kernel<float, 16>), grid, dim3(256), 0, s, a);
    } else {
        if (bf16) hipLaunchKernelGGL((linattn_update_kernel<uint16_t, 64>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((linattn_update_kernel<float, 64>), grid, dim3(256), 0, s, a);
    }
    return launch_status(s);
}

}  // namespace ssm
