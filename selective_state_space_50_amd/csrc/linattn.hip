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

// LDS by 32-bit address.  A lane's base address is kept in a register the compiler cannot see
// through, and everything else about an access is a constant in the instruction: left to itself
// it keeps a register for every constant, which the sweep has not got.
using Lds = uint32_t;
template <class V>
__device__ __forceinline__ V lds_get(Lds a) { return *(const __attribute__((address_space(3))) V *)(a); }
template <class V>
__device__ __forceinline__ void lds_put(Lds a, V v) { *(__attribute__((address_space(3))) V *)(a) = v; }
__device__ __forceinline__ Lds lds_of(const void *p) { return (Lds)(uintptr_t)((const __attribute__((address_space(3))) char *)p); }
__device__ __forceinline__ Lds opaque(Lds a) {
    asm("" : "+v"(a));
    return a;
}

// Operands of a 16x16 product over K = 32, lane l = 16 lg + lr: row (A) or column (B) lr, and
// eight k in two runs of four: 4 lg + e and 16 + 4 lg + e.  That is the order in which two
// 16x16 results (lane: rows 4 lg + j, column lr) stand side by side, so a result is the next
// product's operand without any exchange between lanes.
//
// LDS tiles are unpadded rows of a multiple of 128 bytes; the 16-byte piece c of a row is kept
// at place c ^ swizzle(row) (within its eight pieces), so that neither reads of one piece of
// 16 rows nor reads of two pieces of four rows (transposed) meet a bank more often than reads of
// 512 bytes in a row do.  (SQ_LDS_BANK_CONFLICT counts two cycles for each of the three.  The bf16 writes pay
// for it, in two halves of 8 bytes: eight cycles for a row's 16 bytes a lane, and four for a tile of q k^T, where
// writes in a row count none.)
template <class T>
struct Op;

template <>
struct Op<uint16_t> {
    using V4 = s4;
    using Frag = s8;
    // bf16 parts that carry an fp32 factor (states, decayed scores, weighted rows) whole.  (Two, 16 bits, in the
    // scores and the state's readout take B4 L4096 H64 128x64 from 228 to 209 us, B1 L32768 H16 128x128 from 273 to
    // 257, and leave 0.25% of bf16 outputs one step off those of 32-bit factors, against 0.04%.)
    static constexpr int kParts = 3;
    static constexpr int kRowOffs = 4, kColOffs = 4;
    static __device__ __forceinline__ Frag cat(V4 a, V4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
    static __device__ __forceinline__ f4 mma(Frag a, Frag b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    }
    // four rows' places four pieces apart, the next four rows' between them; rows 8 to 15 of
    // sixteen with their two 8-byte halves of a piece exchanged (reads of 8 bytes take all 16)
    static __device__ __forceinline__ int swizzle(int row) { return (row & 3) << 1 | (row >> 2 & 1); }
    // place of a piece: of its first and second half
    static __device__ __forceinline__ void place16(int row_bytes, int row, int piece, Lds (&at)[2]) {
        const Lds p = row * row_bytes + ((piece ^ swizzle(row)) << 4);
        at[0] = p + (row & 8);
        at[1] = p + (8 - (row & 8));
    }
    static __device__ __forceinline__ void put16(const Lds (&at)[2], Lds more, uint4 u) {
        lds_put(at[0] + more, u2{u.x, u.y});
        lds_put(at[1] + more, u2{u.z, u.w});
    }
    // byte offsets of a lane's operand runs in rows lr (run e of K block c: element c / 2 at [2 (c % 2) + e])
    static __device__ __forceinline__ int row_off(int i, int lr, int lg, int row_bytes) {
        return lr * row_bytes + (((2 * i + (lg >> 1)) ^ swizzle(lr)) << 4) + (((lg & 1) ^ (lr >> 3)) << 3);
    }
    static __device__ __forceinline__ Frag row(Lds block, const Lds (&off)[4], int c) {
        const Lds p = block + (c >> 1) * 128;
        return cat(lds_get<s4>(off[2 * (c & 1)] + p), lds_get<s4>(off[2 * (c & 1) + 1] + p));
    }
    // columns 16 t + lr of rows 4 lg .. + 3 by the LDS transpose read: the sixteen lanes of group lg
    // address those four rows, four lanes of 8 bytes to a row
    static __device__ __forceinline__ int col_off(int i, int lr, int lg, int row_bytes) {
        const int row = 4 * lg + (lr >> 2);
        return row * row_bytes + (((2 * i + (lr >> 1 & 1)) ^ swizzle(row)) << 4) + (((lr & 1) ^ (lg >> 1)) << 3);
    }
    static __device__ __forceinline__ V4 col(Lds block, const Lds (&off)[4], int t) {
        return col1(off[t & 3] + block + (t >> 2) * 128);
    }
    static __device__ __forceinline__ V4 col1(Lds p) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)(p));
    }
    // one column block of narrow rows (v): its offset is the lane's own
    static constexpr int kOneCol = 1;
    static __device__ __forceinline__ int one_off(int, int t, int lr, int lg, int row_bytes) { return col_off(t, lr, lg, row_bytes); }
    static __device__ __forceinline__ V4 one(Lds block, const Lds (&off)[1]) { return col1(off[0] + block); }
    static __device__ __forceinline__ Frag pair(Lds a) { return lds_get<s8>(a); }
    static __device__ __forceinline__ f4 widen4(V4 v) {
        const u2 r = __builtin_bit_cast(u2, v);
        return f4{bf_lo(r.x), bf_hi(r.x), bf_lo(r.y), bf_hi(r.y)};
    }
    static __device__ __forceinline__ float element(V4 v, int j) { return widen_v(static_cast<uint16_t>(v[j])); }
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
    static constexpr int kParts = 1;
    static constexpr int kRowOffs = 2, kColOffs = 8;
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
    static __device__ __forceinline__ int swizzle(int row) { return row & 7; }
    static __device__ __forceinline__ void place16(int row_bytes, int row, int piece, Lds (&at)[2]) {
        at[0] = row * row_bytes + ((piece ^ swizzle(row)) << 4);
        at[1] = 0;
    }
    static __device__ __forceinline__ void put16(const Lds (&at)[2], Lds more, uint4 u) {
        lds_put(at[0] + more, __builtin_bit_cast(f4, u));
    }
    static __device__ __forceinline__ int row_off(int i, int lr, int lg, int row_bytes) {
        return lr * row_bytes + (((4 * i + lg) ^ swizzle(lr)) << 4);
    }
    static __device__ __forceinline__ Frag row(Lds block, const Lds (&off)[2], int c) {
        return Frag{lds_get<f4>(off[0] + block + c * 128), lds_get<f4>(off[1] + block + c * 128)};
    }
    // (four loads, one per row)
    static __device__ __forceinline__ int col_off(int i, int lr, int lg, int row_bytes) {
        const int row = 4 * lg + (i & 3);
        return row * row_bytes + (((4 * (i >> 2) + (lr >> 2)) ^ swizzle(row)) << 4) + ((lr & 3) << 2);
    }
    static __device__ __forceinline__ V4 col(Lds block, const Lds (&off)[8], int t) {
        f4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = lds_get<float>(off[4 * (t & 1) + j] + block + (t >> 1) * 128);
        return v;
    }
    static constexpr int kOneCol = 4;
    static __device__ __forceinline__ int one_off(int j, int t, int lr, int lg, int row_bytes) {
        return col_off(4 * (t & 1) + j, lr, lg, row_bytes) + (t >> 1) * 128;
    }
    static __device__ __forceinline__ V4 one(Lds block, const Lds (&off)[4]) {
        f4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = lds_get<float>(off[j] + block);
        return v;
    }
    static __device__ __forceinline__ Frag pair(Lds a) { return Frag{lds_get<f4>(a), lds_get<f4>(a + 16)}; }
    static __device__ __forceinline__ f4 widen4(V4 v) { return v; }
    static __device__ __forceinline__ float element(V4 v, int j) { return v[j]; }
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
    static constexpr int kRow = DK * sizeof(T), kVRow = kN * sizeof(T);   // bytes
    static constexpr int kBlocks = kQ / 16;
    // tiles of q k^T on and below the diagonal, two of a row side by side (an operand over K = 32; the
    // second of the last pair of an even row is zero)
    static constexpr int kPairs = kBlocks == 4 ? 6 : 2;
    // operands are read one step ahead of their products where the registers allow it
    static constexpr bool kAhead = sizeof(T) == 2 ? DK <= 128 : DK <= 64;
};

// pair of row block i that holds column block k
__host__ __device__ constexpr int pair_of(int k, int i) { return (i < 2 ? i : 2 * i - 2) + k / 2; }

// What one workgroup works on: value columns n0 .. n0 + ncols of one (b, h), rows [first, end) of
// the sequence.  Rows are counted in the sweep's direction (row t is token t, or token Lb - 1 - t),
// in 32 bits (the planner's bound on seqlen) and scalar registers.
template <class T>
struct Part {
    int64_t b, h, seg;
    int nt, n0, ncols, Lb, first, end, seg_len;
    int64_t origin, dir;
    const T *q, *k, *v;   // row 0

    // workgroup -> (b, h, segment, column tile): the hardware deals workgroups to the 8 XCDs in
    // turn; the column tiles of one segment read the same q and k and go to one XCD
    __device__ __forceinline__ bool set(const LinAttnArgs &a, int64_t segs) {
        const int64_t per = (a.work + 7) / 8;
        int64_t id = static_cast<int64_t>(blockIdx.x) % 8 * per + blockIdx.x / 8;
        if (id >= a.work) return false;
        nt = static_cast<int>(id % a.ntiles);
        id /= a.ntiles;
        seg = id % segs;
        id /= segs;
        h = id % a.H;
        b = id / a.H;
        n0 = nt * kN;
        ncols = min(static_cast<int>(a.dn) - n0, kN);
        const int L = static_cast<int>(a.L);
        Lb = a.lengths ? __builtin_amdgcn_readfirstlane(min(max(a.lengths[b], 0), L)) : L;
        seg_len = static_cast<int>(a.seg_len);
        origin = a.reverse ? Lb - 1 : 0;
        dir = a.reverse ? -1 : 1;
        q = static_cast<const T *>(a.q) + (b * a.L + origin) * a.q_row + (h / (a.H / a.q_heads)) * a.dk;
        k = static_cast<const T *>(a.k) + (b * a.L + origin) * a.k_row + (h / (a.H / a.k_heads)) * a.dk;
        v = static_cast<const T *>(a.v) + (b * a.L + origin) * a.v_row + (h / (a.H / a.v_heads)) * a.dn + n0;
        return true;
    }
};

// Rows to registers (16 bytes each), registers to LDS (zeros outside the operand), by THREADS
// threads.  VEC: a chunk's loads are the same instructions whatever the chunk, with no branch
// around them, so that waiting for one set leaves the later ones in flight.  The last chunk loads
// the segment's last Q rows (rows before it among them) and sorts them on the way to LDS; a
// sequence shorter than Q rows repeats its last row.  Addresses: a scalar base and a 32-bit
// offset per lane; backward in time the base is the last row, the lowest address.
template <class T, int DK, int THREADS, bool WITH_Q, bool VEC>
struct Rows {
    using G = Tile<T, DK>;
    static constexpr int Q = G::kQ, VE = 16 / sizeof(T), PER = DK / VE, VPER = kN / VE;   // pieces of a row
    static constexpr int NQ = Q * PER / THREADS, NV = Q * VPER / THREADS;
    static_assert(NQ >= 1 && NV >= 1, "a thread loads whole 16-byte pieces");
    struct Set { uint4 q[WITH_Q ? NQ : 1], k[NQ], v[NV]; };
    const Lds k_base, v_base;
    const LinAttnArgs &a;
    const Part<T> &p;
    const int tid, dk, top, latest;   // top, latest: last row of a load, last start of one
    const bool whole_cols;
    uint32_t oq[NQ], ok[NQ], ov[NV];
    // LDS: a thread's pieces stand RS (VRS) rows apart, which a swizzle does not see
    static constexpr int RS = THREADS / PER, VRS = THREADS / VPER;
    static_assert(RS % 8 == 0 && VRS % 8 == 0 && (sizeof(T) == 4 || RS % 16 == 0), "pieces in rows of one swizzle");
    Lds at[2], vat[2];           // its first pieces of k and v in buffer 0
    const Lds q_from_k, kb, vb;  // bytes from k's to q's place, from buffer 0 to buffer 1

    __device__ __forceinline__ Rows(const LinAttnArgs &a_, const Part<T> &p_, int tid_, Lds q0, Lds k0, Lds v0, Lds kb_, Lds vb_)
        : k_base(k0), v_base(v0), a(a_), p(p_), tid(tid_), dk(static_cast<int>(a_.dk)), top(min(Q, p_.Lb) - 1), latest(max(p_.end - Q, 0)),
          whole_cols(a_.dk == DK && p_.ncols == kN), q_from_k(q0 - k0), kb(kb_), vb(vb_) {
        Op<T>::place16(G::kRow, tid / PER, tid % PER, at);
        Op<T>::place16(G::kVRow, tid / VPER, tid % VPER, vat);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at[i] = opaque(at[i] + k0);
            vat[i] = opaque(vat[i] + v0);
        }
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            const int s = tid + r * THREADS, row = min(s / PER, top), c = s % PER * VE;
            const uint32_t at = a.reverse ? top - row : row, col = c < dk ? c : 0;
            oq[r] = at * static_cast<uint32_t>(a.q_row) + col;
            ok[r] = at * static_cast<uint32_t>(a.k_row) + col;
        }
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int s = tid + r * THREADS, row = min(s / VPER, top), c = s % VPER * VE;
            ov[r] = (a.reverse ? top - row : row) * static_cast<uint32_t>(a.v_row) + (c < p.ncols ? c : 0);
        }
    }
    static __device__ __forceinline__ uint4 piece(const T *base, uint32_t off) {
        return *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + static_cast<uint64_t>(off) * sizeof(T));
    }
    // (single elements where rows or heads do not start on 16 bytes)
    __device__ __forceinline__ uint4 elements(const T *g, int64_t stride, int t, int col, int cols) const {
        const T *at = g + p.dir * t * stride + col;
        struct { T e[VE]; } x;
#pragma unroll
        for (int i = 0; i < VE; ++i) x.e[i] = t < p.end && col + i < cols ? at[i] : T(0);
        return __builtin_bit_cast(uint4, x);
    }
    __device__ __forceinline__ void load(int t0, Set &set) const {
        const int64_t at = a.reverse ? -static_cast<int64_t>(min(t0, latest) + top) : min(t0, latest);
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            const int s = tid + r * THREADS, row = s / PER, col = s % PER * VE;
            if constexpr (WITH_Q) set.q[r] = VEC ? piece(p.q + at * a.q_row, oq[r]) : elements(p.q, a.q_row, t0 + row, col, dk);
            set.k[r] = VEC ? piece(p.k + at * a.k_row, ok[r]) : elements(p.k, a.k_row, t0 + row, col, dk);
        }
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int s = tid + r * THREADS, row = s / VPER, col = s % VPER * VE;
            set.v[r] = VEC ? piece(p.v + at * a.v_row, ov[r]) : elements(p.v, a.v_row, t0 + row, col, p.ncols);
        }
        __builtin_amdgcn_sched_barrier(0);   // sets are waited for in the order of their loads
    }
    // the chunk at row t0 to LDS buffer buf; whether this thread staged an infinity or NaN of v
    template <bool INSIDE>
    __device__ __forceinline__ bool stage_rows(int t0, const Set &set, int buf) const {
        constexpr bool IN = INSIDE || !VEC;
        // m: the chunk's rows (none past the end: the turn of the last chunk stages zeros); shift: the
        // loaded rows that come before it, 0 .. Q, whose places the rows behind its end take
        const int m = max(p.end - t0, 0), shift = IN || p.Lb < Q ? 0 : Q - min(m, Q);
        auto place = [&](int row) __attribute__((always_inline)) { return row >= shift ? row - shift : row - shift + Q; };
        auto within = [&](uint4 u, int row, int col, int cols) __attribute__((always_inline)) {
            return row < m && col < cols ? u : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            if constexpr (IN) {
                if constexpr (WITH_Q) Op<T>::put16(at, r * RS * G::kRow + buf * kb + q_from_k, set.q[r]);
                Op<T>::put16(at, r * RS * G::kRow + buf * kb, set.k[r]);
            } else {
                const int row = place(tid / PER + r * RS), c = tid % PER;
                Lds x[2];
                Op<T>::place16(G::kRow, row, c, x);
                if constexpr (WITH_Q) Op<T>::put16(x, k_base + buf * kb + q_from_k, within(set.q[r], row, c * VE, dk));
                Op<T>::put16(x, k_base + buf * kb, within(set.k[r], row, c * VE, dk));
            }
        }
        uint32_t odd = 0;
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            uint4 u = set.v[r];
            if constexpr (IN) Op<T>::put16(vat, r * VRS * G::kVRow + buf * vb, u);
            else {
                const int row = place(tid / VPER + r * VRS), c = tid % VPER;
                Lds x[2];
                Op<T>::place16(G::kVRow, row, c, x);
                u = within(u, row, c * VE, p.ncols);
                Op<T>::put16(x, v_base + buf * vb, u);
            }
            odd |= Op<T>::odd_bits(u);
        }
        return odd != 0;
    }
    __device__ __forceinline__ bool stage(int t0, const Set &set, int buf) const {
        return t0 + Q <= p.end && whole_cols ? stage_rows<true>(t0, set, buf) : stage_rows<false>(t0, set, buf);
    }
};

// One chunk's rows take the state of a wave on: S <- lambda^m S + s_wr sum_j lambda^(m-1-j+sh) k_j v_j^T,
// for contraction rows 16 (TB + t) + 4 lg + j (t < NT) and column lr of its block; AGE: R = dS/da likewise,
// R <- lambda^m (R + m S) + s_wr sum_j (m-1-j) lambda^(m-1-j) k_j v_j^T.  The row weights go into v, split into
// as many bf16 parts as carry them whole: a state's error must not grow with the sequence.
template <class T, int Q, int ROW, int NT, bool AGE, bool AHEAD, int NR>
__device__ __forceinline__ void update_state(f4 (&S)[NT], f4 (&R)[NR], int TB, Lds k, const Lds (&koff)[Op<T>::kColOffs],
                                             const typename Op<T>::V4 (&vp)[Q / 16], Lds w_up, Lds w_age,
                                             Decay d, int m) {
    using O = Op<T>;
    constexpr int NJ = Q / 32;
    typename O::V4 wp[2 * NJ][O::kParts], ap[AGE ? 2 * NJ : 1][O::kParts];
#pragma unroll
    for (int j = 0; j < 2 * NJ; ++j) {
        const f4 x = O::widen4(vp[j]);
        O::template split<O::kParts>(x * lds_get<f4>(w_up + 64 * j), wp[j]);
        if constexpr (AGE) O::template split<O::kParts>(x * lds_get<f4>(w_age + 64 * j), ap[j]);
    }
    // AHEAD: two tiles at a time (their products are chains of accumulations), the next two tiles'
    // columns of k read meanwhile
    constexpr int STEP = AHEAD && NT > 1 ? 2 : 1;
    typename O::Frag kf[AHEAD ? 2 : 1][STEP][NJ];
    auto read = [&](int t, typename O::Frag (&f)[STEP][NJ]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < STEP; ++u)
#pragma unroll
            for (int c = 0; c < NJ; ++c)
                f[u][c] = O::cat(O::col(k + 32 * c * ROW, koff, TB + t + u), O::col(k + (32 * c + 16) * ROW, koff, TB + t + u));
    };
    if constexpr (AHEAD) read(0, kf[0]);
#pragma unroll
    for (int t = 0; t < NT; t += STEP) {
        const int at = AHEAD ? t / STEP & 1 : 0;
        if constexpr (!AHEAD) read(t, kf[0]);
        else if (t + STEP < NT) read(t + STEP, kf[at ^ 1]);
#pragma unroll
        for (int u = 0; u < STEP; ++u) {
            if constexpr (AGE) {
                f4 r = R[t + u] + S[t + u] * static_cast<float>(m);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = __builtin_fmaf(r[j], d.lo, r[j] * d.hi);
                R[t + u] = r;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) S[t + u][j] = __builtin_fmaf(S[t + u][j], d.lo, S[t + u][j] * d.hi);
        }
#pragma unroll
        for (int c = 0; c < NJ; ++c)
#pragma unroll
            for (int n = 0; n < O::kParts; ++n)
#pragma unroll
                for (int u = 0; u < STEP; ++u) {
                    S[t + u] = O::mma(kf[at][u][c], O::cat(wp[2 * c][n], wp[2 * c + 1][n]), S[t + u]);
                    if constexpr (AGE) R[t + u] = O::mma(kf[at][u][c], O::cat(ap[2 * c][n], ap[2 * c + 1][n]), R[t + u]);
                }
        __builtin_amdgcn_sched_barrier(0);   // (no further ahead: the registers are full)
    }
}

// row weights of the update, of a whole chunk and of the segment's last one (0 past its rows)
template <int Q, bool AGE>
__device__ __forceinline__ void fill_update_weights(float (&up)[2][Q], float *age, int i, float la, float s_wr, int sh, int tail) {
    const int t = i % Q, which = i / Q, left = (which == 0 ? Q : tail) - 1 - t;
    const Decay d = decay_of(la, static_cast<float>(max(left, 0) + sh));
    const float x = left >= 0 ? s_wr * (d.hi + d.lo) : 0.0f;
    up[which][t] = x;
    if constexpr (AGE) age[which * Q + t] = left > 0 ? x * static_cast<float>(left) : 0.0f;
}

// ---- the sweep.  One workgroup: 64 value columns of one (b, h), one segment of the sequence,
// chunk by chunk, in two roles of four waves, one of each on every SIMD:
//  * state waves hold the state in registers (wave w: value columns 16 w .. + 15, all contraction
//    columns).  They write the carried state's share of the chunk's output to LDS, pass the
//    barrier and take the state on;
//  * chunk waves build the chunk's tiles of q k^T, pass the barrier, take them times v, add the
//    state waves' share and store the output.
// All waves bring the next chunk to LDS, whose rows they loaded into registers one or two chunks
// ahead.  Two barriers a chunk.  A state's rows are never read twice and nothing is computed twice: with
// all eight waves in one role (half a state each) the weights of v and the sum of two output
// shares cost a third more VALU instructions and LDS traffic.
//
// Measured: B4 L4096 H64 128x64 bf16 (one segment, 256 workgroups) 209 us, 3.9 TB/s (228 us on another
// machine); a copy reaches 5.2.  Chunks of 64 take 3.2 us (128 columns): per SIMD 1.3 us of VALU and 0.8 us of
// matrix instructions, in two roles that meet at two barriers; without any product the same loads and stores take 168 us.
// Smaller chunks would cost more state updates, larger ones more in-chunk products and LDS (121 KB now).
// AGE doubles the readout and the update (dq of B2 L4096 H32 128x128: 189 us against 108 for dk or dv).
template <class T, int DK, bool AGE>
struct __align__(16) Smem {
    using G = Tile<T, DK>;
    using V4 = typename Op<T>::V4;
    char q[G::kBufs][G::kQ * G::kRow];
    char k[G::kBufs][G::kQ * G::kRow];
    char v[G::kBufs][G::kQ * G::kVRow];
    V4 p[Op<T>::kParts][G::kPairs][64][2];                          // decayed (q k^T)^T, operand-ready
    V4 pa[AGE ? Op<T>::kParts : 1][AGE ? G::kPairs : 1][64][2];       // the same times i - j (AGE)
    f4 y[4][G::kBlocks][64];                                    // the carried state's share of y^T
    f4 ya[AGE ? 4 : 1][AGE ? G::kBlocks : 1][64];               // and of its derivative
    float w_up[2][G::kQ], w_age[AGE ? 2 * G::kQ : 4];           // row weights of the update (AGE: and its derivative)
    uint32_t odd[2][8];                                         // waves that staged an infinity or NaN of v
    float red[kThreads];
};

template <class T, int DK, bool AGE, bool VEC>
__global__ void __launch_bounds__(kThreads) linattn_kernel(LinAttnArgs a) {
    using G = Tile<T, DK>;
    using O = Op<T>;
    using V4 = typename O::V4;
    using Frag = typename O::Frag;
    constexpr int Q = G::kQ, NT = DK / 16, NC = DK / 32, NB = G::kBlocks, kB = G::kBufs;
    constexpr int NS = O::kParts;
    __shared__ Smem<T, DK, AGE> sm;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), w = wv & 3;
    const int lr = lane & 15, lg = lane >> 4;
    Part<T> p;
    if (!p.set(a, a.nseg)) return;
    const int first = p.first = static_cast<int>(p.seg) * p.seg_len, end = p.end = min(first + p.seg_len, p.Lb);

    // rows past the sequence's end: zeros (a padded batch)
    if (p.Lb < static_cast<int>(a.L)) {
        const int from = max(first, p.Lb), to = min(first + p.seg_len, static_cast<int>(a.L));
        for (int64_t e = tid; e < static_cast<int64_t>(to - from) * p.ncols; e += kThreads) {
            const int64_t at = ((p.b * a.L + from + e / p.ncols) * a.H + p.h) * a.dn + p.n0 + e % p.ncols;
            if (a.out_f32) static_cast<float *>(a.y)[at] = 0.0f;
            else put(static_cast<T *>(a.y), at, 0.0f);
        }
    }
    const int64_t share = ((p.b * a.H + p.h) * a.nseg + p.seg) * a.ntiles + p.nt;
    if (first >= p.Lb && !(p.Lb == 0 && p.seg == 0)) {
        if (AGE && tid == 0) a.age_part[share] = 0.0f;
        return;
    }

    const int sh = a.reverse ? 1 : 0, tail = max(end - first, 0) % Q;   // tail: rows of the last chunk, if not whole
    const float la = a.log_decay[p.h];
    if (tid < 2 * Q) fill_update_weights<Q, AGE>(sm.w_up, sm.w_age, tid, la, a.s_wr, sh, tail);
    float age = 0.0f;   // the thread's share of dlog_decay, over its segment (shares are added in 64 bits)
    // factor of the age products: row t of the sequence, value columns 16 w + 4 lg .. + 3 of this tile
    // (0 past the columns and the rows; VEC: one load, always of the operand)
    const T *age_w = AGE ? static_cast<const T *>(a.age_w) + p.b * a.L * a.age_row + (p.h / (a.H / a.age_heads)) * a.dn + p.n0 : nullptr;
    auto age_factor = [&](int t) __attribute__((always_inline)) {
        const int n = 16 * w + 4 * lg;
        V4 g;
        if constexpr (VEC) {
            const V4 u = *reinterpret_cast<const V4 *>(age_w + min(t, p.Lb - 1) * a.age_row + (n < p.ncols ? n : 0));
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = n < p.ncols && t < end ? u[j] : 0;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = n + j < p.ncols && t < end ? age_w[t * a.age_row + n + j] : T(0);
        }
        return g;
    };
    const Lds sq = lds_of(sm.q), sk = lds_of(sm.k), sv = lds_of(sm.v);
    constexpr Lds KB = G::kQ * G::kRow, VB = G::kQ * G::kVRow;   // bytes of one buffer
    Lds qoff[O::kRowOffs], voff[O::kOneCol];   // the lane's places in rows of q, in columns of v
#pragma unroll
    for (int i = 0; i < O::kRowOffs; ++i) qoff[i] = opaque(sq + O::row_off(i, lr, lg, G::kRow));
#pragma unroll
    for (int i = 0; i < O::kOneCol; ++i) voff[i] = opaque(sv + O::one_off(i, w, lr, lg, G::kVRow));
    const Lds py = opaque(lds_of(sm.y) + w * sizeof(sm.y[0]) + lane * 16);
    using SmemT = Smem<T, DK, AGE>;
    constexpr Lds YA = offsetof(SmemT, ya) - offsetof(SmemT, y);   // from a share of y to its derivative's

    // every wave loads and stages an eighth of the rows, PF chunks ahead (AGE: one, as R takes the registers of
    // a second set, and spills cost more than the shorter lead)
    constexpr int PF = AGE ? 1 : kB;
    using Loader = Rows<T, DK, kThreads, true, VEC>;
    const Loader rows(a, p, tid, sq, sk, sv, KB, VB);
    typename Loader::Set set[PF];
    auto stage = [&](int t0, int buf, const typename Loader::Set &from) __attribute__((always_inline)) {
        const bool odd = rows.stage(t0, from, buf);
        const bool any = __ballot(odd) != 0;
        if (lane == 0) sm.odd[buf][wv] = any;
    };
    if (first < end) {
#pragma unroll
        for (int i = 0; i < PF; ++i) rows.load(first + i * Q, set[i]);
        stage(first, 0, set[0]);
        rows.load(first + PF * Q, set[0]);
    }
    // chunk by chunk: whole turns of kB chunks, then the rest (a way out in the middle of a turn would
    // make the compiler's waits at the top of the loop cover all loads).  The chunk at row t0 is in
    // LDS buffer `which`, its successor's rows in set (which + 1) % PF; further: rows are loaded ahead
    auto walk = [&](auto chunk) __attribute__((always_inline)) {
        __syncthreads();   // chunk 0 staged
        int t0 = first;
        for (; t0 + (kB - 1) * Q < end; t0 += kB * Q) {
            chunk(t0, std::integral_constant<int, 0>{}, std::true_type{});
            if constexpr (kB > 1) chunk(t0 + Q, std::integral_constant<int, 1 % kB>{}, std::true_type{});
        }
        if constexpr (kB > 1)
            if (t0 < end) chunk(t0, std::integral_constant<int, 0>{}, std::false_type{});
    };
    // With two buffers the next chunk is staged first thing (its buffer's last readers passed the barrier
    // before), beside the products instead of after them: B2 L4096 H32 128x128 bf16, forward and
    // backward, 533 -> 525 us.  (Single elements: at the end, else their addresses spill.)
    constexpr bool kEarly = kB == 2 && VEC;
    auto next_rows = [&](int t0, auto which, auto further) __attribute__((always_inline)) {
        constexpr int nbuf = (decltype(which)::value + 1) % kB, next = (decltype(which)::value + 1) % PF;
        if constexpr (kB == 1) __syncthreads();   // this chunk's rows read
        stage(t0 + Q, nbuf, set[next]);
        if constexpr (decltype(further)::value) rows.load(t0 + (PF + 1) * Q, set[next]);
    };

    if (wv < 4) {
        // ================= state waves =================
        Lds koff[O::kColOffs];
#pragma unroll
        for (int i = 0; i < O::kColOffs; ++i) koff[i] = opaque(sk + O::col_off(i, lr, lg, G::kRow));
        const Lds wup = opaque(lds_of(sm.w_up) + 16 * lg), wage = AGE ? opaque(lds_of(sm.w_age) + 16 * lg) : 0;
        f4 S[NT], R[AGE ? NT : 1];   // contraction row 16 t + 4 lg + j, column 16 w + lr
        const int n = p.n0 + 16 * w + lr;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kk = 16 * t + 4 * lg + j;
                float s0 = 0.0f, r0 = 0.0f;
                if (kk < a.dk && n < a.dn) {
                    if (p.seg > 0) {
                        const int64_t at = ((p.b * a.H + p.h) * (a.nseg - 1) + p.seg) * a.nsub * a.dk * a.dn -
                                           a.dk * a.dn + kk * a.ws_sr + n * a.ws_sc;   // the slot before its own first
                        s0 = a.ws_S[at];
                        if constexpr (AGE) r0 = a.ws_R[at];
                    } else if (a.h0) {
                        s0 = a.h0[(p.b * a.H + p.h) * a.dk * a.dn + kk * a.h_sr + n * a.h_sc];
                    }
                }
                S[t][j] = s0;
                if constexpr (AGE) R[t][j] = r0;
            }
        }
        const Decay full = decay_of(la, static_cast<float>(Q)), part = decay_of(la, static_cast<float>(tail));
        float w_rd[NB];   // s_rd lambda^(t + 1 - sh) of the lane's rows
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const Decay d = decay_of(la, static_cast<float>(16 * i + lr + 1 - sh));
            w_rd[i] = a.s_rd * (d.hi + d.lo);
        }
        walk([&](int t0, auto which, auto further) __attribute__((always_inline)) {
            constexpr int buf = decltype(which)::value;
            const int m = min(Q, end - t0);
            if constexpr (kEarly) next_rows(t0, which, further);
            // ---- the carried state's readout, y^T: lane column n = 4 lg + j, row t = lr
            f4 acc[NB], acca[AGE ? NB : 1];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                acc[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (AGE) acca[i] = acc[i];
            }
            constexpr bool AHEAD = G::kAhead && !AGE;
            Frag qf[AHEAD ? 2 : 1][NB];
            if constexpr (AHEAD)
#pragma unroll
                for (int i = 0; i < NB; ++i) qf[0][i] = O::row(buf * KB + 16 * i * G::kRow, qoff, 0);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int at = AHEAD ? c & 1 : 0, c1 = AHEAD ? c + 1 : c;
                if (c1 < NC)   // (AHEAD: the next rows' read meanwhile)
#pragma unroll
                    for (int i = 0; i < NB; ++i) qf[AHEAD ? at ^ 1 : 0][i] = O::row(buf * KB + 16 * i * G::kRow, qoff, c1);
                V4 s0[NS], s1[NS], r0[NS], r1[NS];
                O::template split<NS>(S[2 * c], s0);
                O::template split<NS>(S[2 * c + 1], s1);
                if constexpr (AGE) {
                    O::template split<NS>(R[2 * c], r0);
                    O::template split<NS>(R[2 * c + 1], r1);
                }
#pragma unroll
                for (int k = 0; k < NS; ++k)
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        acc[i] = O::mma(O::cat(s0[k], s1[k]), qf[at][i], acc[i]);
                        if constexpr (AGE) acca[i] = O::mma(O::cat(r0[k], r1[k]), qf[at][i], acca[i]);
                    }
                __builtin_amdgcn_sched_barrier(0);   // (no further ahead: the registers are full)
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                lds_put(py + i * 1024, acc[i] * w_rd[i]);
                if constexpr (AGE) lds_put(py + YA + i * 1024, acca[i] * w_rd[i] + acc[i] * (w_rd[i] * static_cast<float>(16 * i + lr + 1)));
            }
            __syncthreads();   // tiles built, shares written
            V4 vp[Q / 16];
#pragma unroll
            for (int j = 0; j < Q / 16; ++j) vp[j] = O::one(buf * VB + 16 * j * G::kVRow, voff);
            const Lds last = m == Q ? 0 : 4 * Q;
            update_state<T, Q, G::kRow, NT, AGE, G::kAhead && !AGE>(S, R, 0, buf * KB, koff, vp, wup + last, wage + last, m == Q ? full : part, m);
            if constexpr (!kEarly) next_rows(t0, which, further);
            __syncthreads();   // the next chunk staged
        });

        // ---- the state passed on
        if (end == p.Lb) {
            const int64_t at0 = (p.b * a.H + p.h) * a.dk * a.dn;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kk = 16 * t + 4 * lg + j;
                    if (kk < a.dk && n < a.dn) {
                        const int64_t at = at0 + kk * a.h_sr + n * a.h_sc;
                        if (a.h_last) a.h_last[at] = S[t][j];
                        // the last state's own gradient sees its age too
                        if constexpr (AGE)
                            if (a.age_dh) age = __builtin_fmaf(R[t][j], a.age_dh[at], age);
                    }
                }
        }
    } else {
        // ================= chunk waves =================
        // The wave's tiles (row block i, column block k), whose products run side by side: all of column
        // block w, where the rows reach it, and wave 3 takes the first tile besides its own
        //   wave 0: (3,0) (2,0) (1,0)   wave 1: (3,1) (2,1) (1,1)   wave 2: (3,2) (2,2)   wave 3: (3,3) (0,0)
        // and with two blocks: wave 0 (1,0), wave 1 (1,1), wave 2 (0,0).
        const int k0 = NB == 2 ? min(w, 1) : w, i1 = NB == 2 || w == 3 ? 0 : 2, k1 = NB == 2 || w == 3 ? 0 : w;
        const bool has0 = NB == 4 || w < 2, has1 = NB == 4 || w == 2, has2 = NB == 4 && w < 2;
        auto weights = [&](int i, int k) __attribute__((always_inline)) {   // s_in lambda^(t - s) of tile (i, k)
            f4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = 16 * (i - k) + lr - 4 * lg - j;
                const Decay p = decay_of(la, static_cast<float>(max(d, 0)));
                x[j] = d >= 0 ? a.s_in * (p.hi + p.lo) : 0.0f;
            }
            return x;
        };
        const f4 wt[3] = {weights(NB - 1, k0), weights(i1, k1), weights(1, k0)};
        Lds k0off[O::kRowOffs];   // the lane's places in rows of k, column block k0
#pragma unroll
        for (int i = 0; i < O::kRowOffs; ++i) k0off[i] = opaque(qoff[i] + (sk - sq) + 16 * k0 * G::kRow);
        const Lds k1_from_k0 = 16 * (k1 - k0) * G::kRow;   // (negative as it may be: addresses wrap)
        const Lds pp = opaque(lds_of(sm.p) + lane * sizeof(Frag)), ppa = AGE ? opaque(lds_of(sm.pa) + lane * sizeof(Frag)) : 0;
        constexpr Lds TB = 64 * sizeof(Frag), PB = G::kPairs * TB;   // bytes of a pair, of a part
        if (w == 0) {   // the pairs' empty halves
            const V4 zero = {};
            for (int i = 0; i < NB; i += 2) {
                for (int n = 0; n < O::kParts; ++n) lds_put(pp + pair_of(i, i) * TB + n * PB + Lds(sizeof(V4)), zero);
                if constexpr (AGE)
                    for (int n = 0; n < O::kParts; ++n) lds_put(ppa + pair_of(i, i) * TB + n * PB + Lds(sizeof(V4)), zero);
            }
        }
        auto product = [&](f4 (&g)[3], int buf, auto own) __attribute__((always_inline)) {
            constexpr bool OWN = decltype(own)::value;   // the second tile is of column block k0, too
            constexpr bool AHEAD = G::kAhead;
            Frag f[AHEAD ? 2 : 1][5];
            auto read = [&](int c, Frag (&x)[5]) __attribute__((always_inline)) {
                x[0] = O::row(buf * KB, k0off, c);
                x[2] = O::row(buf * KB + 16 * (NB - 1) * G::kRow, qoff, c);
                if (!OWN) x[1] = O::row(buf * KB + k1_from_k0, k0off, c);
                x[3] = O::row(buf * KB + 16 * i1 * G::kRow, qoff, c);
                if (OWN && NB == 4) x[4] = O::row(buf * KB + 16 * G::kRow, qoff, c);
            };
#pragma unroll
            for (int x = 0; x < 3; ++x) g[x] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (AHEAD) read(0, f[0]);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int at = AHEAD ? c & 1 : 0;
                if constexpr (!AHEAD) read(c, f[0]);
                else if (c + 1 < NC) read(c + 1, f[at ^ 1]);   // the next rows' read meanwhile
                g[0] = O::mma(f[at][0], f[at][2], g[0]);   // (a wave without a tile: not used)
                g[1] = O::mma(f[at][OWN ? 0 : 1], f[at][3], g[1]);
                if (OWN && NB == 4) g[2] = O::mma(f[at][0], f[at][4], g[2]);
                __builtin_amdgcn_sched_barrier(0);   // (no further ahead: the registers are full)
            }
        };
        auto put_tile = [&](const f4 &g, const f4 &wt, int i, int k) __attribute__((always_inline)) {
            // lane: s = 16 k + 4 lg + j, t = 16 i + lr
            const Lds at = pair_of(k, i) * TB + (k & 1) * sizeof(V4);
            const int d0 = 16 * (i - k) + lr - 4 * lg;
            f4 x = g * wt;
            if (i == k)   // rows after the output's: zero whatever q and k hold
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = d0 - j >= 0 ? x[j] : 0.0f;
            V4 part[O::kParts];
            O::template split<O::kParts>(x, part);
#pragma unroll
            for (int n = 0; n < O::kParts; ++n) lds_put(pp + at + n * PB, part[n]);
            if constexpr (AGE) {
                f4 xa;
#pragma unroll
                for (int j = 0; j < 4; ++j) xa[j] = x[j] * static_cast<float>(max(d0 - j, 0));
                V4 wide[O::kParts];
                O::template split<O::kParts>(xa, wide);
#pragma unroll
                for (int n = 0; n < O::kParts; ++n) lds_put(ppa + at + n * PB, wide[n]);
            }
        };
        const int col = 16 * w + 4 * lg;
        const int64_t ystep = p.dir * a.H * a.dn;
        const int64_t y0 = ((p.b * a.L + p.origin) * a.H + p.h) * a.dn + p.n0 + col;
        const bool full_cols = a.y_vec && col + 4 <= p.ncols;

        walk([&](int t0, auto which, auto further) __attribute__((always_inline)) {
            constexpr int buf = decltype(which)::value;
            const int m = min(Q, end - t0);
            V4 age_g[AGE ? NB : 1];
            if constexpr (AGE)
#pragma unroll
                for (int i = 0; i < NB; ++i) age_g[i] = age_factor(t0 + 16 * i + lr);
            if constexpr (kEarly) next_rows(t0, which, further);
            // ---- tiles of (q k^T)^T with their decay
            {
                f4 g[3];
                if (NB == 4 && w < 3) product(g, buf, std::true_type{});
                else if (NB == 4 || w < 3) product(g, buf, std::false_type{});
                if (has0) put_tile(g[0], wt[0], NB - 1, k0);
                if (has1) put_tile(g[1], wt[1], i1, k1);
                if (has2) put_tile(g[2], wt[2], 1, k0);
            }
            __syncthreads();   // tiles built, shares written
            const uint4 o0 = *reinterpret_cast<const uint4 *>(&sm.odd[buf][0]), o1 = *reinterpret_cast<const uint4 *>(&sm.odd[buf][4]);
            const bool odd = __builtin_amdgcn_readfirstlane(o0.x | o0.y | o0.z | o0.w | o1.x | o1.y | o1.z | o1.w) != 0;
            // The diagonal tiles' zeros (rows after the output's) must not meet an infinity or NaN: where
            // a chunk has one (next to none does), such values are taken out of the products, and added
            // to the shares of their own and later rows here, one by one
            if (odd) {
#pragma unroll 1
                for (int i = 0; i < NB; ++i) {
                    f4 y = lds_get<f4>(py + i * 1024), ya = lds_get<f4>(py + (AGE ? YA + i * 1024 : 0));
#pragma unroll 1
                    for (int r = 0; r <= lr; ++r) {
                        // the lane that holds row r, column lr of the tile
                        const Lds from = ((r >> 2) * 16 + lr - lane) * sizeof(Frag) + pair_of(i, i) * TB + (i & 1) * sizeof(V4);
                        float pr = 0.0f;
                        for (int n = 0; n < O::kParts; ++n) pr += O::element(lds_get<V4>(pp + n * PB + from), r & 3);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = 16 * i + r, c = col + j, piece = c / (16 / static_cast<int>(sizeof(T)));
                            const int in = c % (16 / static_cast<int>(sizeof(T))) * static_cast<int>(sizeof(T)) ^ (sizeof(T) == 2 ? at & 8 : 0);
                            const float x = widen_v(lds_get<T>(sv + buf * VB + at * G::kVRow + ((piece ^ O::swizzle(at)) << 4) + in));
                            if ((__float_as_uint(x) & 0x7f800000u) != 0x7f800000u) continue;
                            y[j] = __builtin_fmaf(pr, x, y[j]);
                            ya[j] = __builtin_fmaf(pr * static_cast<float>(lr - r), x, ya[j]);
                        }
                    }
                    lds_put(py + i * 1024, y);
                    if constexpr (AGE) lds_put(py + YA + i * 1024, ya);
                }
            }
            // ---- the tiles times v, on top of the carried state's share
            f4 acc[NB], acca[AGE ? NB : 1];
            V4 vp[NB], vd[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                vp[i] = vd[i] = O::one(buf * VB + 16 * i * G::kVRow, voff);
                acc[i] = lds_get<f4>(py + i * 1024);
                if constexpr (AGE) acca[i] = lds_get<f4>(py + YA + i * 1024);
            }
            if (odd) {
                asm volatile("");   // (a branch, not selects)
#pragma unroll
                for (int i = 0; i < NB; ++i) vd[i] = O::only_finite4(vp[i]);
            }
            // (all pairs of a part read before the products: read one by one, each product waited for its own)
            auto times_v = [&](f4 (&to)[NB], Lds from) __attribute__((always_inline)) {
                Frag f[G::kPairs];
#pragma unroll
                for (int x = 0; x < G::kPairs; ++x) f[x] = O::pair(from + x * TB);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < NB; k += 2)
#pragma unroll
                    for (int i = k; i < NB; ++i)
                        to[i] = O::mma(O::cat(k == i ? vd[k] : vp[k], i <= k + 1 ? vd[k + 1] : vp[k + 1]), f[pair_of(k, i)], to[i]);
            };
#pragma unroll
            for (int n = 0; n < O::kParts; ++n) times_v(acc, pp + n * PB);
            if constexpr (AGE)
#pragma unroll
                for (int n = 0; n < O::kParts; ++n) times_v(acca, ppa + n * PB);
            const int64_t yt = y0 + (t0 + lr) * ystep;
            if (sizeof(T) == 2 && !a.out_f32 && full_cols) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if (16 * i + lr < m)
                        *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.y) + yt + 16 * i * ystep) =
                            u2{pack_bf16(acc[i][0], acc[i][1]), pack_bf16(acc[i][2], acc[i][3])};
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (16 * i + lr >= m) continue;
                    const int64_t at = yt + 16 * i * ystep;
                    if (sizeof(T) == 2 && !a.out_f32) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (col + j < p.ncols) put(static_cast<uint16_t *>(a.y), at + j, acc[i][j]);
                    } else if (full_cols) {
                        *reinterpret_cast<f4 *>(static_cast<float *>(a.y) + at) = acc[i];
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (col + j < p.ncols) static_cast<float *>(a.y)[at + j] = acc[i][j];
                    }
                }
            }
            if constexpr (AGE)
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const f4 g = O::widen4(age_g[i]);
                    const bool in = 16 * i + lr < m;   // (a growing "decay" may overflow in the rows behind the last)
#pragma unroll
                    for (int j = 0; j < 4; ++j) age = __builtin_fmaf(in ? acca[i][j] : 0.0f, g[j], age);
                }
            if constexpr (!kEarly) next_rows(t0, which, further);
            __syncthreads();   // the next chunk staged
        });
    }
    if constexpr (AGE) {
        // the workgroup's share of dlog_decay, summed in a fixed order
        sm.red[tid] = age;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o) sm.red[tid] += sm.red[tid + o];
            __syncthreads();
        }
        if (tid == 0) a.age_part[share] = sm.red[0];
    }
}

// ---- the segments' own contributions to the state (from zero), into the workspace, in nsub parts of a
// segment that run side by side: eight waves, wave w value columns 16 (w % 4) .. + 15 and half w / 4 of
// the contraction columns.  B1 L32768 H16 128x128 bf16 (7 of 8 segments, two parts each): 77 us, 3.1 TB/s,
// bound by the loads' latency at one or two workgroups a CU.
template <class T, int DK, bool AGE, bool VEC>
__global__ void __launch_bounds__(kThreads) linattn_state_kernel(LinAttnArgs a) {
    using G = Tile<T, DK>;
    using O = Op<T>;
    constexpr int Q = G::kQ, NT = DK / 32;
    __shared__ __align__(16) char tk[2][Q * G::kRow], tv[2][Q * G::kVRow];
    __shared__ __align__(16) float w_up[2][Q], w_age[AGE ? 2 * Q : 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), w = wv & 3, hf = wv >> 2;
    const int lr = lane & 15, lg = lane >> 4;
    Part<T> p;
    if (!p.set(a, (a.nseg - 1) * a.nsub)) return;
    const int of = static_cast<int>(p.seg / a.nsub), sub = static_cast<int>(p.seg % a.nsub), sub_len = static_cast<int>(a.sub_len);
    const int seg_end = (of + 1) * p.seg_len;
    if (seg_end >= p.Lb) return;   // no later segment starts from this one's state
    p.first = of * p.seg_len + sub * sub_len;
    p.end = min(p.first + sub_len, seg_end);
    const float la = a.log_decay[p.h];
    if (tid < 2 * Q) fill_update_weights<Q, AGE>(w_up, w_age, tid, la, a.s_wr, a.reverse ? 1 : 0, 0);
    const Lds sk = lds_of(tk), sv = lds_of(tv);
    constexpr Lds KB = sizeof(tk[0]), VB = sizeof(tv[0]);
    Lds koff[O::kColOffs], voff[O::kOneCol];
#pragma unroll
    for (int i = 0; i < O::kColOffs; ++i) koff[i] = opaque(sk + O::col_off(i, lr, lg, G::kRow));
#pragma unroll
    for (int i = 0; i < O::kOneCol; ++i) voff[i] = opaque(sv + O::one_off(i, w, lr, lg, G::kVRow));
    const Lds wup = opaque(lds_of(w_up) + 16 * lg), wage = AGE ? opaque(lds_of(w_age) + 16 * lg) : 0;
    f4 S[NT], R[AGE ? NT : 1];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        S[t] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (AGE) R[t] = S[t];
    }
    const Decay full = decay_of(la, static_cast<float>(Q));
    using Loader = Rows<T, DK, kThreads, false, VEC>;
    const Loader rows(a, p, tid, sk, sk, sv, KB, VB);
    typename Loader::Set set[2];
    rows.load(p.first, set[0]);
    rows.load(p.first + Q, set[1]);
    rows.stage(p.first, set[0], 0);
    rows.load(p.first + 2 * Q, set[0]);
    __syncthreads();
    // (whole chunks: seg_len and sub_len are multiples of Q)
    auto chunk = [&](int t0, auto which, auto further) __attribute__((always_inline)) {
        constexpr int buf = decltype(which)::value;
        typename O::V4 vp[Q / 16];
#pragma unroll
        for (int j = 0; j < Q / 16; ++j) vp[j] = O::one(buf * VB + 16 * j * G::kVRow, voff);
        update_state<T, Q, G::kRow, NT, AGE, G::kAhead>(S, R, hf * NT, buf * KB, koff, vp, wup, wage, full, Q);
        rows.stage(t0 + Q, set[buf ^ 1], buf ^ 1);
        if constexpr (decltype(further)::value) rows.load(t0 + 3 * Q, set[buf ^ 1]);
        __syncthreads();
    };
    int t0 = p.first;
    for (; t0 + Q < p.end; t0 += 2 * Q) {
        chunk(t0, std::integral_constant<int, 0>{}, std::true_type{});
        chunk(t0 + Q, std::integral_constant<int, 1>{}, std::true_type{});
    }
    if (t0 < p.end) chunk(t0, std::integral_constant<int, 0>{}, std::false_type{});
    const int64_t at0 = ((p.b * a.H + p.h) * (a.nseg - 1) * a.nsub + p.seg) * a.dk * a.dn;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t kk = 16 * (hf * NT + t) + 4 * lg + j, n = p.n0 + 16 * w + lr;
            if (kk < a.dk && n < a.dn) {
                a.ws_S[at0 + kk * a.dn + n] = S[t][j];
                if constexpr (AGE) a.ws_R[at0 + kk * a.dn + n] = R[t][j];
            }
        }
}

// Own contributions of the segments' parts -> the states that segments 1, 2, ... start from, each in the
// slot of its predecessor's last part: H <- lambda^T H + own over the parts (T rows to a part), and with
// R its derivative by log_decay.  Bound by latency: a thread takes four elements of one state, and reads
// eight parts of them ahead of the chain.
template <bool AGE>
__global__ void __launch_bounds__(256) linattn_combine_kernel(LinAttnArgs a) {
    constexpr int E = 4, P = AGE ? 4 : 8;
    __shared__ Decay decay[2];
    const int64_t sz = a.dk * a.dn, per = (sz + 256 * E - 1) / (256 * E);
    const int64_t bh = blockIdx.x / per, e0 = blockIdx.x % per * (256 * E) + threadIdx.x;
    int64_t Lb = a.L;
    if (a.lengths) Lb = min(max(static_cast<int64_t>(a.lengths[bh / a.H]), int64_t(0)), a.L);
    const int starts = static_cast<int>(min(a.nseg - 1, (Lb - 1) / a.seg_len)), nsub = static_cast<int>(a.nsub), parts = starts * nsub;
    if (parts <= 0) return;
    // (the last part of a segment is what the others leave)
    const int64_t last_len = a.seg_len - (a.nsub - 1) * a.sub_len;
    // (hi + lo, as within a part: the parts' decays are all alike, and so is what rounding them would lose)
    if (threadIdx.x < 2) {
        const double x = exp(static_cast<double>(a.log_decay[bh % a.H]) * static_cast<double>(threadIdx.x ? last_len : a.sub_len));
        const float hi = static_cast<float>(x);
        decay[threadIdx.x] = Decay{hi, hi < INFINITY ? static_cast<float>(x - static_cast<double>(hi)) : 0.0f};
    }
    __syncthreads();
    const Decay d = decay[0], d1 = decay[1];
    const float T = static_cast<float>(a.sub_len), T1 = static_cast<float>(last_len);
    const int64_t at0 = bh * (a.nseg - 1) * nsub * sz;
    float S[E], R[E];
#pragma unroll
    for (int x = 0; x < E; ++x) {
        const int64_t e = min(e0 + x * 256, sz - 1);
        S[x] = a.h0 ? a.h0[bh * sz + e / a.dn * a.h_sr + e % a.dn * a.h_sc] : 0.0f;
        R[x] = 0.0f;
    }
    for (int s0 = 0; s0 < parts; s0 += P) {
        float own[P][E], own_R[AGE ? P : 1][E];
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (s0 + i < parts)
#pragma unroll
                for (int x = 0; x < E; ++x) {
                    const int64_t at = at0 + (s0 + i) * sz + min(e0 + x * 256, sz - 1);
                    own[i][x] = a.ws_S[at];
                    if constexpr (AGE) own_R[i][x] = a.ws_R[at];
                }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (s0 + i >= parts) continue;
            const bool last = (s0 + i + 1) % nsub == 0;
            const Decay by = last ? d1 : d;
#pragma unroll
            for (int x = 0; x < E; ++x) {
                if constexpr (AGE) {
                    const float r = __builtin_fmaf(last ? T1 : T, S[x], R[x]);
                    R[x] = __builtin_fmaf(by.hi, r, __builtin_fmaf(by.lo, r, own_R[i][x]));
                }
                S[x] = __builtin_fmaf(by.hi, S[x], __builtin_fmaf(by.lo, S[x], own[i][x]));
                if (last && e0 + x * 256 < sz) {
                    const int64_t at = at0 + (s0 + i) * sz + e0 + x * 256;
                    a.ws_S[at] = S[x];
                    if constexpr (AGE) a.ws_R[at] = R[x];
                }
            }
        }
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
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t d = i % D, g = i / D % G, row = i / (D * G);
        const float *p = part + (row * G + g) * per * D + d;
        float s = 0.0f;
        for (int64_t j = 0; j < per; ++j) s += p[j * D];
        put(out, i, s);
    }
}

// One token: every state element is read and written once, so the launch is bound by the
// state's traffic.  A workgroup takes 64 value columns of one (b, h); thread: four columns (16
// bytes) of every sixteenth contraction row.  (B256 H32 128x64 bf16: 85 us, 6.3 TB/s of state, some of it
// from the Infinity Cache; 16 columns to a workgroup 138 us, and where that fills more CUs 6.7 against
// 5.2 us (B4), 5.3 against 4.9 us (B1, 128x128), 4.0 against 4.2 us (B1 H16 64x64).)
template <class T>
__global__ void __launch_bounds__(256) linattn_update_kernel(LinAttnArgs a) {
    constexpr int CW = kN, C4 = CW / 4, RG = 256 / C4;
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

template <class T, int DK, bool AGE>
hipError_t launch_sweep(const LinAttnArgs &a0, hipStream_t s) {
    LinAttnArgs a = a0;
    static_assert(sizeof(Smem<T, DK, AGE>) <= kLdsPerCU, "LDS of one CU");
    auto grid = [&](int64_t segs) {
        a.work = a.B * a.H * segs * a.ntiles;
        return dim3(static_cast<unsigned>((a.work + 7) / 8 * 8));
    };
    if (a.nseg > 1 && !a.have_states) {
        const dim3 g = grid((a.nseg - 1) * a.nsub);
        if (a.vec) hipLaunchKernelGGL((linattn_state_kernel<T, DK, AGE, true>), g, dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((linattn_state_kernel<T, DK, AGE, false>), g, dim3(kThreads), 0, s, a);
        hipError_t e = launch_status(s);
        if (e != hipSuccess) return e;
        const dim3 blocks(static_cast<unsigned>(a.B * a.H * ((a.dk * a.dn + 1023) / 1024)));
        hipLaunchKernelGGL((linattn_combine_kernel<AGE>), blocks, dim3(256), 0, s, a);
        e = launch_status(s);
        if (e != hipSuccess) return e;
    }
    const dim3 g = grid(a.nseg);
    if (a.vec) hipLaunchKernelGGL((linattn_kernel<T, DK, AGE, true>), g, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((linattn_kernel<T, DK, AGE, false>), g, dim3(kThreads), 0, s, a);
    return launch_status(s);
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
    if (a.age_part) a.vec = a.vec && a.age_row % ve == 0;
    a.y_vec = a.dn % 4 == 0;
    return bf16 ? launch_typed<uint16_t>(a, s) : launch_typed<float>(a, s);
}

hipError_t launch_linattn_age_sum(const LinAttnArgs &a, float *dlog_decay, hipStream_t s) {
    hipLaunchKernelGGL(linattn_age_sum_kernel, dim3(static_cast<unsigned>(a.H)), dim3(64), 0, s, a.age_part, dlog_decay, a.B,
                       a.H, a.nseg * a.ntiles);
    return launch_status(s);
}

hipError_t launch_linattn_share(const float *part, void *out, int64_t rows, int64_t H, int64_t G, int64_t D, bool bf16, hipStream_t s) {
    const int64_t n = rows * G * D;
    const dim3 grid(static_cast<unsigned>(n < (int64_t(1) << 30) ? (n + 255) / 256 : int64_t(1) << 22));
    if (bf16) hipLaunchKernelGGL((linattn_share_kernel<uint16_t>), grid, dim3(256), 0, s, part, static_cast<uint16_t *>(out), n, G, D, H / G);
    else hipLaunchKernelGGL((linattn_share_kernel<float>), grid, dim3(256), 0, s, part, static_cast<float *>(out), n, G, D, H / G);
    return launch_status(s);
}

hipError_t launch_linattn_update(const LinAttnArgs &a0, bool bf16, hipStream_t s) {
    LinAttnArgs a = a0;
    a.y_vec = a.dn % 4 == 0;
    const dim3 grid(static_cast<unsigned>(a.B * a.H * ((a.dn + kN - 1) / kN)));
    if (bf16) hipLaunchKernelGGL((linattn_update_kernel<uint16_t>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((linattn_update_kernel<float>), grid, dim3(256), 0, s, a);
    return launch_status(s);
}

}  // namespace ssm
