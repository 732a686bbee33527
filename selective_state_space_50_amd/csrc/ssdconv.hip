// A Mamba-2 layer's mixer as it is served: the short causal convolution (+ SiLU) over the channels of x, B and C and
// the multi-head scan behind it (the recurrence of ssd.hip), over packed sequences whose states lie in a pool, and for
// one token of every sequence.
//
// Per sequence and token, xbc the row of all channels (x [H, P], B [G, N], C [G, N]):
//     a_t = bias + sum_{k < W} w[:, k] xbc_{t-W+1+k},   (x, B, C) = silu(a_t)
//     dt  = delta (+ bias, softplus optional),   S_t = exp(dt A_h) S_{t-1} + dt x_t B_t^T   (S [P, N] per head)
//     y_t = (S_t C_t + D_h x_t) silu(z_t)
// and over a chunk of 64 tokens from the state S, cum the running sum of dt A within the chunk:
//     y_t = sum_{s<=t} (C_t . B_s) e^(cum_t - cum_s) dt_s x_s + e^(cum_t) S C_t + D x_t
//     S'  = e^(cum_64) S + sum_s e^(cum_64 - cum_s) dt_s x_s B_s^T
//
// Three parts:
//  * prep (a workgroup per chunk and B/C group, and per chunk and 64 heads): what all heads of a group share. B and C
//    behind the convolution, cut into bf16 parts and stored as the lanes' operands of the products to come, C B^T of the
//    chunk, and per head the decays. A sequence's first chunk starts at its first token, so no chunk holds two sequences.
//  * sweep (a workgroup per sequence, head and 64 channels): walks the chunks with the state in registers.  x is
//    convolved on its way to LDS: neither x, B nor C behind the convolution is ever rounded to the input type, and x goes to
//    memory once less than with a convolution of its own.
//  * few heads over long sequences: the sequence in segments. A sweep without outputs makes each segment's own end state,
//    join passes the states on, and the sweep starts every segment from its own.
//
// Numbers: a product of two 32-bit factors runs on v_mfma_f32_16x16x32_bf16 in parts: v = hi + mid + lo, bf16 each, holds
// all 24 bits, and six products of parts those whose order of magnitude is above 2^-24.  That holds for the state and for y,
// whatever the input type: two parts of y's factors left 0.23% of bf16 outputs a step off, three 0.010% (a 32-bit form 0.011%).
// Exponents are sums over at most 32 tokens, made in 64 bits: forwards for reads and backwards for writes, which decays between
// the halves are products of.  Within a half the decay from s to t is 2 to the difference of two sums from the half's start.  A
// difference keeps their absolute error, so one large step would spoil every later pair (fp32, a step of dt A = 1600: 2e-4 of a
// pair's weight): the sums are kept as hi + lo, lo in the input type (32 bits in all for bf16, 48 for fp32), and the
// difference is as good as its own 24 bits.
//
// What bounds it (B4 L4096 H64 P64 N128, gated, bf16; 347 us, whose 422 MB would take 84 at a copy's rate): the sweep, 94% of
// the time.  Per chunk and head 14.9 MFLOP of products in parts (201 us at a large library product's rate) run beside about 580
// vector instructions a wave (convolution, decays, cutting into parts), 600 KB through LDS and 200 KB from the L2; the vector units
// are busy 52% of the time, the matrix cores 32%, LDS about half, at a clock that the load itself holds near 1.95 GHz.  The prep's
// 22 us are the 45 MB of operands and decays that it writes (all heads read them from the L2s; written past the caches: 2 us
// slower).  B1 L32768 H24: 384 us in segments, 2477 whole.  With y's factors in two parts, workgroups of four waves and 32 channels,
// two to a CU, took 304 us against 276.
#include "ssm_device.h"

#include <type_traits>

namespace ssm {
namespace {

constexpr int kQ = 64;                 // tokens of a chunk
constexpr int kThreads = 512;          // of a sweep
constexpr int kPrepThreads = 1024;
constexpr int kParts = 3;              // bf16 parts of a product's factors
// A head's tables of a chunk, 64 values each but kWb:
enum {
    kWr = 0,            // e^(cum_64 - cum_s) dt_s    weight of token s in the state passed on
    kC32 = kWr + kQ,    // exponent of the decay from the 32-token half's start to t, to the base 2 (the carried state's decay
                        // up to t is 2 to it, times the first half's whole in the second half)
    kDt = kC32 + kQ,    // dt_s
    kWb = kDt + kQ,     // e^(to the half's end) dt_s: weight of the first half's token s in what the second half reads (32 values)
    kLo = kWb + kQ / 2  // what kC32 was rounded by, in the input type
};
template <class T>
constexpr int kTab = kLo + kQ * static_cast<int>(sizeof(T)) / 4;   // words of a head's tables

typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
// 16 bytes at the address of an element: z may be a part of a wider row, whose length is no multiple of 16 bytes
template <class T>
struct Piece;
template <> struct Piece<uint16_t> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct Piece<float> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4))); };

__device__ __forceinline__ f4 mfma(s8 a, s8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// the sum of the parts' products that lie above 2^-(8 N): i + j < N
template <int N>
__device__ __forceinline__ f4 product(const s8 (&a)[N], const s8 (&b)[N], f4 c) {
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
#pragma unroll
        for (int j = N - 1 - i; j >= 0; --j) c = mfma(a[i], b[j], c);
    return c;
}

// v[0 .. K - 1] in N bf16 parts, two to a word: part n's words at w[n]
template <int N, int K>
__device__ __forceinline__ void split(const float *v, uint32_t (&w)[N][K / 2]) {
#pragma clang fp contract(off)   // (the parts of v as it was rounded, wherever it comes from)
#pragma unroll
    for (int i = 0; i < K / 2; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            w[n][i] = pack_bf16(a, b);
            if (n + 1 < N) {
                a -= bf_lo(w[n][i]);
                b -= bf_hi(w[n][i]);
            }
        }
    }
}
template <int N>
__device__ __forceinline__ void split8(const float *v, s8 (&out)[N]) {
    uint32_t w[N][4];
    split<N, 8>(v, w);
#pragma unroll
    for (int n = 0; n < N; ++n) out[n] = __builtin_bit_cast(s8, u4{w[n][0], w[n][1], w[n][2], w[n][3]});
}

// which sequence chunk (or segment) v belongs to, sequence s owning the numbers from offset_s / len + s on (as many as
// its tokens can need: no sums over the sequences before it); -1: none.  Wave-uniform.  Where offsets decrease it may be
// another sequence, whose numbers start behind v: callers look for that.
__device__ __forceinline__ int clamped(const SsdConvArgs &a, int s) {
    const int o = a.offsets[s];
    return o < 0 ? 0 : o > a.T ? static_cast<int>(a.T) : o;
}
__device__ __forceinline__ int find_sequence(const SsdConvArgs &a, int len, int64_t v) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.S;
    while (true) {
        const int step = (n + 63) >> 6, s = lo + lane * step;
        const bool in = lane * step < n && static_cast<int64_t>(clamped(a, s) / len + s) <= v;
        const int c = __popcll(__ballot(in));
        if (c == 0) return -1;
        lo += (c - 1) * step;
        n -= (c - 1) * step;
        if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
        if (n > step) n = step;
    }
}

struct Sequence {
    int s, first, len, slot;      // first row, tokens, slot of the states (-1: none)
    bool old;                     // goes on from the slot's states
    __device__ Sequence(const SsdConvArgs &a, int s_) : s(s_) {
        first = clamped(a, s);
        const int end = clamped(a, s + 1);
        len = end > first ? end - first : 0;
        slot = a.slots ? a.slots[s] : s;
        if (slot < 0 || slot >= a.nslots) slot = -1;
        old = slot >= 0 && !(a.fresh && a.fresh[s]);
        first = __builtin_amdgcn_readfirstlane(first);
        len = __builtin_amdgcn_readfirstlane(len);
        slot = __builtin_amdgcn_readfirstlane(slot);
    }
};

// Rows t0 - 3 .. t0 + K - 1 of one channel of a sequence (t0 counted from its start; what lies before the start comes
// from the convolution's state, zeros without one; what lies behind the end is not used).
template <class T, int K>
struct Window {
    T x[K + 3];
    // (t0 >= 3: rows one after another, the last one again behind the end)
    __device__ __forceinline__ void load_on(const SsdConvArgs &a, const Sequence &q, int channel, int t0) {
        int t = t0 - 3 < q.len - 1 ? t0 - 3 : q.len - 1;
        const T *X = static_cast<const T *>(a.xbc) + (q.first + static_cast<int64_t>(t)) * a.x_row;
#pragma unroll
        for (int i = 0; i < K + 3; ++i, ++t) {
            x[i] = X[channel];
            X += t < q.len - 1 ? a.x_row : 0;
        }
    }
    __device__ __forceinline__ void load(const SsdConvArgs &a, const Sequence &q, int channel, int t0) {
        const T *X = static_cast<const T *>(a.xbc) + channel;
#pragma unroll
        for (int i = 0; i < K + 3; ++i) {
            int t = t0 + i - 3;
            t = t < 0 ? 0 : t >= q.len ? q.len - 1 : t;      // a row that is there
            x[i] = X[(q.first + static_cast<int64_t>(t)) * a.x_row];
        }
        if (t0 < 3) before(a, q, channel, t0);
    }
    __device__ void before(const SsdConvArgs &a, const Sequence &q, int channel, int t0) {
        const int W1 = a.W - 1;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int t = t0 + i - 3;
            if (t >= 0) continue;
            x[i] = T{};
            if (q.old && t + W1 >= 0)
                x[i] = static_cast<const T *>(a.conv_state)[(static_cast<int64_t>(q.slot) * a.C + channel) * W1 + t + W1];
        }
    }
};

// silu of the convolution over eight tokens of a window, from its token r on.  A filter of W < 4 columns leaves the earliest
// rows out, or (FULL) has weights of 0 for them: of x a NaN there is in its channel's state already, and branches would
// part the code that the compiler may overlap.
template <bool FULL, class T, int K>
__device__ __forceinline__ void convolve(const Window<T, K> &in, int r, const float (&w)[4], float bias, int W, float *o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = bias;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (FULL || k >= 4 - W) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __builtin_fmaf(w[k], widen_v(in.x[r + i + k]), o[i]);
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = silu_f(o[i]);
}

__device__ __forceinline__ void filter(const SsdConvArgs &a, int channel, float (&w)[4], float &bias) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = k >= 4 - a.W ? a.w[static_cast<int64_t>(channel) * a.W + k - (4 - a.W)] : 0.0f;
    bias = a.bias ? a.bias[channel] : 0.0f;
}

// One channel's last W - 1 inputs (what a sequence shorter than that leaves of the old ones in front), and into its slot.
template <class T>
__device__ __forceinline__ void last_inputs(const SsdConvArgs &a, const Sequence &q, int channel, T (&v)[3]) {
    const int W1 = a.W - 1;
    const T *st = static_cast<const T *>(a.conv_state) + (static_cast<int64_t>(q.slot) * a.C + channel) * W1;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int k = q.len + j;            // of the old columns and the tokens side by side
        if (j >= W1) v[j] = T{};
        else if (k < W1) v[j] = q.old ? st[k] : T{};
        else v[j] = static_cast<const T *>(a.xbc)[(q.first + static_cast<int64_t>(k - W1)) * a.x_row + channel];
    }
}
template <class T>
__device__ __forceinline__ void keep_inputs(const SsdConvArgs &a, const Sequence &q, int channel, const T (&v)[3]) {
    const int W1 = a.W - 1;
    T *st = static_cast<T *>(a.conv_state) + (static_cast<int64_t>(q.slot) * a.C + channel) * W1;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (j < W1) st[j] = v[j];
}

// ---------------------------------------------------------------------------- prep

// Sums over the lanes up to (BACK: from) a lane, within each half of 32: four row shifts, then the first (second) row's whole.
template <bool BACK>
__device__ __forceinline__ double half_scan(double v, int lane) {
    const auto moved = [&](auto how) __attribute__((always_inline)) {
        const int2 w = __builtin_bit_cast(int2, v);
        return __builtin_bit_cast(double, int2{how(w.x), how(w.y)});
    };
    const auto add = [&](auto ctrl) __attribute__((always_inline)) {
        v += moved([](int w) { return __builtin_amdgcn_update_dpp(0, w, decltype(ctrl)::value, 0xf, 0xf, true); });
    };
    constexpr int kShift = BACK ? 0x100 : 0x110;     // row_shl, row_shr: what would come from another row is zero
    add(std::integral_constant<int, kShift + 1>{});
    add(std::integral_constant<int, kShift + 2>{});
    add(std::integral_constant<int, kShift + 4>{});
    add(std::integral_constant<int, kShift + 8>{});
    const double lo = moved([](int w) { return __builtin_amdgcn_readlane(w, BACK ? 16 : 15); });
    const double hi = moved([](int w) { return __builtin_amdgcn_readlane(w, BACK ? 48 : 47); });
    if ((lane & 16) == (BACK ? 0 : 16)) v += lane < 32 ? lo : hi;
    return v;
}

// NP: the states padded to 64 or 128.  Sixteen waves: 22 us on B4 L4096 H64, about 5 of one thing
// waiting for the other, then 45 MB of operands and tables written (eight took as long as sixteen).
template <class T, int NP>
__global__ void __launch_bounds__(kPrepThreads) ssdconv_prep_kernel(SsdConvArgs a) {
    constexpr int kRow = NP + 4;
    __shared__ __align__(16) float tile[2][kQ][kRow];    // B and C, token by token
    const int64_t u = blockIdx.x;
    const int s = find_sequence(a, kQ, u);
    if (s < 0) return;
    const Sequence q(a, s);
    const int64_t own = u - (q.first / kQ + s);           // (below 0 only where offsets decrease)
    const int t0 = static_cast<int>(own) * kQ;
    if (own < 0 || t0 >= q.len) return;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;

    if (static_cast<int>(blockIdx.y) >= a.G) {   // ---- the decays of 64 heads, four to a wave
        const int h0 = (static_cast<int>(blockIdx.y) - a.G) * 64 + wv * 4;
        const T *D = static_cast<const T *>(a.delta) + (q.first + static_cast<int64_t>(t0 + lane < q.len ? t0 + lane : q.len - 1)) * a.d_row;
        T raw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) raw[k] = D[h0 + k < a.H ? h0 + k : a.H - 1];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + k;
            if (h >= a.H) break;
            float dt = widen_v(raw[k]);
            if (a.dbias) dt += a.dbias[h];
            if (a.softplus) dt = softplus_f(dt);
            if (t0 + lane >= q.len) dt = 0.0f;
            const double step = static_cast<double>(dt) * (static_cast<double>(a.A[h]) * 1.4426950408889634074);
            const double pre = half_scan<false>(step, lane);                                             // inclusive
            const float c32 = static_cast<float>(pre), suf = static_cast<float>(half_scan<true>(step, lane));
            const float behind = __shfl_down(suf, 1, 32);
            const float wb = __builtin_amdgcn_exp2f((lane & 31) == 31 ? 0.0f : behind) * dt;
            const float half1 = __shfl(__builtin_amdgcn_exp2f(c32), 63, 64);
            float *t = a.ws_tab + (u * a.H + h) * kTab<T>;
            t[kWr + lane] = lane < 32 ? wb * half1 : wb;
            t[kC32 + lane] = c32;
            t[kDt + lane] = dt;
            if (lane < 32) t[kWb + lane] = wb;
            put(reinterpret_cast<T *>(t + kLo), lane, static_cast<float>(pre - static_cast<double>(c32)));
        }
        return;
    }

    // ---- B and C of group g behind the convolution: a thread per channel and run of tokens
    const int g = blockIdx.y;
    constexpr int kTok = kQ * 2 * NP / kPrepThreads;     // 16 or 8
    const int ch = threadIdx.x % (2 * NP), n = ch % NP, which = ch / NP, from = threadIdx.x / (2 * NP) * kTok;
    const int channel = a.H * a.P + (which * a.G + g) * a.N + n;
    s8 *bt = reinterpret_cast<s8 *>(a.ws_bt) + (u * a.G + g) * (NP / 16 * 2 * kParts * 64);
    Window<T, 8> in;
    float w[4], bias = 0.0f;
    if (n < a.N) {
        in.load(a, q, channel, t0 + from);
        filter(a, channel, w, bias);
    }
#pragma unroll 1
    for (int t = from; t < from + kTok; t += 8) {
        float o[8];
        if (n < a.N) {
            const Window<T, 8> now = in;
            in.load_on(a, q, channel, t0 + t + 8);
            convolve<false>(now, 0, w, bias, a.W, o);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (n >= a.N || t0 + t + i >= q.len) o[i] = 0.0f;
            tile[which][t + i][n] = o[i];
        }
        if (which == 0) {
            // operands of the state's product: lane (n % 16, s / 8 % 4) of slice n / 16 holds B[s .. s + 7][n]
            s8 part[kParts];
            split8<kParts>(o, part);
#pragma unroll
            for (int k = 0; k < kParts; ++k)
                bt[((n / 16 * 2 + t / 32) * kParts + k) * 64 + n % 16 + 16 * (t % 32 / 8)] = part[k];
        }
    }
    __syncthreads();
    // ---- operands of C, and C B^T below the diagonal: wave (i, k) takes C's tokens 16 i .. and B's 16 k .., and of the
    // operands every fourth
    const int i = wv & 3, k = wv >> 2;
    s8 *cs = reinterpret_cast<s8 *>(a.ws_c) + ((u * a.G + g) * 4 + i) * (NP / 32 * kParts * 64) + lane;
    f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kk = 0; kk < NP / 32; ++kk) {
        if (k > i && kk != k) continue;
        s8 cf[kParts], bf[kParts];
        split8<kParts>(&tile[1][16 * i + lr][32 * kk + 8 * lg], cf);
        if (kk == k) {
#pragma unroll
            for (int e = 0; e < kParts; ++e) cs[(kk * kParts + e) * 64] = cf[e];
        }
        if (k > i) continue;
        split8<kParts>(&tile[0][16 * k + lr][32 * kk + 8 * lg], bf);
        acc = product<kParts>(bf, cf, acc);
    }
    // lane: token 16 i + lr, s = 16 k + 4 lg + 0 .. 3
    if (k <= i) *reinterpret_cast<f4 *>(a.ws_cb + ((u * a.G + g) * kQ + 16 * i + lr) * kQ + 16 * k + 4 * lg) = acc;
}

// ---------------------------------------------------------------------------- sweep

// 16-byte units of a row of LDS are swapped by its number, so that lanes that read a column of rows meet all banks, and
// those that write one do: readers go by bits 0, 1, 3 and 4 of the row, writers by bits 0 to 3.
// (unit ^ number: where unit is 4 kk + lg, the place for kk is that for 0 with the bits of 4 kk turned over; four rows on, bit 2
// is another, and the place is that of kk with its higher bit turned over.)
__device__ __forceinline__ int at_w(int p, int unit) { return p * kQ + ((unit ^ ((p >> 1) & 7)) << 3); }
template <int NP>
__device__ __forceinline__ int at_s(int p, int unit) {
    const int top = (p >> 2 ^ p >> 4) & 1;
    const int h = NP == 128 ? top << 3 | (p >> 3 & 1) << 2 | (p & 3) : top << 2 | (p >> 3 & 1) << 1 | (p >> 1 & 1);
    return p * NP + ((unit ^ h) << 3);
}
__device__ __forceinline__ int at_x(int p, int unit) { return at_s<kQ>(p, unit); }
// kk and k of the place in a row four on from a reader's own
template <int NP>
__device__ __forceinline__ constexpr int turned(int kk, int k) { return 32 * (kk ^ (NP == 128 ? 2 * k : k)); }

template <class T, int NP>
struct SweepLds {
    static constexpr int kStates = NP == 128 ? 1 : 2;       // (two copies of the state's parts where they fit)
    uint16_t xw[2][kParts][kQ * kQ];       // x behind the convolution, weighted for the state: [channel][token]
    float tab[3][kTab<T>];
    uint16_t xt[2][kParts][kQ * kQ];        // x behind the convolution
    uint16_t st[kStates][kParts][kQ * NP];  // the chunk's start state: [channel][state]
    int bad[3];                         // whether a chunk's x has a NaN or infinity
    int first_bad[2][8][kQ];            // and where: [wave][channel] the first such token (64: none)
};
template <class T>
struct StateLds {
    uint16_t xw[2][kParts][kQ * kQ];
    float tab[3][kTab<T>];
};

// PARTS: kParts.  OWN: the segments' own end states, nothing else.  FAST: z and y in 16-byte pieces (headdim a multiple of
// 8).  The chunk's work is one block of code, so that products, LDS and VALU overlap within a wave; what would branch is
// done for nothing instead (channels behind the head's last, tokens behind the sequence's: their weights are zero and
// their outputs are not stored; columns that the filter lacks: branches over them took 147 us instead of 122 on 13
// sequences of 9001 tokens, H12 48x96, fp32, three columns).
template <class T, int NP, int PARTS, bool OWN, bool FAST>
__global__ void __launch_bounds__(kThreads, OWN ? 4 : 2) ssdconv_sweep_kernel(SsdConvArgs a) {
    typedef SweepLds<T, NP> Lds;
    __shared__ __align__(16) typename std::conditional<OWN, StateLds<T>, Lds>::type sm;
    constexpr int kPT = NP == 128 ? 4 : 2;           // 16-channel tiles of a wave's states
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;

    // workgroup -> (segment, head, channels).  The hardware deals workgroups to the 8 XCDs in turn: runs of heads_run heads,
    // which read the same operands of B and C, get one XCD (its L2), and the runs go round, so that each has its share
    // whichever segments are empty
    const int64_t run = blockIdx.x / 8 / a.heads_run * 8 + blockIdx.x % 8;
    const int64_t id = run * a.heads_run + blockIdx.x / 8 % a.heads_run;
    if (id >= a.items * a.H * a.PB) return;
    const int pb = static_cast<int>(id % a.PB), h = static_cast<int>(id / a.PB % a.H);
    const int64_t item = id / a.PB / a.H;
    const int s = find_sequence(a, a.seg_len, item);
    if (s < 0) return;
    const Sequence q(a, s);
    const int64_t seg = item - (q.first / a.seg_len + s);
    if (seg < 0 || (seg * a.seg_len >= q.len && seg > 0)) return;   // (below 0 only where offsets decrease)
    const int begin = static_cast<int>(seg * a.seg_len);
    const bool last = q.len - begin <= a.seg_len;
    if (OWN && last) return;                         // nobody reads its own state
    const int end = last ? q.len : begin + a.seg_len, nch = (end - begin + kQ - 1) / kQ;
    const int g = h / (a.H / a.G);
    const int64_t u0 = q.first / kQ + s + begin / kQ;   // the first chunk's number (seg_len is a multiple of 64)
    const int p0 = pb * kQ, np = a.P - p0 < kQ ? a.P - p0 : kQ;   // channels p0 .. p0 + np - 1 of the head

    // ---- the state: wave wv has states 16 sl + 4 lg + j and channels 16 (pt0 + i) + lr
    const int sl = NP == 128 ? wv : wv & 3, pt0 = NP == 128 ? 0 : wv >> 2 << 1;
    f4 S[kPT];
    {
        const float *from = OWN ? nullptr : a.nseg_split ? a.ws_state + (item * a.H + h) * a.P * a.N
                                : q.old ? a.h + (static_cast<int64_t>(q.slot) * a.H + h) * a.P * a.N : nullptr;
#pragma unroll
        for (int i = 0; i < kPT; ++i) {
            const int p = 16 * (pt0 + i) + lr, n = 16 * sl + 4 * lg;
            const float *row = from + static_cast<int64_t>(p0 + p) * a.N + n;
            S[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            if (!from || p >= np || n >= a.N) continue;
            if (a.h_vec) S[i] = *reinterpret_cast<const f4 *>(row);
            else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N) S[i][j] = row[j];
        }
    }
    auto put_state = [&](int b) __attribute__((always_inline)) {
        if constexpr (!OWN) {
#pragma unroll
            for (int i = 0; i < kPT; ++i) {
                uint32_t w[PARTS][2];
                const float v[4] = {S[i][0], S[i][1], S[i][2], S[i][3]};
                split<PARTS, 4>(v, w);
                const int at = at_s<NP>(16 * (pt0 + i) + lr, 2 * sl + (lg >> 1)) + 4 * (lg & 1);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) *reinterpret_cast<u2 *>(&sm.st[b][k][at]) = u2{w[k][0], w[k][1]};
            }
        }
    };

    // Every operand's pointer is a lane's own and moves by a chunk (scalar bases for all of them spilled).
    // (a value made new where it is used: kept, as the compiler would have it, what follows from it takes registers all loop long)
    auto fresh = [](int v) __attribute__((always_inline)) {
        asm volatile("" : "+v"(v));
        return v;
    };
    // ---- staging: thread (channel lane, tokens 8 wv .. 8 wv + 7)
    const bool mine = lane < np;
    const int channel = h * a.P + p0 + (mine ? lane : 0);
    float fw[4], fbias;
    filter(a, channel, fw, fbias);
    Window<T, 8> win;
    const int row_bytes = static_cast<int>(a.x_row) * static_cast<int>(sizeof(T)), x_at = channel * static_cast<int>(sizeof(T));
    int t_x = begin + 8 * wv;                        // first token of the next chunk to load
    auto load_x = [&]() __attribute__((always_inline)) {
        // (chunks behind the first: three rows are in front; rows behind the sequence's end are out of the buffer and read as
        // zeros, which their weights take out)
        const int t = t_x - 3 < q.len ? t_x - 3 : q.len;
        const int64_t bytes = static_cast<int64_t>(q.len - t) * row_bytes;
        const auto rows = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T *>(static_cast<const T *>(a.xbc) + (q.first + static_cast<int64_t>(t)) * a.x_row), 0,
            static_cast<int>(t == q.len ? 0 : bytes < 0x7fffffff ? bytes - row_bytes + a.C * static_cast<int64_t>(sizeof(T)) : 0x7fffffff), 0x00020000);
#pragma unroll
        for (int i = 0; i < 11; ++i) {
            if constexpr (sizeof(T) == 2) win.x[i] = static_cast<T>(__builtin_amdgcn_raw_buffer_load_b16(rows, x_at, i * row_bytes, 0));
            else win.x[i] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(rows, x_at, i * row_bytes, 0));
        }
        t_x += kQ;
    };
    const float *tab_p = a.ws_tab + (u0 * a.H + h) * kTab<T> + 4 * (threadIdx.x < kTab<T> / 4 ? threadIdx.x : 0);
    f4 tq;
    int tabs = nch;                                  // tables still to load
    auto load_tab = [&]() __attribute__((always_inline)) {
        tq = *reinterpret_cast<const f4 *>(tab_p);
        tab_p += --tabs > 0 ? static_cast<int64_t>(a.H) * kTab<T> : 0;
    };
    auto put_tab = [&](int k3) __attribute__((always_inline)) {
        if (threadIdx.x < kTab<T> / 4) *reinterpret_cast<f4 *>(&sm.tab[k3][4 * threadIdx.x]) = tq;
    };
    auto stage = [&](int c, int k3) __attribute__((always_inline)) {     // (k3: c % 3)
        const int b = c & 1;
        float o[8];
        convolve<true>(win, 0, fw, fbias, 4, o);    // (a column that the filter lacks has weight 0)
        // (the convolution of rows behind the end may be an infinity where no token's is: a weight of zero would not do)
        const int left = q.len - (begin + c * kQ + 8 * wv);
        if (left < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = i < left ? o[i] : 0.0f;
        }
        const f4 w0 = *reinterpret_cast<const f4 *>(&sm.tab[k3][kWr + 8 * wv]);
        const f4 w1 = *reinterpret_cast<const f4 *>(&sm.tab[k3][kWr + 8 * wv + 4]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = o[i] * (i < 4 ? w0[i & 3] : w1[i & 3]);
        s8 part[PARTS];
        split8<PARTS>(v, part);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) *reinterpret_cast<s8 *>(&sm.xw[b][k][at_w(lane, wv)]) = part[k];
        if constexpr (!OWN) {
            s8 y[PARTS];
            split8<PARTS>(o, y);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) *reinterpret_cast<s8 *>(&sm.xt[b][k][at_x(lane, wv)]) = y[k];
            // A NaN or infinity of x must not meet the zeros above the diagonal: it is taken out here, and y gets
            // NaN from its token on (through the state, from the next chunk on, all by itself).  (The sum of eight
            // times zero is not zero where one of them is such a value.)
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) z = __builtin_fmaf(o[i], 0.0f, z);
            int first = kQ;
            if (__any(z != 0.0f)) {
#pragma unroll
                for (int i = 7; i >= 0; --i)
                    if (!(__builtin_fabsf(o[i]) <= 3.4028234663852886e38f)) {
                        first = 8 * wv + i;
                        o[i] = 0.0f;
                    }
                split8<PARTS>(o, y);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) *reinterpret_cast<s8 *>(&sm.xt[b][k][at_x(lane, wv)]) = y[k];
                if (first < kQ) sm.bad[k3] = 1;
            }
            sm.first_bad[b][wv][lane] = first;
        }
    };

    // ---- operands of B (the wave's 16 states)
    s8 bf[2][PARTS];
    const s8 *b_p = reinterpret_cast<const s8 *>(a.ws_bt) + ((u0 * a.G + g) * (NP / 16) + sl) * (2 * PARTS * 64) + lane;
    const int64_t b_step = static_cast<int64_t>(a.G) * (NP / 16 * 2 * PARTS * 64);
    auto load_b = [&](bool more) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) bf[ks][k] = b_p[(ks * PARTS + k) * 64];
        b_p += more ? b_step : 0;
    };

    // ---- outputs: wave (i, ph) has tokens 16 i + lr and, of the channels 32 ph .., 8 lg .. 8 lg + 7
    const int i = wv < 4 ? wv : 7 - wv, ph = wv >> 2;      // (a SIMD's two waves: token blocks of 0 and 3, or of 1 and 2)
    const int t_l = 16 * i + lr, out_p = 32 * ph + 8 * lg;
    const float dsk = a.Dskip ? a.Dskip[h] : 0.0f;
    s8 cf[NP / 32][PARTS];
    const s8 *c_p = reinterpret_cast<const s8 *>(a.ws_c) + ((u0 * a.G + g) * 4 + i) * (NP / 32 * PARTS * 64) + lane;
    const int64_t c_step = static_cast<int64_t>(a.G) * (4 * NP / 32 * PARTS * 64);
    auto load_c = [&](bool more) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < NP / 32; ++kk)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) cf[kk][k] = c_p[(kk * PARTS + k) * 64];
        c_p += more ? c_step : 0;
    };
    // s <= t of the block on the diagonal as all bits or none, and D where s = t, for the lane's eight s
    uint32_t below[8];
    float diag[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = t_l - (32 * (i >> 1) + 8 * lg + e);
        below[e] = static_cast<uint32_t>(~(d >> 31));
        diag[e] = d == 0 ? dsk : 0.0f;
    }
    f4 cb[2][2];
    const float *cb_p = a.ws_cb + ((u0 * a.G + g) * kQ + t_l) * kQ + 8 * lg;
    // cb[0]: C_t . B_s for the token's own half of the chunk (what lies above the diagonal is not used), cb[1]: for the
    // first half
    auto load_cb = [&](bool more) __attribute__((always_inline)) {
        cb[0][0] = *reinterpret_cast<const f4 *>(cb_p + 32 * (i >> 1));
        cb[0][1] = *reinterpret_cast<const f4 *>(cb_p + 32 * (i >> 1) + 4);
        cb[1][0] = *reinterpret_cast<const f4 *>(cb_p);
        cb[1][1] = *reinterpret_cast<const f4 *>(cb_p + 4);
        cb_p += more ? static_cast<int64_t>(a.G) * (kQ * kQ) : 0;
    };
    T zq[8];
    const T *z_p = a.z ? static_cast<const T *>(a.z) + h * a.P + p0 + (out_p < np ? out_p : 0) : nullptr;
    int t_z = begin + t_l;
    auto load_z = [&]() __attribute__((always_inline)) {
        if (!z_p) return;
        const T *z = z_p + (q.first + static_cast<int64_t>(t_z < end ? t_z : end - 1)) * a.z_row;   // (a row that is there)
        t_z += kQ;
        if constexpr (FAST) {
#pragma unroll
            for (int k = 0; k < 8; k += 16 / static_cast<int>(sizeof(T)))
                *reinterpret_cast<u4 *>(zq + k) = *reinterpret_cast<const typename Piece<T>::type *>(z + k);
        } else {
            const int has = fresh(np - out_p);
#pragma unroll
            for (int k = 0; k < 8; ++k) zq[k] = z[k < has ? k : 0];
        }
    };
    // Places of this lane's operands in LDS; within the loop they are made new for each chunk (kept, as the compiler would
    // have it, each of the twenty takes a register, and the registers spill)
    int st_at = at_s<NP>(32 * ph + 8 * (lr >> 2) + (lr & 3), lg), xt_at = at_x(32 * ph + 8 * (lr >> 2) + (lr & 3), lg);
    int xw_at = at_w(16 * pt0 + lr, lg);
    T *y_p = static_cast<T *>(a.y) + ((q.first + static_cast<int64_t>(begin) + t_l) * a.H + h) * a.P + p0 + out_p;
    const int64_t y_step = static_cast<int64_t>(kQ) * a.H * a.P;

    // ---- a chunk's products.  Their LDS operands are requested a group ahead of the instructions that take them; the
    // groups' order is held by ahead() (left to itself the compiler reads two operands, waits, multiplies, and reads on:
    // 306 us against 294 on B4 L4096 H64 64x128, with two parts of y's factors).
    auto ahead = []() __attribute__((always_inline)) { __builtin_amdgcn_sched_barrier(0); };
    constexpr int kKK = NP / 32;
    f4 acc[2];             // outputs: the wave's tokens, 4 lg + j of both tiles
    s8 sf[2][PARTS];       // operands of the carried state, 32 states of a tile and the next ones'.  Row r of tile k is channel
                           // 32 ph + 8 (r / 4) + 4 k + r % 4, so that a lane gets eight channels side by side
    s8 xf[2][PARTS];       // of x
    s8 xw[2][PARTS];       // of x weighted, of 32 tokens for a tile of the state, and the next ones'
    auto read_state = [&](int at, int kk, int k) __attribute__((always_inline)) {
        if constexpr (!OWN) {
#pragma unroll
            for (int e = 0; e < PARTS; ++e) sf[k][e] = *reinterpret_cast<const s8 *>(&sm.st[0][e][0] + ((at ^ turned<NP>(kk, k)) + 4 * NP * k));
        }
    };
    auto read_x = [&](int c, int ks) __attribute__((always_inline)) {
        if constexpr (!OWN) {
            const int at = fresh(xt_at + (c & 1) * (PARTS * kQ * kQ));
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < PARTS; ++e) xf[k][e] = *reinterpret_cast<const s8 *>(&sm.xt[0][e][0] + ((at ^ turned<kQ>(ks, k)) + 4 * kQ * k));
        }
    };
    auto read_w = [&](int at, int j, int ks) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < PARTS; ++k) xw[ks][k] = *reinterpret_cast<const s8 *>(&sm.xw[0][k][0] + ((at ^ 32 * ks) + 16 * kQ * j));
    };
    float whole = 1.0f;      // decay over the segment
    auto products = [&](int c, int k3, bool more2) __attribute__((always_inline)) {
        const float(&tab)[kTab<T>] = sm.tab[k3];
        const T *lows = reinterpret_cast<const T *>(&tab[kLo]);
        const float first = __builtin_amdgcn_exp2f(tab[kC32 + 31]), dec = first * __builtin_amdgcn_exp2f(tab[kC32 + 63]);
        const int w_at = fresh(xw_at + (c & 1) * (PARTS * kQ * kQ));
        if constexpr (OWN) {
            whole *= dec;
            read_w(w_at, 0, 0);
        } else {
            // the carried state's share
            const int at = fresh(st_at + (Lds::kStates == 2 ? c & 1 : 0) * (PARTS * kQ * NP));
            read_state(at, 0, 0);
            const float ct = tab[kC32 + t_l], ct_lo = widen_v(lows[t_l]);
            const int s0 = 32 * (i >> 1) + 8 * lg;
            f4 d0, d1, c0, c1;
            T lo[8];
            acc[0] = acc[1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < kKK; ++kk) {
                read_state(at, kk, 1);
                ahead();
                acc[0] = product<PARTS>(sf[0], cf[kk], acc[0]);
                if (kk + 1 < kKK) read_state(at, kk + 1, 0);
                else {
                    c0 = *reinterpret_cast<const f4 *>(&tab[kC32 + s0]);
                    c1 = *reinterpret_cast<const f4 *>(&tab[kC32 + s0 + 4]);
#pragma unroll
                    for (int q = 0; q < 8; q += 16 / static_cast<int>(sizeof(T)))
                        *reinterpret_cast<u4 *>(lo + q) = *reinterpret_cast<const u4 *>(lows + s0 + q);
                    read_x(c, i >> 1);
                }
                ahead();
                acc[1] = product<PARTS>(sf[1], cf[kk], acc[1]);
            }
            d0 = *reinterpret_cast<const f4 *>(&tab[kDt + s0]);
            d1 = *reinterpret_cast<const f4 *>(&tab[kDt + s0 + 4]);
            read_w(w_at, 0, 0);
            ahead();
            const float et = __builtin_amdgcn_exp2f(ct), e = i < 2 ? et : et * first;
            // the chunk's own share from the token's half of it: (C_t . B_s) decayed, D on the diagonal, times x
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float x = (ct - (q < 4 ? c0[q & 3] : c1[q & 3])) + (ct_lo - widen_v(lo[q]));
                const float f = __builtin_amdgcn_exp2f(x) * (q < 4 ? d0[q & 3] : d1[q & 3]);
                v[q] = __uint_as_float(__float_as_uint(cb[0][q >> 2][q & 3] * f) & below[q]) + diag[q];
            }
            s8 m[PARTS];
            split8<PARTS>(v, m);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                acc[k] *= e;
                acc[k] = product<PARTS>(xf[k], m, acc[k]);
            }
            if (i >= 2) {   // and from the first half, of the second half's tokens
                read_x(c, 0);
                const f4 w0 = *reinterpret_cast<const f4 *>(&tab[kWb + 8 * lg]), w1 = *reinterpret_cast<const f4 *>(&tab[kWb + 8 * lg + 4]);
                ahead();
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = cb[1][q >> 2][q & 3] * (et * (q < 4 ? w0[q & 3] : w1[q & 3]));
                split8<PARTS>(v, m);
#pragma unroll
                for (int k = 0; k < 2; ++k) acc[k] = product<PARTS>(xf[k], m, acc[k]);
            }
            load_c(more2);
            load_cb(more2);
            // x, z and tables of the chunks to come are waited for here, between the products, and not where they are used: 277
            // us against 283 with waits as late as can be (B4 L4096 H64 64x128, two parts of y's factors)
            constexpr int kNewer = kKK * PARTS + 4;                                    // the loads of C and C B^T above
            __builtin_amdgcn_s_waitcnt(0x0f70 | (kNewer & 15) | (kNewer >> 4) << 14);   // vmcnt
            if constexpr (Lds::kStates == 1) __syncthreads();   // the old state's parts are read
        }
        // the state behind the chunk
#pragma unroll
        for (int j = 0; j < kPT; ++j) {
            const bool there = FAST || 16 * (pt0 + j) < np;
            read_w(w_at, j, 1);
            ahead();
            f4 v = S[j] * dec;
            if (there) v = product<PARTS>(bf[0], xw[0], v);
            if (j + 1 < kPT) read_w(w_at, j + 1, 0);
            ahead();
            if (there) S[j] = product<PARTS>(bf[1], xw[1], v);
        }
        load_b(more2);
        put_state(!OWN && Lds::kStates == 2 ? (c & 1) ^ 1 : 0);
    };
    auto store = [&](int c, int k3) __attribute__((always_inline)) {
        if constexpr (!OWN) {
            float y[8] = {acc[0][0], acc[0][1], acc[0][2], acc[0][3], acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
            if (sm.bad[k3]) {
                for (int k = 0; k < 8; ++k)
                    for (int o = 0; o < 8; ++o)
                        if (sm.first_bad[c & 1][o][out_p + k] <= t_l) y[k] = __builtin_nanf("");
            }
            if (z_p) {
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] *= silu_f(widen_v(zq[k]));
            }
            if (begin + c * kQ + t_l < end && out_p < np) {
                if constexpr (FAST) {
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<typename Piece<T>::type *>(y_p) = u4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])};
                    else
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<typename Piece<T>::type *>(y_p + 4 * k) = __builtin_bit_cast(u4, f4{y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]});
                } else {
                    const int has = fresh(np - out_p);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < has) put(y_p, k, y[k]);
                }
            }
            y_p += y_step;
            load_z();
        }
    };

    // Every chunk issues the same loads in the same order, the last ones again where there are no more: a wait for one of
    // them then leaves the later ones in flight.  (Loads in branches were waited for all together, at the top of each chunk.)
    // Of a SIMD's two waves, one stages before a chunk's products, the other behind them, so that VALU and matrix
    // instructions meet: waves 4 to 7 pass the barrier first and stage the chunk after next then, which comes to the same
    // order with one loop.
    const int early = wv >> 2;
    auto next = [&](int c, int k3) __attribute__((always_inline)) {
        if (c < nch) stage(c, k3);
        load_x();
    };
    // The convolution's state, by the sequence's first segment, which alone still reads it: this workgroup's own channels of x,
    // and, one workgroup for each group, those of B and C (read by prep).  A channel a thread; loaded here, stored when all
    // have read the old one.
    const int extra = pb == 0 && h % (a.H / a.G) == 0 ? 2 * a.N : 0, e = static_cast<int>(threadIdx.x) - np;
    const bool keeps = !OWN && seg == 0 && q.slot >= 0 && a.W > 1 && e < extra;
    const int kept = e < 0 ? h * a.P + p0 + e + np : a.H * a.P + (e < a.N ? g * a.N + e : (a.G + g) * a.N + e - a.N);
    T inputs[3];
    if (keeps) last_inputs<T>(a, q, kept, inputs);
    if (nch > 0) {
        win.load(a, q, channel, t_x);
        t_x += kQ;
        load_tab();
        put_tab(0);
        load_tab();
        load_b(nch > 1);
        if constexpr (!OWN) {
            if (threadIdx.x < 3) sm.bad[threadIdx.x] = 0;
            load_c(nch > 1);
            load_cb(nch > 1);
            load_z();
            put_state(0);
        }
        put_tab(1);
        load_tab();
        // (all that is loaded so far is there: else the waits of the loop, which hold for its first round as well, would be for
        // the order of the loads above)
        __builtin_amdgcn_s_waitcnt(0x0f70);     // vmcnt(0)
        __syncthreads();
        if (keeps) keep_inputs<T>(a, q, kept, inputs);
#pragma unroll 1
        for (int c = 0; c <= early; ++c) next(c, c);
        __syncthreads();
        const auto follow = [](int k) { return k == 2 ? 0 : k + 1; };
        int k3 = 0, c = 0;                           // c % 3, c
        do {
            const bool more2 = c + 2 < nch;
            const int n3 = follow(k3), m3 = follow(n3);
            if constexpr (!OWN)
                if (threadIdx.x == 0) sm.bad[m3] = 0;
            products(c, k3, more2);
            store(c, k3);
            put_tab(m3);
            load_tab();
            if (early) __syncthreads();
            next(c + 1 + early, early ? m3 : n3);
            if (!early) __syncthreads();
            k3 = n3;
        } while (++c < nch);
    } else if (keeps) keep_inputs<T>(a, q, kept, inputs);

    // ---- end states
    float *to = OWN ? a.ws_state + (item * a.H + h) * a.P * a.N
              : last && q.slot >= 0 ? a.h + (static_cast<int64_t>(q.slot) * a.H + h) * a.P * a.N : nullptr;
    if (to) {
#pragma unroll
        for (int k = 0; k < kPT; ++k) {
            const int p = 16 * (pt0 + k) + lr;
            const int n = 16 * sl + 4 * lg;
            if (p >= np || n >= a.N) continue;
            float *row = to + static_cast<int64_t>(p0 + p) * a.N + n;
            if (a.h_vec) *reinterpret_cast<f4 *>(row) = S[k];
            else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N) row[j] = S[k][j];
        }
    }
    if constexpr (OWN) {
        if (pb == 0 && threadIdx.x == 0) a.ws_dec[item * a.H + h] = whole;
    }
}

// ---------------------------------------------------------------------------- segments

// The segments' own end states become their start states: per sequence and head, four elements a thread (V; single ones where
// the number of states or the pool's address does not allow it: 11 us instead of 6 on 13 sequences of H12 48x96), eight
// segments' states requested at once.
template <int V>
__global__ void __launch_bounds__(256) ssdconv_join_kernel(SsdConvArgs a) {
    typedef float vec __attribute__((ext_vector_type(V)));
    const int64_t hp = static_cast<int64_t>(a.P) * a.N, e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
    const int h = blockIdx.y, s = blockIdx.z;
    if (e >= hp) return;
    const Sequence q(a, s);
    const int64_t item = q.first / a.seg_len + s, n = q.len > 0 ? (q.len + a.seg_len - 1) / a.seg_len : 1;
    vec v = {};
    if (q.old) v = *reinterpret_cast<const vec *>(a.h + (static_cast<int64_t>(q.slot) * a.H + h) * hp + e);
    float *p = a.ws_state + (item * a.H + h) * hp + e;
    const float *d = a.ws_dec + item * a.H + h;
    constexpr int kAtOnce = 8;
    const int64_t step = a.H * hp;
    for (int64_t k = 0; k < n; k += kAtOnce) {
        vec own[kAtOnce];
        float dec[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {        // (of the last segment nothing is asked)
            own[j] = vec{};
            dec[j] = 0.0f;
            if (k + j + 1 < n) {
                own[j] = *reinterpret_cast<const vec *>(p + j * step);
                dec[j] = d[static_cast<int64_t>(j) * a.H];
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (k + j < n) {
                *reinterpret_cast<vec *>(p + j * step) = v;
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = __builtin_fmaf(dec[j], v[i], own[j][i]);
            }
        p += kAtOnce * step;
        d += kAtOnce * a.H;
    }
}

// ---------------------------------------------------------------------------- one token

// The convolution of one token, all channels, into 32 bits; its state moves on.  (A launch of its own, 3 us for one sequence and 7
// for 128: every head of a group needs its B and C, and no head may read a state that another one has moved on.)
template <class T>
__global__ void __launch_bounds__(256) ssdconv_token_conv_kernel(SsdConvArgs a) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, b = blockIdx.y;
    if (c >= a.C) return;
    int slot = a.slots ? a.slots[b] : static_cast<int>(b);
    if (slot < 0 || slot >= a.nslots) slot = -1;
    const int W1 = a.W - 1;
    T *st = static_cast<T *>(a.conv_state) + (static_cast<int64_t>(slot) * a.C + c) * W1;
    const T x = static_cast<const T *>(a.xbc)[b * a.x_row + c];
    T old[3];
    float v = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < W1) {
            old[k] = slot >= 0 ? st[k] : T{};
            v = __builtin_fmaf(a.w[c * a.W + k], widen_v(old[k]), v);
        }
    v = __builtin_fmaf(a.w[c * a.W + W1], widen_v(x), v);
    a.ws_x[b * a.C + c] = silu_f(v);
    if (slot >= 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < W1) st[k] = k + 1 < W1 ? old[k + 1 < 3 ? k + 1 : 2] : x;
    }
}

// One token of the scan: a workgroup per sequence and head (gridDim.y: shares of its channels).  Rows of N states are read
// by teams of lanes, V states a lane and turn (16 bytes where N and the addresses allow it), four rows at a time, past the caches.
// Memory bound: 8 bytes for every state (B128 H64 64x128: 106 us for 537 MB, 5.1 TB/s, the rate of a large copy).
template <class T, int V>
__global__ void __launch_bounds__(256) ssdconv_token_kernel(SsdConvArgs a) {
    const int64_t id = blockIdx.x;
    const int h = static_cast<int>(id % a.H);
    const int64_t b = id / a.H;
    int slot = a.slots ? a.slots[b] : static_cast<int>(b);
    if (slot < 0 || slot >= a.nslots) slot = -1;
    const int team = a.team, lane = threadIdx.x & (team - 1), me = threadIdx.x / team, teams = 256 / team;
    constexpr int kU = V == 4 ? 1 : 2;               // 128 states: 32 lanes of four, or 64 lanes of two single ones
    constexpr int kR = 4;
    float dt = widen_v(static_cast<const T *>(a.delta)[b * a.d_row + h]);
    if (a.dbias) dt += a.dbias[h];
    if (a.softplus) dt = softplus_f(dt);
    const float dec = __builtin_amdgcn_exp2f(dt * (a.A[h] * kLog2e)), dsk = a.Dskip ? a.Dskip[h] : 0.0f;
    const float *xs = a.ws_x + b * a.C, *X = xs + static_cast<int64_t>(h) * a.P;
    const int g = h / (a.H / a.G);
    const float *Bv = xs + static_cast<int64_t>(a.H) * a.P + g * a.N, *Cv = Bv + a.G * a.N;
    float bv[kU][V], cv[kU][V];
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int n = (lane + k * team) * V + j;
            bv[k][j] = n < a.N ? dt * Bv[n] : 0.0f;
            cv[k][j] = n < a.N ? Cv[n] : 0.0f;
        }
    float *hs = a.h + (static_cast<int64_t>(slot < 0 ? 0 : slot) * a.H + h) * a.P * a.N;
    const int share = (a.P + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
    const int pa = static_cast<int>(blockIdx.y) * share, pe = pa + share < a.P ? pa + share : a.P;
    for (int p0 = pa + me; p0 < pe; p0 += kR * teams) {
        float st[kR][kU][V];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int p = p0 + r * teams;
            const float *row = hs + static_cast<int64_t>(p) * a.N;
#pragma unroll
            for (int k = 0; k < kU; ++k) {
                const int n = (lane + k * team) * V;
                const bool in = slot >= 0 && p < pe && n < a.N;
                if constexpr (V == 4) {
                    const f4 v = in ? __builtin_nontemporal_load(reinterpret_cast<const f4 *>(row + n)) : f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 4; ++j) st[r][k][j] = v[j];
                } else st[r][k][0] = in ? row[n] : 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int p = p0 + r * teams;
            const float x = X[p < pe ? p : pe - 1];
            float y = 0.0f;
#pragma unroll
            for (int k = 0; k < kU; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    st[r][k][j] = __builtin_fmaf(dec, st[r][k][j], bv[k][j] * x);
                    y = __builtin_fmaf(cv[k][j], st[r][k][j], y);
                }
            for (int o = team >> 1; o > 0; o >>= 1) y += __shfl_xor(y, o, 64);
            if (p >= pe) continue;
            float *row = hs + static_cast<int64_t>(p) * a.N;
#pragma unroll
            for (int k = 0; k < kU; ++k) {
                const int n = (lane + k * team) * V;
                if (slot < 0 || n >= a.N) continue;
                if constexpr (V == 4)
                    __builtin_nontemporal_store(f4{st[r][k][0], st[r][k][1], st[r][k][2], st[r][k][3]}, reinterpret_cast<f4 *>(row + n));
                else row[n] = st[r][k][0];
            }
            if (lane == 0) {
                float v = __builtin_fmaf(dsk, x, y);
                if (a.z) v *= silu_f(widen(static_cast<const T *>(a.z), b * a.z_row + static_cast<int64_t>(h) * a.P + p));
                put(static_cast<T *>(a.y), (b * a.H + h) * a.P + p, v);
            }
        }
    }
}

template <class T, int NP>
hipError_t prompts(const SsdConvArgs &a, hipStream_t s) {
    const unsigned heads = static_cast<unsigned>((a.H + 63) / 64);
    hipLaunchKernelGGL((ssdconv_prep_kernel<T, NP>), dim3(static_cast<unsigned>(a.chunks), static_cast<unsigned>(a.G) + heads),
                       dim3(kPrepThreads), 0, s, a);
    hipError_t e = launch_status(s);
    if (e != hipSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.items * a.H * a.PB / a.heads_run + 7) / 8 * 8 * a.heads_run));
    if (a.nseg_split) {
        hipLaunchKernelGGL((ssdconv_sweep_kernel<T, NP, kParts, true, true>), grid, dim3(kThreads), 0, s, a);
        e = launch_status(s);
        if (e != hipSuccess) return e;
        const int wide = a.h_vec ? 4 : 1;
        const dim3 each(static_cast<unsigned>((static_cast<int64_t>(a.P) * a.N / wide + 255) / 256), static_cast<unsigned>(a.H), static_cast<unsigned>(a.S));
        if (a.h_vec) hipLaunchKernelGGL(ssdconv_join_kernel<4>, each, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(ssdconv_join_kernel<1>, each, dim3(256), 0, s, a);
        e = launch_status(s);
        if (e != hipSuccess) return e;
    }
    if (a.P % 8 == 0) hipLaunchKernelGGL((ssdconv_sweep_kernel<T, NP, kParts, false, true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((ssdconv_sweep_kernel<T, NP, kParts, false, false>), grid, dim3(kThreads), 0, s, a);
    return launch_status(s);
}

template <class T>
hipError_t token(const SsdConvArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((ssdconv_token_conv_kernel<T>), dim3(static_cast<unsigned>((a.C + 255) / 256), static_cast<unsigned>(a.S)),
                       dim3(256), 0, s, a);
    hipError_t e = launch_status(s);
    if (e != hipSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.S * a.H), static_cast<unsigned>(a.shares));
    if (a.h_vec) hipLaunchKernelGGL((ssdconv_token_kernel<T, 4>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((ssdconv_token_kernel<T, 1>), grid, dim3(256), 0, s, a);
    return launch_status(s);
}

}  // namespace

hipError_t launch_ssdconv(const SsdConvArgs &a, bool bf16, hipStream_t s) {
    if (bf16) return a.N > 64 ? prompts<uint16_t, 128>(a, s) : prompts<uint16_t, 64>(a, s);
    return a.N > 64 ? prompts<float, 128>(a, s) : prompts<float, 64>(a, s);
}

hipError_t launch_ssdconv_token(const SsdConvArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? token<uint16_t>(a, s) : token<float>(a, s);
}

}  // namespace ssm
