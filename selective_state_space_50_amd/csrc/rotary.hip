// Rotary positions of queries and keys, by themselves or behind an RMS norm of every head.
//
// Per token t and head row x [dim], with the angle th_j = position[t] freqs[j] of pair j < rot / 2:
//     u = x                                   or, normed, u = x rstd w,  rstd = 1 / sqrt(mean(x^2) + eps)
//     (y_a, y_b) = m (u_a cos th - u_b sin th, u_b cos th + u_a sin th)    a, b the columns of pair j
//     y_c = u_c                               for the columns behind the first rot
// The turn R is m times an orthogonal map, so its gradient is the turn by the opposite angle:
// g = R^T dy (dx of the plain form); normed, with xh = x rstd and e = g w,
//     dw = sum over tokens and heads of g xh,   dx = rstd (e - xh mean(e xh)).
//
// Memory bound: q and k are read and written once (backward: two reads, one write): 336 MB of B4 L4096 32+8 heads of 128
// bf16 in 50 us, the training pass of B2 L4096 32+32 heads, 671 MB, in 43 + 81 + 4; fp32, B4 L2048 32+8 heads, 336 MB, in
// 50, normed 57.  A workgroup takes a few tokens: its threads make their cosines and sines once, in LDS, for all heads of q
// and k (an angle is position * frequency in 64 bits, cut to a part of a turn there, and only then 32 bits, with the rest kept: at
// position 10^6 a 32-bit product would be off by 0.06 rad).  Then teams of lanes take the tokens' heads row by row.  A lane
// holds a unit of 2 V columns: the V of one side of V pairs and the V of their other side (half layout), or 2 V side
// by side (interleaved, and columns that do not turn), so that pairs never cross lanes and loads stay vectors.
// 16-byte loads where the sizes and addresses allow them (V = 8 bf16, 4 fp32), else 8-byte ones (bf16), else
// single elements.  Rows are requested kRows at a time.
#include "ssm_device.h"

#include <type_traits>

namespace ssm {
namespace {

constexpr int kWG = 256;
constexpr int kRows = 4;    // rows of a team in flight

template <class T, int V>
struct Raw;                 // V elements of type T as they lie in memory
template <> struct Raw<uint16_t, 8> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <> struct Raw<uint16_t, 4> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Raw<uint16_t, 1> { typedef uint16_t type; };
template <> struct Raw<float, 4> { typedef float type __attribute__((ext_vector_type(4))); };
template <> struct Raw<float, 1> { typedef float type; };

template <class T, int V>
__device__ __forceinline__ typename Raw<T, V>::type fetch(const T *p) {
    return *reinterpret_cast<const typename Raw<T, V>::type *>(p);
}
template <class T, int V>
__device__ __forceinline__ void open(typename Raw<T, V>::type r, float *v) {
    if constexpr (V == 1) v[0] = widen_v(r);
    else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) { v[2 * i] = bf_lo(r[i]); v[2 * i + 1] = bf_hi(r[i]); }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = r[i];
    }
}
// Outputs are rounded once, to nearest even, and stored past the caches: they are written once (the 168 MB of B4 L4096 32+8
// heads of 128 bf16 57 -> 50 us, the training pass of B2 L4096 32+32 heads 144 -> 128; loads past them 10 us slower).
template <class T, int V>
__device__ __forceinline__ void keep(T *p, const float *v) {
    if constexpr (V == 1) put(p, 0, v[0]);
    else {
        typename Raw<T, V>::type r;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = v[i];
        }
        __builtin_nontemporal_store(r, reinterpret_cast<typename Raw<T, V>::type *>(p));
    }
}

// the unit's pairs turned by (cos, sin) = cs[0 .. V - 1]; back: by the opposite angles
template <int V, bool INTER>
__device__ __forceinline__ void turn(float *a, float *b, const float2 *cs, bool back) {
    float c[V], s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[i] = cs[i].x;
        s[i] = back ? -cs[i].y : cs[i].y;
    }
    if constexpr (INTER && V > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float *side = i < V / 2 ? a : b;
            const int k = 2 * (i % (V / 2));
            const float u = side[k], v = side[k + 1];
            side[k] = __builtin_fmaf(u, c[i], -v * s[i]);
            side[k + 1] = __builtin_fmaf(v, c[i], u * s[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = a[i], v = b[i];
            a[i] = __builtin_fmaf(u, c[i], -v * s[i]);
            b[i] = __builtin_fmaf(v, c[i], u * s[i]);
        }
    }
}

__device__ __forceinline__ float team_sum(float v, int team) {
    for (int o = team >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// cosines and sines of the tokens t0 .. t0 + n - 1, times the magnitude, into cs[token][pair]
__device__ __forceinline__ void angles(const RotaryArgs &a, int64_t t0, int n, float2 *cs) {
    for (int i = threadIdx.x; i < n * a.pairs; i += kWG) {
        const int k = static_cast<int>(static_cast<uint64_t>(i) * a.by_pairs >> 32), j = i - k * a.pairs;
        const int64_t t = t0 + k;
        const int p = a.positions[a.period ? t % a.period : t];
        const double turns = static_cast<double>(p) * (a.freqs[j] * 0.15915494309189533577);   // 1 / (2 pi)
        // (what rounding the part of a turn to 32 bits takes, up to 2^-26 of one, turns cosine and sine once more: 1 and d)
        const double part = turns - rint(turns);
        const float near = static_cast<float>(part), d = 6.2831853f * static_cast<float>(part - static_cast<double>(near));
        float sn, cn;
        sincospif(2.0f * near, &sn, &cn);
        cs[i] = make_float2(a.magnitude * __builtin_fmaf(-d, sn, cn), a.magnitude * __builtin_fmaf(d, cn, sn));
    }
}

// Where a lane's units lie in a row: offsets of their two sides, and which pairs they turn by (-1: none).
template <int V, int UL, bool INTER>
struct Units {
    int oa[UL], ob[UL], pair[UL];
    bool a_in[UL], b_in[UL];
    __device__ Units(const RotaryArgs &a, int lane) {
#pragma unroll
        for (int i = 0; i < UL; ++i) {
            const int u = lane + i * a.team;
            const bool turns = u * V < a.pairs;
            oa[i] = turns && !INTER ? V * u : 2 * V * u;
            ob[i] = turns && !INTER ? a.pairs + V * u : 2 * V * u + V;
            pair[i] = turns ? V * u : -1;
            a_in[i] = oa[i] < a.dim;
            b_in[i] = ob[i] < a.dim;   // (single elements: an odd dim's last unit has one side only)
            if (!a_in[i]) oa[i] = 0;   // (what is not there counts as zeros, with the first columns' weights)
            if (!b_in[i]) ob[i] = 0;
        }
    }
};

// where row i (of n tokens from t0) starts in q or k, and in their contiguous counterparts
struct RowAt {
    int token;        // of the workgroup's
    bool is_q;
    int64_t in, out;  // elements from the tensor's start
    __device__ RowAt(const RotaryArgs &a, int64_t t0, int i) {
        token = static_cast<int>(static_cast<uint64_t>(i) * a.by_heads >> 32);
        const int h = i - token * a.heads;
        is_q = h < a.q_heads;
        const int64_t t = t0 + token;
        in = is_q ? t * a.q_row + h * a.dim : t * a.k_row + (h - a.q_heads) * a.dim;
        out = is_q ? (t * a.q_heads + h) * a.dim : (t * (a.heads - a.q_heads) + h - a.q_heads) * a.dim;
    }
};

template <class T, int V, int UL, bool INTER, bool NORM>
__global__ void __launch_bounds__(kWG) rotary_kernel(RotaryArgs a) {
    extern __shared__ __align__(16) float lds[];
    float *w = lds;                                     // [2][dim]: of q, of k
    float2 *cs = reinterpret_cast<float2 *>(lds + (NORM ? 2 * a.dim_even : 0));
    typedef typename Raw<T, V>::type raw_t;
    const int lane = threadIdx.x & (a.team - 1), teams = kWG / a.team;
    const int me = threadIdx.x / a.team;
    const Units<V, UL, INTER> un(a, lane);
    if constexpr (NORM) {
        for (int i = threadIdx.x; i < a.dim; i += kWG) {
            w[i] = a.wq ? a.wq[i] : 1.0f;
            w[a.dim_even + i] = a.wk ? a.wk[i] : 1.0f;
        }
    }
    for (int64_t g = blockIdx.x; g < a.groups; g += gridDim.x) {
        const int64_t t0 = g * a.tokens_per;
        const int n = static_cast<int>(a.tokens - t0 < a.tokens_per ? a.tokens - t0 : a.tokens_per);
        const int rows = n * a.heads;
        angles(a, t0, n, cs);
        __syncthreads();
        for (int i0 = me; i0 < rows; i0 += kRows * teams) {
            raw_t ra[kRows][UL], rb[kRows][UL];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int i = i0 + r * teams;
                const RowAt at(a, t0, i < rows ? i : rows - 1);     // (past the end: a row that is there)
                const T *x = static_cast<const T *>(at.is_q ? a.q : a.k) + at.in;
#pragma unroll
                for (int j = 0; j < UL; ++j) {
                    ra[r][j] = un.a_in[j] ? fetch<T, V>(x + un.oa[j]) : raw_t{};
                    rb[r][j] = un.b_in[j] ? fetch<T, V>(x + un.ob[j]) : raw_t{};
                }
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int i = i0 + r * teams;
                const RowAt at(a, t0, i < rows ? i : rows - 1);
                T *y = static_cast<T *>(at.is_q ? a.q_out : a.k_out) + at.out;
                float xa[UL][V], xb[UL][V];
#pragma unroll
                for (int j = 0; j < UL; ++j) {
                    open<T, V>(ra[r][j], xa[j]);
                    open<T, V>(rb[r][j], xb[j]);
                }
                if constexpr (NORM) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < UL; ++j)
#pragma unroll
                        for (int e = 0; e < V; ++e) ss = __builtin_fmaf(xa[j][e], xa[j][e], __builtin_fmaf(xb[j][e], xb[j][e], ss));
                    ss = team_sum(ss, a.team);
                    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, a.inv_dim, a.eps));
                    const float *wr = w + (at.is_q ? 0 : a.dim_even);
#pragma unroll
                    for (int j = 0; j < UL; ++j)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            xa[j][e] *= rstd * wr[un.oa[j] + e];
                            xb[j][e] *= rstd * wr[un.ob[j] + e];
                        }
                }
                if (i >= rows) continue;
#pragma unroll
                for (int j = 0; j < UL; ++j) {
                    if (un.pair[j] >= 0) turn<V, INTER>(xa[j], xb[j], cs + at.token * a.pairs + un.pair[j], a.back);
                    if (un.a_in[j]) keep<T, V>(y + un.oa[j], xa[j]);
                    if (un.b_in[j]) keep<T, V>(y + un.ob[j], xb[j]);
                }
            }
        }
        __syncthreads();   // the angles are read
    }
}

// The normed form's gradients.  Each lane keeps its columns' sums of dw over all its rows, q's and k's apart; the
// teams' sums are added in LDS in their order, the workgroups' by column_sum_kernel in theirs.
template <class T, int V, int UL, bool INTER>
__global__ void __launch_bounds__(kWG) qknorm_bwd_kernel(RotaryArgs a) {
    extern __shared__ __align__(16) float lds[];
    float *w = lds;
    float2 *cs = reinterpret_cast<float2 *>(lds + 2 * a.dim_even);
    typedef typename Raw<T, V>::type raw_t;
    constexpr int kAhead = 2;
    const int lane = threadIdx.x & (a.team - 1), teams = kWG / a.team;
    const int me = threadIdx.x / a.team;
    const Units<V, UL, INTER> un(a, lane);
    for (int i = threadIdx.x; i < a.dim; i += kWG) {
        w[i] = a.wq ? a.wq[i] : 1.0f;
        w[a.dim_even + i] = a.wk ? a.wk[i] : 1.0f;
    }
    float dw[2][UL][2][V] = {};
    for (int64_t g = blockIdx.x; g < a.groups; g += gridDim.x) {
        const int64_t t0 = g * a.tokens_per;
        const int n = static_cast<int>(a.tokens - t0 < a.tokens_per ? a.tokens - t0 : a.tokens_per);
        const int rows = n * a.heads;
        angles(a, t0, n, cs);
        __syncthreads();
        for (int i0 = me; i0 < rows; i0 += kAhead * teams) {
            raw_t ra[kAhead][UL], rb[kAhead][UL], da[kAhead][UL], db[kAhead][UL];
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int i = i0 + r * teams;
                const RowAt at(a, t0, i < rows ? i : rows - 1);
                const T *x = static_cast<const T *>(at.is_q ? a.q : a.k) + at.in;
                const T *dy = static_cast<const T *>(at.is_q ? a.dq_out : a.dk_out) + at.out;
#pragma unroll
                for (int j = 0; j < UL; ++j) {
                    ra[r][j] = un.a_in[j] ? fetch<T, V>(x + un.oa[j]) : raw_t{};
                    rb[r][j] = un.b_in[j] ? fetch<T, V>(x + un.ob[j]) : raw_t{};
                    da[r][j] = un.a_in[j] ? fetch<T, V>(dy + un.oa[j]) : raw_t{};
                    db[r][j] = un.b_in[j] ? fetch<T, V>(dy + un.ob[j]) : raw_t{};
                }
            }
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int i = i0 + r * teams;
                const RowAt at(a, t0, i < rows ? i : rows - 1);
                float xa[UL][V], xb[UL][V], ga[UL][V], gb[UL][V];
                const float *wr = w + (at.is_q ? 0 : a.dim_even);
                float wa[UL][V], wb[UL][V], ss = 0.0f, ex = 0.0f;
#pragma unroll
                for (int j = 0; j < UL; ++j) {
                    open<T, V>(ra[r][j], xa[j]);
                    open<T, V>(rb[r][j], xb[j]);
                    open<T, V>(da[r][j], ga[j]);
                    open<T, V>(db[r][j], gb[j]);
                    if (un.pair[j] >= 0) turn<V, INTER>(ga[j], gb[j], cs + at.token * a.pairs + un.pair[j], true);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        wa[j][e] = wr[un.oa[j] + e];
                        wb[j][e] = wr[un.ob[j] + e];
                        ss = __builtin_fmaf(xa[j][e], xa[j][e], __builtin_fmaf(xb[j][e], xb[j][e], ss));
                        ex = __builtin_fmaf(ga[j][e] * wa[j][e], xa[j][e], __builtin_fmaf(gb[j][e] * wb[j][e], xb[j][e], ex));
                    }
                }
                ss = team_sum(ss, a.team);
                ex = team_sum(ex, a.team);
                if (i >= rows) continue;
                const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, a.inv_dim, a.eps));
                const float c = rstd * (rstd * (ex * a.inv_dim));           // dx = rstd e - c xh (rstd^3 could be infinite)
                T *dx = static_cast<T *>(at.is_q ? a.q_out : a.k_out) + at.out;
#pragma unroll
                for (int j = 0; j < UL; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        xa[j][e] *= rstd;
                        xb[j][e] *= rstd;
                    }
                auto sums = [&](float (&d)[UL][2][V]) __attribute__((always_inline)) {
#pragma unroll
                    for (int j = 0; j < UL; ++j)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            d[j][0][e] = __builtin_fmaf(ga[j][e], xa[j][e], d[j][0][e]);
                            d[j][1][e] = __builtin_fmaf(gb[j][e], xb[j][e], d[j][1][e]);
                        }
                };
                if (at.is_q) sums(dw[0]);
                else sums(dw[1]);
#pragma unroll
                for (int j = 0; j < UL; ++j) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        ga[j][e] = __builtin_fmaf(ga[j][e] * rstd, wa[j][e], -c * xa[j][e]);
                        gb[j][e] = __builtin_fmaf(gb[j][e] * rstd, wb[j][e], -c * xb[j][e]);
                    }
                    if (un.a_in[j]) keep<T, V>(dx + un.oa[j], ga[j]);
                    if (un.b_in[j]) keep<T, V>(dx + un.ob[j], gb[j]);
                }
            }
        }
        __syncthreads();
    }
    if (!a.part) return;
    // [team][2 dim] over the weights and angles (the last barrier passed)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < UL; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float *to = lds + (2 * me + k) * a.dim;
                if (un.a_in[j]) to[un.oa[j] + e] = dw[k][j][0][e];
                if (un.b_in[j]) to[un.ob[j] + e] = dw[k][j][1][e];
            }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.dim; c += kWG) {
        double s[4] = {};        // (at least four teams; chains a quarter as long)
        for (int t = 0; t < teams; t += 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += lds[2 * (t + i) * a.dim + c];
        a.part[static_cast<int64_t>(blockIdx.x) * 2 * a.dim + c] = static_cast<float>((s[0] + s[1]) + (s[2] + s[3]));
    }
}

// v[0] = the sum of v[0 .. N - 1], by halves
template <int N>
__device__ __forceinline__ void by_halves(double *v) {
#pragma unroll
    for (int o = N / 2; o > 0; o /= 2)
#pragma unroll
        for (int i = 0; i < o; ++i) v[i] += v[i + o];
}

// dw[c] = the sum of part[row][c] over the rows (1024 at most), eight columns a workgroup: 128 sums of every 128th row, then
// those, in two steps, all by halves and in 64 bits (a tree of 32-bit sums was 0.4e-7 of the result worse; 4 us, most of it waiting)
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *part, int rows, int dim, float *dwq, float *dwk) {
    __shared__ double s[128][9];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3, c = blockIdx.x * 8 + x;
    double v[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c < 2 * dim && y + 128 * k < rows ? part[static_cast<int64_t>(y + 128 * k) * 2 * dim + c] : 0.0;
    by_halves<8>(v);
    s[y][x] = v[0];
    __syncthreads();
    if (y < 8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = s[16 * y + i][x];
        by_halves<16>(v);
    }
    __syncthreads();
    if (y < 8) s[y][x] = v[0];
    __syncthreads();
    if (y || c >= 2 * dim) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s[i][x];
    by_halves<8>(v);
    if (c < dim) { if (dwq) dwq[c] = static_cast<float>(v[0]); }
    else if (dwk) dwk[c - dim] = static_cast<float>(v[0]);
}

template <class T, int V, int UL, bool INTER>
hipError_t typed(const RotaryArgs &a, bool norm, bool bwd, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.blocks));
    size_t lds = static_cast<size_t>(a.tokens_per) * a.pairs * sizeof(float2) + (norm ? 2 * a.dim_even * sizeof(float) : 0);
    if (!bwd) {
        if (norm) hipLaunchKernelGGL((rotary_kernel<T, V, UL, INTER, true>), grid, dim3(kWG), lds, s, a);
        else hipLaunchKernelGGL((rotary_kernel<T, V, UL, INTER, false>), grid, dim3(kWG), lds, s, a);
        return launch_status(s);
    }
    const size_t sums = static_cast<size_t>(kWG / a.team) * 2 * a.dim * sizeof(float);
    if (a.part && sums > lds) lds = sums;
    hipLaunchKernelGGL((qknorm_bwd_kernel<T, V, UL, INTER>), grid, dim3(kWG), lds, s, a);
    hipError_t e = launch_status(s);
    if (e != hipSuccess || !a.part) return e;
    hipLaunchKernelGGL(column_sum_kernel, dim3(static_cast<unsigned>((2 * a.dim + 7) / 8)), dim3(1024), 0, s, a.part,
                       static_cast<int>(a.blocks), a.dim, a.dwq, a.dwk);
    return launch_status(s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, bool bf16, int vec, bool inter, bool norm, bool bwd, hipStream_t s) {
    if (vec == 1) {
        const bool two = a.units > a.team;
        if (bf16) {
            if (inter) return two ? typed<uint16_t, 1, 2, true>(a, norm, bwd, s) : typed<uint16_t, 1, 1, true>(a, norm, bwd, s);
            return two ? typed<uint16_t, 1, 2, false>(a, norm, bwd, s) : typed<uint16_t, 1, 1, false>(a, norm, bwd, s);
        }
        if (inter) return two ? typed<float, 1, 2, true>(a, norm, bwd, s) : typed<float, 1, 1, true>(a, norm, bwd, s);
        return two ? typed<float, 1, 2, false>(a, norm, bwd, s) : typed<float, 1, 1, false>(a, norm, bwd, s);
    }
    if (!bf16) return inter ? typed<float, 4, 1, true>(a, norm, bwd, s) : typed<float, 4, 1, false>(a, norm, bwd, s);
    if (vec == 8) return inter ? typed<uint16_t, 8, 1, true>(a, norm, bwd, s) : typed<uint16_t, 8, 1, false>(a, norm, bwd, s);
    return inter ? typed<uint16_t, 4, 1, true>(a, norm, bwd, s) : typed<uint16_t, 4, 1, false>(a, norm, bwd, s);
}

}  // namespace ssm
