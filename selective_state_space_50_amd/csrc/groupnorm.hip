// Group norm, channels last, with an activation or a gate; forward and backward.
//
// x [N, L, C], the channels in G groups of S = C / G; one mean and variance for every (n, g),
// over its M = L S values (L = 1: the norm of single tokens):
//     xh = (x - mean) / sqrt(var + eps),   u = xh w_c + b_c,   y = act(u) silu(z)
// with act the identity or silu, and w, b, z optional.  Backward, with
//     g = dy silu(z) act'(u),   e = g w_c:
//     dz = dy act(u) silu'(z),  db_c = sum g,  dw_c = sum g xh,
//     dx = rstd (e - (sum_M e + xh sum_M e xh) / M)
//
// The work is bound by memory: a few operations per element.  Every value is read once where
// the M values of a group fit the registers of a team of lanes (a part of a wave, a wave, or a
// workgroup): mean first, then the sum of squared deviations from it.  Larger groups are cut
// into slabs of rows: a pass for the statistics (deviations from running means, merged in a
// fixed order), then a pass that reads x again.  Their backward sums g and g xh per channel,
// which gives dw and db and, weighted with w, both sums of dx.  Over few positions (or with more rows of
// statistics than a launch has slabs for) the backward walks every group by a team of lanes instead.
//
// All sums are in fp32, in lanes of a few hundred terms and trees of them.  (3x1001x330 in 10 groups, fp32, forward and
// backward: every output within 1.5e-7 of exact in norm; with dw and db summed in 64 bits, in torch, 1.0e-7.)
//
// Measured, bf16 (a copy reaches 5.2 TB/s): 16384 rows of 4096 channels in 64 groups, gated: forward 91 us
// (4.4 TB/s), backward 132 us (5.1 TB/s) and 6 us for the sums of dw and db.  8 x 4000 x 512 in 32 groups
// over whole sequences: statistics 8 us (4.1 TB/s), 5 us for their merging, y 16 us (4.1 TB/s of
// reads and writes).  A group of 128 KB held by one workgroup instead: 25.3 us against 28.5 in all, but
// 17.6 against 14.8 with a quarter as many groups and 84 against 75 with four times as many.
#include "ssm_device.h"

#include <type_traits>

namespace ssm {
namespace {

constexpr int kWG = 256;
typedef float f4 __attribute__((ext_vector_type(4)));

// VE consecutive elements of type T as fp32
template <class T, int VE>
struct Vec {
    float v[VE];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VE == 1) v[0] = widen_v(p[0]);
        else if constexpr (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[2 * i] = bf_lo(r[i]); v[2 * i + 1] = bf_hi(r[i]); }
        } else {
            const f4 u = *reinterpret_cast<const f4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = u[i];
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VE == 1) put(p, 0, v[0]);
        else if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        else *reinterpret_cast<f4 *>(p) = f4{v[0], v[1], v[2], v[3]};
    }
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = x;
    }
};

// VE consecutive channels of w or b (aligned as x's), or a constant where there is none
template <int VE>
__device__ __forceinline__ void channels(const float *p, int64_t c, float none, float (&v)[VE]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = none;
    } else if constexpr (VE == 1) v[0] = p[c];
    else {
#pragma unroll
        for (int k = 0; k < VE / 4; ++k) {
            const f4 u = *reinterpret_cast<const f4 *>(p + c + 4 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * k + i] = u[i];
        }
    }
}

// (hardware exp2 and reciprocal, a step of fp32 each: SiLU and its gradient are within a few steps of exact, below the
// sums' own roundings)
__device__ __forceinline__ float sigmoid_f(float u) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u * kLog2e)); }

__device__ __forceinline__ float norm_out(float xh, float w, float b, bool silu, bool gate, float z) {
    float y = __builtin_fmaf(xh, w, b);
    if (silu) y *= sigmoid_f(y);
    if (gate) y *= z * sigmoid_f(z);
    return y;
}
// g = dLoss/du, and dz
__device__ __forceinline__ float norm_grad(float xh, float w, float b, bool silu, bool gate, float z, float dy, float &dz) {
    const float u = __builtin_fmaf(xh, w, b);
    float a = u, g = dy;
    float su = 0.0f;
    if (silu) { su = sigmoid_f(u); a = u * su; }
    if (gate) {
        const float sz = sigmoid_f(z);
        dz = dy * a * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f);
        g = dy * (z * sz);
    }
    if (silu) g *= su * __builtin_fmaf(u, 1.0f - su, 1.0f);
    return g;
}

// sum over a team of P lanes (a power of two up to 64) or (WG) over the workgroup, in a fixed order
template <bool WG>
__device__ __forceinline__ float team_sum(float v, int P, float *lds) {
    if constexpr (WG) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
        __syncthreads();   // lds may still be read from the sum before
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        return (lds[0] + lds[1]) + (lds[2] + lds[3]);
    } else {
        for (int o = P >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
        return v;
    }
}

// ---- groups that fit a team's registers: lane t of the team holds the vectors t, t + P, ...  (Teams that
// walk rows and keep w and b, two rows at a time, were no faster: 95 us before the divisions went, as this was.)
// (ONE: L = 1, no division for the place of a vector)
template <class T, int VE, int MAXV, bool WG, bool ONE>
__global__ void __launch_bounds__(kWG) gn_team_kernel(GroupNormArgs a) {
    __shared__ float lds[4];
    const int P = WG ? kWG : a.team, sh = __builtin_ctz(P), tl = threadIdx.x & (P - 1);   // (a power of two)
    const uint32_t team = (blockIdx.y * gridDim.x + blockIdx.x) * (kWG >> sh) + (threadIdx.x >> sh);
    const bool on = team < static_cast<uint32_t>(a.N * a.G);
    const uint32_t G = static_cast<uint32_t>(a.G), n = (on ? team : 0) / G, g = (on ? team : 0) % G;
    const uint32_t nvec = static_cast<uint32_t>(a.nvec), lpg = static_cast<uint32_t>(a.S / VE);
    const int64_t base = static_cast<int64_t>(n) * a.L * a.C + static_cast<int64_t>(g) * a.S;
    const T *x = static_cast<const T *>(a.x) + base;
    Vec<T, VE> v[MAXV], z[MAXV];
    uint32_t off[MAXV], ch[MAXV];   // (M and so every offset fits 32 bits: the planner's bound)
    bool in[MAXV];
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
        const uint32_t e = tl + i * P, l = ONE ? 0 : e / lpg, j = ONE ? e : e % lpg;
        in[i] = on && e < nvec;
        ch[i] = j * VE;
        off[i] = in[i] ? l * static_cast<uint32_t>(a.C) + ch[i] : 0;
        v[i].fill(0.0f);
        if (in[i]) v[i].load(x + off[i]);
    }
    if (a.z)
#pragma unroll
        for (int i = 0; i < MAXV; ++i)
            if (in[i]) z[i].load(static_cast<const T *>(a.z) + base + off[i]);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
#pragma unroll
        for (int k = 0; k < VE; ++k) s += v[i].v[k];
    const float inv_m = a.inv_m;
    const float mean = team_sum<WG>(s, P, lds) * inv_m;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
        if (in[i])
#pragma unroll
            for (int k = 0; k < VE; ++k) { const float d = v[i].v[k] - mean; s = __builtin_fmaf(d, d, s); }
    const float rstd = 1.0f / sqrtf(team_sum<WG>(s, P, lds) * inv_m + a.eps);
    if (on && tl == 0) {
        if (a.mean) a.mean[team] = mean;
        if (a.rstd) a.rstd[team] = rstd;
    }
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
        if (in[i]) {
            float w[VE], b[VE];
            channels<VE>(a.w, static_cast<int64_t>(g) * a.S + ch[i], 1.0f, w);
            channels<VE>(a.b, static_cast<int64_t>(g) * a.S + ch[i], 0.0f, b);
            Vec<T, VE> y;
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y.v[k] = norm_out((v[i].v[k] - mean) * rstd, w[k], b[k], a.silu, a.z != nullptr, a.z ? z[i].v[k] : 0.0f);
            y.store(static_cast<T *>(a.y) + base + off[i]);
        }
}

// count, mean and sum of squared deviations of a set of values
struct Stat { float n, mean, m2; };
__device__ __forceinline__ Stat merge(const Stat &p, const Stat &q) {
    const float n = p.n + q.n;
    if (n == 0.0f) return p;
    const float d = q.mean - p.mean, f = q.n / n;
    return Stat{n, __builtin_fmaf(d, f, p.mean), p.m2 + q.m2 + d * d * p.n * f};
}

// ---- statistics of one slab of rows: blockIdx = (slab, block of whole groups, n)
template <class T, int VE>
__global__ void __launch_bounds__(kWG) gn_stats_kernel(GroupNormArgs a) {
    __shared__ Stat st[kWG];
    const int lpg = static_cast<int>(a.S / VE);
    const int gpb = lpg >= kWG ? 1 : kWG / lpg;   // groups of one block
    const int64_t g0 = static_cast<int64_t>(blockIdx.y) * gpb;
    const int groups = static_cast<int>(min(static_cast<int64_t>(gpb), a.G - g0));
    const int cols = min(groups * lpg, kWG), R = kWG / cols;   // columns in use, rows side by side
    const int r = threadIdx.x / cols, j0 = threadIdx.x % cols;
    const int64_t n = blockIdx.z, row0 = static_cast<int64_t>(blockIdx.x) * a.slab_rows;
    const int64_t rows = min(a.slab_rows, a.L - row0);
    Stat s = {0.0f, 0.0f, 0.0f};
    if (r < R)
        for (int64_t l = r; l < rows; l += R)
            for (int j = j0; j < groups * lpg; j += kWG) {   // (more than one turn: one group, wider than the block)
                Vec<T, VE> v;
                v.load(static_cast<const T *>(a.x) + (n * a.L + row0 + l) * a.C + g0 * a.S + static_cast<int64_t>(j) * VE);
                Stat q = {static_cast<float>(VE), 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < VE; ++k) q.mean += v.v[k];
                q.mean *= 1.0f / VE;
#pragma unroll
                for (int k = 0; k < VE; ++k) { const float d = v.v[k] - q.mean; q.m2 = __builtin_fmaf(d, d, q.m2); }
                s = merge(s, q);
            }
    st[threadIdx.x] = s;
    __syncthreads();
    // rows, then the columns of a group, merged pairwise
    int half = 1;
    while (half < R) half <<= 1;
    for (half >>= 1; half > 0; half >>= 1) {
        if (r < half && r + half < R) st[threadIdx.x] = merge(st[threadIdx.x], st[threadIdx.x + half * cols]);
        __syncthreads();
    }
    const int width = min(lpg, kWG), p = j0 % width;
    half = 1;
    while (half < width) half <<= 1;
    for (half >>= 1; half > 0; half >>= 1) {
        if (r == 0 && p < half && p + half < width) st[threadIdx.x] = merge(st[threadIdx.x], st[threadIdx.x + half]);
        __syncthreads();
    }
    if (r == 0 && p == 0 && j0 / width < groups) {
        float *o = a.part + ((n * a.nslab + blockIdx.x) * a.G + g0 + j0 / width) * 2;
        o[0] = st[threadIdx.x].mean;
        o[1] = st[threadIdx.x].m2;
    }
}

// slabs' statistics -> mean and rstd of every (n, g); one wave each
__global__ void __launch_bounds__(64) gn_finalize_kernel(GroupNormArgs a) {
    const int64_t n = blockIdx.y, g = blockIdx.x, ng = n * a.G + g;
    Stat s = {0.0f, 0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < a.nslab; i += 64) {
        const float *p = a.part + ((n * a.nslab + i) * a.G + g) * 2;
        const float rows = static_cast<float>(min(a.slab_rows, a.L - i * a.slab_rows));
        s = merge(s, Stat{rows * static_cast<float>(a.S), p[0], p[1]});
    }
    for (int o = 1; o < 64; o <<= 1) {
        const Stat q = {__shfl_xor(s.n, o, 64), __shfl_xor(s.mean, o, 64), __shfl_xor(s.m2, o, 64)};
        s = (threadIdx.x & o) ? merge(q, s) : merge(s, q);
    }
    if (threadIdx.x == 0) {
        a.mean[ng] = s.mean;
        a.rstd[ng] = 1.0f / sqrtf(s.m2 / (static_cast<float>(a.L) * static_cast<float>(a.S)) + a.eps);
    }
}

// ---- y of one slab: blockIdx = (slab, block of columns, n)
template <class T, int VE>
__global__ void __launch_bounds__(kWG) gn_apply_kernel(GroupNormArgs a) {
    const int64_t vecs = a.C / VE, v0 = static_cast<int64_t>(blockIdx.y) * kWG;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kWG), vecs - v0)), R = kWG / cols;
    const int r = threadIdx.x / cols;
    const int64_t c = (v0 + threadIdx.x % cols) * VE, n = blockIdx.z;
    if (r >= R) return;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.slab_rows, end = min(row0 + a.slab_rows, a.L), g = c / a.S;
    const float mean = a.mean[n * a.G + g], rstd = a.rstd[n * a.G + g];
    float w[VE], b[VE];
    channels<VE>(a.w, c, 1.0f, w);
    channels<VE>(a.b, c, 0.0f, b);
    for (int64_t l = row0 + r; l < end; l += R) {
        const int64_t at = (n * a.L + l) * a.C + c;
        Vec<T, VE> v, z, y;
        v.load(static_cast<const T *>(a.x) + at);
        if (a.z) z.load(static_cast<const T *>(a.z) + at);
#pragma unroll
        for (int k = 0; k < VE; ++k)
            y.v[k] = norm_out((v.v[k] - mean) * rstd, w[k], b[k], a.silu, a.z != nullptr, a.z ? z.v[k] : 0.0f);
        y.store(static_cast<T *>(a.y) + at);
    }
}

// ---- backward, L = 1, groups that fit a team's registers.  A workgroup keeps its groups and
// walks rows, so each lane sums dw and db of its own channels: blockIdx = (groups, rows)
template <class T, int VE, int MAXV, bool WG>
__global__ void __launch_bounds__(kWG) gn_bwd_team_kernel(GroupNormArgs a) {
    __shared__ float lds[4];
    const int P = WG ? kWG : a.team, sh = __builtin_ctz(P), tl = threadIdx.x & (P - 1), teams = kWG >> sh;
    const int gb = static_cast<int>(min(static_cast<int64_t>(teams), a.G)), side = teams / gb;   // groups, rows side by side
    const int team = threadIdx.x >> sh;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * gb + team % gb, rl = team / gb;
    const bool on = g < a.G && rl < side;
    const int nvec = static_cast<int>(a.nvec);
    float w[MAXV][VE], b[MAXV][VE], dw[MAXV][VE], db[MAXV][VE];
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
        const int e = tl + i * P;
#pragma unroll
        for (int k = 0; k < VE; ++k) w[i][k] = b[i][k] = dw[i][k] = db[i][k] = 0.0f;
        if (on && e < nvec) {
            channels<VE>(a.w, g * a.S + e * VE, 1.0f, w[i]);
            channels<VE>(a.b, g * a.S + e * VE, 0.0f, b[i]);
        }
    }
    const float inv_m = a.inv_m;
    // (every lane of a workgroup makes the same number of turns: the team sums are collective)
    for (int64_t n0 = static_cast<int64_t>(blockIdx.y) * side; n0 < a.N; n0 += static_cast<int64_t>(gridDim.y) * side) {
        const int64_t n = n0 + rl;
        const bool row = on && n < a.N;
        const int64_t base = n * a.C + g * a.S;
        Vec<T, VE> x[MAXV], dy[MAXV], z[MAXV];
        const float mean = row ? a.mean[n * a.G + g] : 0.0f, rstd = row ? a.rstd[n * a.G + g] : 0.0f;
#pragma unroll
        for (int i = 0; i < MAXV; ++i) {
            const int e = tl + i * P;
            x[i].fill(0.0f);
            dy[i].fill(0.0f);
            z[i].fill(0.0f);
            if (row && e < nvec) {
                x[i].load(static_cast<const T *>(a.x) + base + e * VE);
                dy[i].load(static_cast<const T *>(a.dy) + base + e * VE);
                if (a.z) z[i].load(static_cast<const T *>(a.z) + base + e * VE);
            }
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < MAXV; ++i) {
            const bool in = row && tl + i * P < nvec;
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float xh = (x[i].v[k] - mean) * rstd;
                float dz = 0.0f;
                const float gr = in ? norm_grad(xh, w[i][k], b[i][k], a.silu, a.z != nullptr, z[i].v[k], dy[i].v[k], dz) : 0.0f;
                db[i][k] += gr;
                dw[i][k] = in ? __builtin_fmaf(gr, xh, dw[i][k]) : dw[i][k];
                const float e = gr * w[i][k];
                s1 += e;
                s2 = in ? __builtin_fmaf(e, xh, s2) : s2;
                x[i].v[k] = xh;
                dy[i].v[k] = e;
                z[i].v[k] = dz;
            }
            if (a.z && in) z[i].store(static_cast<T *>(a.dz) + base + (tl + i * P) * VE);
        }
        s1 = team_sum<WG>(s1, P, lds) * inv_m;
        s2 = team_sum<WG>(s2, P, lds) * inv_m;
#pragma unroll
        for (int i = 0; i < MAXV; ++i)
            if (row && tl + i * P < nvec) {
                Vec<T, VE> dx;
#pragma unroll
                for (int k = 0; k < VE; ++k) dx.v[k] = rstd * (dy[i].v[k] - __builtin_fmaf(x[i].v[k], s2, s1));
                dx.store(static_cast<T *>(a.dx) + base + (tl + i * P) * VE);
            }
    }
    if (!a.part || !on) return;
    float *p = a.part + (static_cast<int64_t>(blockIdx.y) * side + rl) * 2 * a.C + g * a.S;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
        const int e = tl + i * P;
        if (e < nvec)
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                p[e * VE + k] = dw[i][k];
                p[a.C + e * VE + k] = db[i][k];
            }
    }
}

// ---- dx and dz where there are many groups, of few values each: a team of lanes walks one (n, g) twice, for
// the two sums of dx and for dx (the second time from the caches), so nothing per row is kept in memory.  dw
// and db come from gn_bwd_sums_kernel over all rows.
template <class T, int VE, bool WG>
__global__ void __launch_bounds__(kWG) gn_bwd_walk_kernel(GroupNormArgs a) {
    __shared__ float lds[4];
    const int P = WG ? kWG : a.team, sh = __builtin_ctz(P), tl = threadIdx.x & (P - 1);
    const uint32_t team = (blockIdx.y * gridDim.x + blockIdx.x) * (kWG >> sh) + (threadIdx.x >> sh);
    const bool on = team < static_cast<uint32_t>(a.N * a.G);
    const uint32_t G = static_cast<uint32_t>(a.G), n = (on ? team : 0) / G, g = (on ? team : 0) % G;
    const int lpg = static_cast<int>(a.S / VE), dl = P / lpg, dj = P % lpg;   // vectors of a row; a lane's step in rows and vectors
    const int64_t base = static_cast<int64_t>(n) * a.L * a.C + static_cast<int64_t>(g) * a.S, c0 = static_cast<int64_t>(g) * a.S;
    const T *x = static_cast<const T *>(a.x) + base, *dy = static_cast<const T *>(a.dy) + base, *z = a.z ? static_cast<const T *>(a.z) + base : nullptr;
    const float mean = on ? a.mean[team] : 0.0f, rstd = on ? a.rstd[team] : 0.0f;
    // what(offset, xh, e, dz) for each of the lane's vectors
    auto walk = [&](auto what) __attribute__((always_inline)) {
        int64_t l = tl / lpg;
        int j = tl % lpg;
        const int64_t rows = on ? a.L : 0;
        while (l < rows) {
            const int64_t at = l * a.C + static_cast<int64_t>(j) * VE;
            Vec<T, VE> xh, e, gate;
            xh.load(x + at);
            e.load(dy + at);
            if (a.z) gate.load(z + at);
            float w[VE], b[VE];
            channels<VE>(a.w, c0 + static_cast<int64_t>(j) * VE, 1.0f, w);
            channels<VE>(a.b, c0 + static_cast<int64_t>(j) * VE, 0.0f, b);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                xh.v[k] = (xh.v[k] - mean) * rstd;
                float dz = 0.0f;
                e.v[k] = norm_grad(xh.v[k], w[k], b[k], a.silu, a.z != nullptr, a.z ? gate.v[k] : 0.0f, e.v[k], dz) * w[k];
                gate.v[k] = dz;
            }
            what(at, xh, e, gate);
            l += dl;
            j += dj;
            if (j >= lpg) {
                j -= lpg;
                ++l;
            }
        }
    };
    float s1 = 0.0f, s2 = 0.0f;
    walk([&](int64_t, const Vec<T, VE> &xh, const Vec<T, VE> &e, const Vec<T, VE> &) __attribute__((always_inline)) {
        float p1 = 0.0f, p2 = 0.0f;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            p1 += e.v[k];
            p2 = __builtin_fmaf(e.v[k], xh.v[k], p2);
        }
        s1 += p1;
        s2 += p2;
    });
    s1 = team_sum<WG>(s1, P, lds) * a.inv_m;
    s2 = team_sum<WG>(s2, P, lds) * a.inv_m;
    walk([&](int64_t at, const Vec<T, VE> &xh, const Vec<T, VE> &e, const Vec<T, VE> &dz) __attribute__((always_inline)) {
        Vec<T, VE> dx;
#pragma unroll
        for (int k = 0; k < VE; ++k) dx.v[k] = rstd * (e.v[k] - __builtin_fmaf(xh.v[k], s2, s1));
        dx.store(static_cast<T *>(a.dx) + base + at);
        if (a.z) dz.store(static_cast<T *>(a.dz) + base + at);
    });
}

// ---- backward of larger groups: sums of g xh and g per channel over one slab, blockIdx =
// (slab, block of columns, n); ALL: over rows of every n, for dw and db alone, blockIdx = (block of
// columns, slab)
template <class T, int VE, bool ALL>
__global__ void __launch_bounds__(kWG) gn_bwd_sums_kernel(GroupNormArgs a) {
    __shared__ float lds[kWG][2 * VE + 1];
    const int64_t vecs = a.C / VE, v0 = static_cast<int64_t>(ALL ? blockIdx.x : blockIdx.y) * kWG, slab = ALL ? blockIdx.y : blockIdx.x;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kWG), vecs - v0)), R = kWG / cols;
    const int r = threadIdx.x / cols;
    const int64_t c = (v0 + threadIdx.x % cols) * VE, n = ALL ? 0 : blockIdx.z;
    const int64_t row0 = slab * a.slab_rows, end = min(row0 + a.slab_rows, ALL ? a.N * a.L : a.L);
    float dw[VE], db[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) dw[k] = db[k] = 0.0f;
    if (r < R) {
        const int64_t g = c / a.S;
        float mean = ALL ? 0.0f : a.mean[n * a.G + g], rstd = ALL ? 0.0f : a.rstd[n * a.G + g];
        float w[VE], b[VE];
        channels<VE>(a.w, c, 1.0f, w);
        channels<VE>(a.b, c, 0.0f, b);
        for (int64_t l = row0 + r; l < end; l += R) {
            const int64_t at = (n * a.L + l) * a.C + c;
            if constexpr (ALL) {
                const int64_t ng = (a.L == 1 ? l : l / a.L) * a.G + g;
                mean = a.mean[ng];
                rstd = a.rstd[ng];
            }
            Vec<T, VE> x, dy, z;
            x.load(static_cast<const T *>(a.x) + at);
            dy.load(static_cast<const T *>(a.dy) + at);
            if (a.z) z.load(static_cast<const T *>(a.z) + at);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float xh = (x.v[k] - mean) * rstd;
                float dz;
                const float g = norm_grad(xh, w[k], b[k], a.silu, a.z != nullptr, a.z ? z.v[k] : 0.0f, dy.v[k], dz);
                dw[k] = __builtin_fmaf(g, xh, dw[k]);
                db[k] += g;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < VE; ++k) {
        lds[threadIdx.x][k] = dw[k];
        lds[threadIdx.x][VE + k] = db[k];
    }
    __syncthreads();
    int half = 1;
    while (half < R) half <<= 1;
    for (half >>= 1; half > 0; half >>= 1) {
        if (r < half && r + half < R)
#pragma unroll
            for (int k = 0; k < 2 * VE; ++k) lds[threadIdx.x][k] += lds[threadIdx.x + half * cols][k];
        __syncthreads();
    }
    if (r == 0) {
        float *p = a.part + (n * a.nslab + slab) * 2 * a.C + c;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            p[k] = lds[threadIdx.x][k];
            p[a.C + k] = lds[threadIdx.x][VE + k];
        }
    }
}

// sums over the rows of [blockIdx.y][rows][width] -> [blockIdx.y][width], in a fixed order; with
// split: the first half of the width into out, the second into out2 (either may be null)
__global__ void __launch_bounds__(1024) gn_column_sum_kernel(const float *part, int64_t rows, int64_t width, float *out, float *out2,
                                                             bool split) {
    __shared__ float lds[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    const float *p = part + static_cast<int64_t>(blockIdx.y) * rows * width;
    float s = 0.0f;
    if (c < width)
        for (int64_t r = ty; r < rows; r += 32) s += p[r * width + c];
    lds[ty][tx] = s;
    __syncthreads();
    for (int o = 16; o > 0; o >>= 1) {
        if (ty < o) lds[ty][tx] += lds[ty + o][tx];
        __syncthreads();
    }
    if (ty == 0 && c < width) {
        if (!split) out[blockIdx.y * width + c] = lds[0][tx];
        else if (c < width / 2) { if (out) out[c] = lds[0][tx]; }
        else if (out2) out2[c - width / 2] = lds[0][tx];
    }
}

// sums [N][2 C] of g xh and g -> per (n, g) the two sums of dx, over M; one wave each
__global__ void __launch_bounds__(64) gn_bwd_group_kernel(GroupNormArgs a) {
    const int64_t n = blockIdx.y, g = blockIdx.x, ng = n * a.G + g;
    const float *p = a.sums + n * 2 * a.C + g * a.S;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < a.S; c += 64) {
        const float w = a.w ? a.w[g * a.S + c] : 1.0f;
        s2 = __builtin_fmaf(w, p[c], s2);
        s1 = __builtin_fmaf(w, p[a.C + c], s1);
    }
    for (int o = 32; o > 0; o >>= 1) {
        s1 += __shfl_xor(s1, o, 64);
        s2 += __shfl_xor(s2, o, 64);
    }
    if (threadIdx.x == 0) {
        const float m = static_cast<float>(a.L) * static_cast<float>(a.S);
        a.gsum[2 * ng] = s1 / m;
        a.gsum[2 * ng + 1] = s2 / m;
    }
}

template <class T, int VE>
__global__ void __launch_bounds__(kWG) gn_bwd_apply_kernel(GroupNormArgs a) {
    const int64_t vecs = a.C / VE, v0 = static_cast<int64_t>(blockIdx.y) * kWG;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kWG), vecs - v0)), R = kWG / cols;
    const int r = threadIdx.x / cols;
    if (r >= R) return;
    const int64_t c = (v0 + threadIdx.x % cols) * VE, n = blockIdx.z, ng = n * a.G + c / a.S;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.slab_rows, end = min(row0 + a.slab_rows, a.L);
    const float mean = a.mean[ng], rstd = a.rstd[ng], s1 = a.gsum[2 * ng], s2 = a.gsum[2 * ng + 1];
    float w[VE], b[VE];
    channels<VE>(a.w, c, 1.0f, w);
    channels<VE>(a.b, c, 0.0f, b);
    for (int64_t l = row0 + r; l < end; l += R) {
        const int64_t at = (n * a.L + l) * a.C + c;
        Vec<T, VE> x, dy, z;
        x.load(static_cast<const T *>(a.x) + at);
        dy.load(static_cast<const T *>(a.dy) + at);
        if (a.z) z.load(static_cast<const T *>(a.z) + at);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const float xh = (x.v[k] - mean) * rstd;
            float dz = 0.0f;
            const float g = norm_grad(xh, w[k], b[k], a.silu, a.z != nullptr, a.z ? z.v[k] : 0.0f, dy.v[k], dz);
            x.v[k] = rstd * (g * w[k] - __builtin_fmaf(xh, s2, s1));
            z.v[k] = dz;
        }
        x.store(static_cast<T *>(a.dx) + at);
        if (a.z) z.store(static_cast<T *>(a.dz) + at);
    }
}

// (slab, block of columns, n)
dim3 blocks(const GroupNormArgs &a, int64_t columns) {
    return dim3(static_cast<unsigned>(a.nslab), static_cast<unsigned>(columns), static_cast<unsigned>(a.N));
}

// a team of lanes for every (n, g) (a launch's threads along one axis are counted in 32 bits)
dim3 team_grid(const GroupNormArgs &a) {
    const int64_t n = (a.N * a.G * a.team + kWG - 1) / kWG, across = n < (1 << 20) ? n : 1 << 20;
    return dim3(static_cast<unsigned>(across), static_cast<unsigned>((n + across - 1) / across));
}

template <class T, int VE>
hipError_t fwd_typed(const GroupNormArgs &a, hipStream_t s) {
    if (a.team > 0) {
        const dim3 grid = team_grid(a);
        auto launch = [&](auto one) {
            constexpr bool ONE = decltype(one)::value;
            if (a.team == kWG) hipLaunchKernelGGL((gn_team_kernel<T, VE, 8, true, ONE>), grid, dim3(kWG), 0, s, a);
            else if (a.nvec <= a.team) hipLaunchKernelGGL((gn_team_kernel<T, VE, 1, false, ONE>), grid, dim3(kWG), 0, s, a);
            else hipLaunchKernelGGL((gn_team_kernel<T, VE, 4, false, ONE>), grid, dim3(kWG), 0, s, a);
        };
        if (a.L == 1) launch(std::true_type{});
        else launch(std::false_type{});
        return launch_status(s);
    }
    const int64_t lpg = a.S / VE, gpb = lpg >= kWG ? 1 : kWG / lpg;
    hipLaunchKernelGGL((gn_stats_kernel<T, VE>), blocks(a, (a.G + gpb - 1) / gpb), dim3(kWG), 0, s, a);
    hipError_t e = launch_status(s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gn_finalize_kernel, dim3(static_cast<unsigned>(a.G), static_cast<unsigned>(a.N)), dim3(64), 0, s, a);
    e = launch_status(s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gn_apply_kernel<T, VE>), blocks(a, (a.C / VE + kWG - 1) / kWG), dim3(kWG), 0, s, a);
    return launch_status(s);
}

template <class T, int VE>
hipError_t bwd_typed(const GroupNormArgs &a, hipStream_t s) {
    const unsigned cols = static_cast<unsigned>((2 * a.C + 31) / 32);
    if (a.walk) {
        const dim3 grid = team_grid(a);
        if (a.team == kWG) hipLaunchKernelGGL((gn_bwd_walk_kernel<T, VE, true>), grid, dim3(kWG), 0, s, a);
        else hipLaunchKernelGGL((gn_bwd_walk_kernel<T, VE, false>), grid, dim3(kWG), 0, s, a);
        hipError_t e = launch_status(s);
        if (e != hipSuccess || !(a.dw || a.db)) return e;
        hipLaunchKernelGGL((gn_bwd_sums_kernel<T, VE, true>),
                           dim3(static_cast<unsigned>((a.C / VE + kWG - 1) / kWG), static_cast<unsigned>(a.nslab)), dim3(kWG), 0, s, a);
        e = launch_status(s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(gn_column_sum_kernel, dim3(cols), dim3(1024), 0, s, a.part, a.nslab, 2 * a.C, a.dw, a.db, true);
        return launch_status(s);
    }
    if (a.team > 0) {
        const int64_t teams = kWG / a.team, gb = teams < a.G ? teams : a.G;
        const dim3 grid(static_cast<unsigned>((a.G + gb - 1) / gb), static_cast<unsigned>(a.nslab));
        if (a.team < kWG) hipLaunchKernelGGL((gn_bwd_team_kernel<T, VE, 1, false>), grid, dim3(kWG), 0, s, a);
        else if (a.nvec <= kWG) hipLaunchKernelGGL((gn_bwd_team_kernel<T, VE, 1, true>), grid, dim3(kWG), 0, s, a);
        else hipLaunchKernelGGL((gn_bwd_team_kernel<T, VE, 2, true>), grid, dim3(kWG), 0, s, a);
        hipError_t e = launch_status(s);
        if (e != hipSuccess || !a.part) return e;
        hipLaunchKernelGGL(gn_column_sum_kernel, dim3(cols), dim3(1024), 0, s, a.part,
                           a.nslab * (teams / gb), 2 * a.C, a.dw, a.db, true);
        return launch_status(s);
    }
    const dim3 grid = blocks(a, (a.C / VE + kWG - 1) / kWG);
    hipLaunchKernelGGL((gn_bwd_sums_kernel<T, VE, false>), grid, dim3(kWG), 0, s, a);
    hipError_t e = launch_status(s);
    if (e != hipSuccess) return e;
    if (a.nslab > 1) {   // (one slab: its sums are the rows' sums)
        hipLaunchKernelGGL(gn_column_sum_kernel, dim3(cols, static_cast<unsigned>(a.N)), dim3(1024), 0, s, a.part, a.nslab, 2 * a.C, a.sums, nullptr, false);
        e = launch_status(s);
        if (e != hipSuccess) return e;
    }
    if (a.dw || a.db) {
        hipLaunchKernelGGL(gn_column_sum_kernel, dim3(cols), dim3(1024), 0, s, a.sums, a.N, 2 * a.C, a.dw, a.db, true);
        e = launch_status(s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(gn_bwd_group_kernel, dim3(static_cast<unsigned>(a.G), static_cast<unsigned>(a.N)), dim3(64), 0, s, a);
    e = launch_status(s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gn_bwd_apply_kernel<T, VE>), grid, dim3(kWG), 0, s, a);
    return launch_status(s);
}

}  // namespace

hipError_t launch_groupnorm_fwd(const GroupNormArgs &a0, bool bf16, bool vec, hipStream_t s) {
    GroupNormArgs a = a0;
    a.inv_m = 1.0f / (static_cast<float>(a.L) * static_cast<float>(a.S));
    if (bf16) return vec ? fwd_typed<uint16_t, 8>(a, s) : fwd_typed<uint16_t, 1>(a, s);
    return vec ? fwd_typed<float, 4>(a, s) : fwd_typed<float, 1>(a, s);
}

hipError_t launch_groupnorm_bwd(const GroupNormArgs &a0, bool bf16, bool vec, hipStream_t s) {
    GroupNormArgs a = a0;
    a.inv_m = 1.0f / (static_cast<float>(a.L) * static_cast<float>(a.S));
    if (bf16) return vec ? bwd_typed<uint16_t, 8>(a, s) : bwd_typed<uint16_t, 1>(a, s);
    return vec ? bwd_typed<float, 4>(a, s) : bwd_typed<float, 1>(a, s);
}

}  // namespace ssm
