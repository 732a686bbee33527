// Host-side argument checks and launch planning for libssm (no HIP here, so
// the same code builds with g++ under sanitizers for CPU tests).
#pragma once

#include <cstddef>
#include <cstdint>

#include "ssm.h"

namespace ssm {

constexpr int kWave = 64;            // lanes per wavefront on gfx950
constexpr int kChannelsPerBlock = 64; // one channel per lane of a wave
constexpr int kMaxWavesPerBlock = 16;
constexpr size_t kWsAlign = 256;
constexpr int64_t kCUs = 256;          // MI355X compute units
constexpr size_t kLdsPerCU = 160 * 1024;

struct ScanPlan {
    int G = 4;            // states of one channel held by one lane
    int NW = 4;           // waves per workgroup = ceil(N / G)
    int TB = 32;          // time steps staged per block
    int64_t chunk_len = 0;
    int64_t n_chunks = 1;
    size_t ws_bytes = 0;  // workspace for chunk carries (0 when n_chunks == 1)
    size_t ws_P_off = 0;  // byte offset of the per-chunk state decays [B][C-1][D][N]
    size_t ws_H_off = 0;  // byte offset of the per-chunk end states [B][C-1][D][N]
    size_t ws_BC_off = 0; // specialised kernel: byte offset of the packed fp32 B/C rows
    int64_t bc_lpad = 0;  // specialised kernel: steps per chunk in the packed B/C rows (multiple of 16)
    uint64_t blocks = 0;  // workgroups of the main scan launch
    bool fast = false;    // dstate == 16 and dim % 64 == 0: the specialised kernel runs
    size_t lds_reserve = 0;  // dynamic LDS that caps residency at one workgroup per CU
    bool structured = true;  // the Mamba kernels may take their structured-A path (device check)
    // Long chunks (chunk_len >= kLocalMinChunk): the workspace also holds what the local-scan
    // carries need (ScanArgs::ws_Hl, S_part, flags; ws_P then receives the prefix rescan's end
    // states).  run_scan uses them for the exponential discretisations.
    bool local = false;
    size_t ws_Hl_off = 0, ws_S_off = 0, ws_F_off = 0;
};
// Local-scan carries: the prefix of every chunk >= 1 that is rescanned from its carried-in
// state, and the shortest chunk for which the local-scan carries are used.
constexpr int64_t kLocalPrefix = 4096;
constexpr int64_t kLocalMinChunk = 4 * kLocalPrefix;

// Per-thread error text (ssm_last_error).
void set_error(const char *fmt, ...);
// Whether the environment variable name is set to something other than "" or "0" (read
// once per name by its callers).
bool env_flag(const char *name);
// SSM_LOG=1: one line per call on stderr describing what the entry point launches (shape,
// kernel path, plan).  Nothing is printed otherwise.
void log_call(const char *fmt, ...);
void clear_error();

// Shape and option checks + plan.  Returns an ssm_status.
int plan_scan(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
              const ssm_scan_opts *opts, ScanPlan *plan);

// Full argument check of ssm_scan_fwd (shape, pointers, alignment, overlap,
// workspace).  Returns an ssm_status; fills *plan on success.
int check_scan(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
               const void *x, const void *delta, const float *A, const void *B, const void *C,
               const float *Dskip, const void *z, const float *h0, const float *h_last,
               const void *y, int delta_softplus, const ssm_variant *variant,
               const ssm_scan_opts *opts, const void *workspace, size_t workspace_bytes,
               ScanPlan *plan);

// Full argument check of ssm_state_update.
int check_state_update(int64_t batch, int64_t dim, int64_t dstate, int dtype, const float *h,
                       const void *x, const void *delta, const float *A, const void *B,
                       const void *C, const float *Dskip, const void *z, const void *y,
                       int delta_softplus, const ssm_variant *variant);

// The discretisation of a variant (NULL = SSM_DISC_MAMBA) and its delta bias.
inline int variant_disc(const ssm_variant *v) { return v ? v->discretization : SSM_DISC_MAMBA; }
inline const float *variant_bias(const ssm_variant *v) { return v ? v->delta_bias : nullptr; }

// Workspace of ssm_scan_bwd: per-workgroup shares of dB/dC, per-(chunk, row) shares of
// dA/dD, the adjoint carries, then (last, so that a call given saved checkpoints needs
// only the part before them) the forward checkpoint pass's own workspace and the state
// checkpoints.
// Buffers of the padded backward, in workspace order: inputs, then outputs, then (with more
// than one group of 16 states) the fp32 sums of the per-channel gradients over the groups.
enum PadBuf {
    kPX, kPDelta, kPZ, kPDy, kPB, kPC, kPA, kPDskip, kPBias, kPH0, kPDhLast,
    kPDx, kPDdelta, kPDz, kPDB, kPDC, kPDA, kPDD, kPDBias, kPDh0,
    kSDx, kSDdelta, kSDz, kSDBias, kPadBufs
};

struct BwdPlan {
    int64_t nblk = 0;       // 8-step blocks of the reverse sweep
    int64_t n_chunks = 1, chunk_len = 0;   // sequence chunks (chunk_len a multiple of 16 when several)
    ScanPlan fwd;           // the checkpoint pass: the specialised forward kernel, same chunks
    size_t partBC_off = 0, partA_off = 0, partD_off = 0, partDB_off = 0;
    size_t lcP_off = 0, lcH_off = 0;   // adjoint carries (several chunks only)
    size_t fwd_off = 0;     // the forward plan's workspace (its carries and packed B/C)
    size_t ckpt_off = 0;    // checkpoints [B][nblk][16][D] fp32
    size_t ckpt_bytes = 0;
    size_t ws_bytes = 0;        // with the checkpoint pass
    size_t ws_bytes_saved = 0;  // given saved checkpoints (= fwd_off)
    // Other shapes (dstate < 16 or dim not a multiple of 64) run the same kernels on copies
    // padded to dim Dp (the next multiple of 64) and 16 states, in the workspace; the pad
    // region comes first, the native plan's workspace (of the padded shape) after it.
    bool pad = false;
    int64_t Dp = 0;
    // More than 16 states: K = ceil(dstate / 16) groups of 16, each run through the native
    // kernels on fp32 copies (the token tensors once, B, C, A and the states per group); the
    // per-channel gradients (dx, ddelta, dz, the bias's) are sums over the groups, D enters
    // in group 0 only.  K == 1 is the padded path above, on copies of the input dtype.
    int64_t K = 1;
    // K > 1 with fp32 tokens of a width that needs no padding: the tokens are read in place and
    // the per-channel gradients summed straight into the caller's outputs (no token copies)
    bool direct = false;
    size_t pad_off[kPadBufs] = {};
    size_t inner_off = 0;
};

int plan_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                  BwdPlan *plan);

// Full argument check of ssm_scan_bwd.
int check_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                   const void *x, const void *delta, const float *A, const void *B, const void *C,
                   const float *Dskip, const void *z, const float *h0, const void *dy,
                   const float *dh_last, const void *dx, const void *ddelta, const float *dA,
                   const void *dB, const void *dC, const float *dD, const void *dz, const float *dh0,
                   int delta_softplus, int discretization, const float *delta_bias,
                   const float *ddelta_bias, const float *checkpoints,
                   const void *workspace, size_t workspace_bytes, BwdPlan *plan);
// Full argument check of ssm_scan_fwd_save: ssm_scan_fwd's on the backward's chunk plan,
// plus the checkpoint output.  Fills *plan (the backward's) on success.
int check_scan_save(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                    const void *x, const void *delta, const float *A, const void *B, const void *C,
                    const float *Dskip, const void *z, const float *h0, const float *h_last,
                    const void *y, int delta_softplus, const ssm_variant *variant,
                    const float *checkpoints, const void *workspace, size_t workspace_bytes,
                    BwdPlan *plan);

// Argument checks of the convolution entry points.
int check_conv1d_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int dtype,
                     const void *x, const float *w, const float *bias, const void *state_in,
                     const void *y, const void *state_out, int silu);
constexpr int kConvBwdTile = 64;   // steps per thread (and per partial sum) in the convolution's backward

// Bytes of the convolution backward's workspace (per-(row, tile) sums of dw, dbias).
size_t conv1d_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t width);
int check_conv1d_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int dtype,
                     const void *x, const float *w, const float *bias, const void *state_in,
                     const void *dy, const void *dx, const float *dw, const float *dbias,
                     const void *dstate, int silu, const void *workspace, size_t workspace_bytes);
int check_conv1d_update(int64_t batch, int64_t dim, int64_t width, int dtype, const void *state,
                        const void *x, const float *w, const float *bias, const void *y, int silu);

// Argument checks of the multi-head SSD scan (ssm_ssd_fwd).
int check_ssd(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups, int dtype,
              const void *x, const void *delta, const float *A, const void *B, const void *C,
              const float *Dskip, const void *z, const float *delta_bias, const float *h0,
              const float *h_last, const void *y, int delta_softplus);

// Linear attention: how the sequence is split and what the workspace holds.
struct LinAttnPlan {
    int64_t q_row = 0, k_row = 0, v_row = 0;   // token strides, with the contiguous default filled in
    // a sweep with contraction size c and n value columns: segments and their length
    struct Sweep {
        int64_t nseg = 1, seg_len = 0, ntiles = 1;
        int64_t nsub = 1, sub_len = 0;   // parts of a segment in the pass for the segments' own states
        bool given = false;              // starts from the states of another sweep
        size_t state_bytes = 0;          // one array of the segments' states (its own)
    };
    Sweep fwd;                  // y: contraction over dk, dv columns
    Sweep bwd;                  // dq and dk: contraction over dv, dk columns
    Sweep dv;                   // as fwd; where it gains, from dk's states
    size_t ws_bytes = 0;        // of the forward
    // backward: states (and their derivatives by log_decay), the shares of dlog_decay, per-head
    // fp32 gradients of rows that several heads share
    size_t ws_R_off = 0, age_off = 0, part_off = 0, ws_bwd_bytes = 0;
};
int plan_linattn(const ssm_linattn_shape *s, bool decay_grad, LinAttnPlan *plan);
int check_linattn_fwd(const ssm_linattn_shape *s, const void *q, const void *k, const void *v, const float *log_decay,
                      const int32_t *lengths, const float *h0, const float *h_last, const void *y,
                      const void *workspace, size_t workspace_bytes, LinAttnPlan *plan);
int check_linattn_bwd(const ssm_linattn_shape *s, const void *q, const void *k, const void *v, const float *log_decay,
                      const int32_t *lengths, const float *h0, const void *dy, const float *dh_last, const void *dq,
                      const void *dk, const void *dv, const float *dlog_decay, const float *dh0,
                      const void *workspace, size_t workspace_bytes, LinAttnPlan *plan);
int check_linattn_update(const ssm_linattn_shape *s, const float *h, const void *q, const void *k, const void *v,
                         const float *log_decay, const void *y, LinAttnPlan *plan);

// Group norm: how groups are held (see groupnorm.hip) and what the workspace holds.
struct GroupNormPlan {
    bool vec = false;        // 16-byte loads
    int team = 0;            // lanes that hold (walk: that walk) one group; 0: slabs of rows
    bool walk = false;       // backward: dx by teams that walk groups, dw and dbias over slabs of all rows
    int64_t nvec = 0;        // vectors (or elements) of one group
    int64_t nslab = 1, slab_rows = 0;
    size_t mean_off = 0, rstd_off = 0, sums_off = 0, gsum_off = 0;   // (the slabs' sums come first)
    size_t ws_bytes = 0;
};
int plan_groupnorm(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int dtype, bool backward, GroupNormPlan *plan);
int check_groupnorm_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int dtype, const void *x,
                        const float *w, const float *bias, const void *z, float eps, int silu, const void *y,
                        const float *mean, const float *rstd, const void *workspace, size_t workspace_bytes,
                        GroupNormPlan *plan);
int check_groupnorm_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int dtype, const void *x,
                        const float *w, const float *bias, const void *z, int silu, const void *dy, const float *mean,
                        const float *rstd, const void *dx, const float *dw, const float *dbias, const void *dz,
                        const void *workspace, size_t workspace_bytes, GroupNormPlan *plan);

// The served Mamba-2 mixer: how sequences are split and what the workspace holds (see ssdconv.hip).
struct SsdConvPlan {
    int64_t x_row = 0, z_row = 0, d_row = 0, channels = 0;
    int64_t blocks64 = 1;             // blocks of 64 channels of a head
    int64_t chunks = 0, items = 0;    // numbers of chunks and segments
    int64_t heads_run = 1;            // workgroups of a segment that share an XCD: divides the segment's
    int64_t seg_len = 0;
    bool split = false;
    bool h_vec = false;
    int team = 1, shares = 1;
    size_t c_off = 0, cb_off = 0, tab_off = 0, state_off = 0, dec_off = 0, ws_bytes = 0;
};
constexpr int64_t kSsdConvWhole = int64_t(1) << 30;   // seg_len of sequences that are not split
int plan_ssdconv(const ssm_ssdconv_shape *s, bool token, SsdConvPlan *plan);
int check_ssdconv(const ssm_ssdconv_shape *s, bool token, const void *xbc, const void *delta, const float *A, const float *w,
                  const float *bias, const float *Dskip, const void *z, const float *delta_bias, int delta_softplus,
                  const int32_t *offsets, const int32_t *slots, const uint8_t *fresh, const float *h, const void *conv_state,
                  const void *y, const void *workspace, size_t workspace_bytes, SsdConvPlan *plan);

// Rotary positions and head norms: how rows are held (see rotary.hip).
struct RotaryPlan {
    int64_t q_row = 0, k_row = 0;
    int vec = 1;                 // elements a load
    int team = 1, units = 1, tokens_per = 1;
    int64_t groups = 0, blocks = 0;
    size_t ws_bytes = 0;         // of the normed form's backward
};
// outs: the contiguous tensors of q and k that are written, grads: incoming gradients (backward), or null
int check_rotary(const ssm_rotary_shape *s, const void *q, const void *k, const float *wq, const float *wk,
                 const int32_t *positions, const double *freqs, float eps, const void *q_out, const void *k_out,
                 const void *dq_out, const void *dk_out, const float *dwq, const float *dwk, bool backward,
                 const void *workspace, size_t workspace_bytes, RotaryPlan *plan);
size_t qknorm_bwd_ws_bytes(const ssm_rotary_shape *s);

inline size_t dtype_size(int dtype) { return dtype == SSM_DTYPE_BF16 ? 2 : 4; }

}  // namespace ssm
