// linattn.cuh -- shared pieces of the linear-attention kernels (decay per head, no erase):
// one run, the cut of long sequences into pieces, and the launchers.
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace gdn2 {
namespace lin {

// Sequences cut into pieces of whole steps (chunks of the tensor-core run, tiles of the fp32 run).  A
// sequence of at least two `target`s of tokens is cut into len / target pieces; the rest stay whole.
constexpr int kChunk = 128;
constexpr int kTile32 = 32;  // tokens of a step of the fp32 run
constexpr int kNoCut = 0x7fffffff;
struct Cut {
  const int32_t *cu;       // device [n_seqs + 1] token offsets, or NULL: n_seqs x seq_len tokens
  const int32_t *seg_off;  // device [n_seqs + 1]: first piece of every sequence (packed batches with
                           // cuts), or NULL: every sequence has `per_seq` pieces
  const int32_t *cut_off;  // device [n_seqs + 1] beside it: pieces of cut sequences in front of every sequence.
                           // Only they have a state of their own to keep: a batch of many short sequences
                           // needs no room for each.
  const int32_t *order;    // device [n_pieces]: the pieces from the longest down (-1 behind the last), or
                           // NULL: as they come.  Blocks start in that order, so that no long piece is left
                           // for the end of a ragged batch.
  int n_seqs, seq_len, H;
  int per_seq;             // pieces per sequence without seg_off
  int n_pieces;            // pieces in all (an upper bound with seg_off)
  int n_cut;               // pieces of cut sequences (an upper bound with cut_off)
  int target, grain;       // pieces are cut at multiples of grain
  int t_total;
  int sorted;              // the call asks for an order
};

// Length of the pieces of a sequence of `len` tokens, and their number.
__host__ __device__ inline int piece_len(int len, int target, int grain) {
  const int count = len / target;
  if (count < 2) return len > 0 ? len : 1;
  const int each = (len + count - 1) / count;
  return (each + grain - 1) / grain * grain;
}
__host__ __device__ inline int piece_count(int len, int target, int grain) {
  const int pl = piece_len(len, target, grain);
  return len > 0 ? (len + pl - 1) / pl : 1;
}

struct Piece {
  int n, s, count;  // sequence, index of the piece in it, pieces of the sequence
  int t0, len;      // first token, tokens
  int unit;         // global index of the piece, times H, plus the head
  int cut;          // its number among the pieces of cut sequences (count > 1)
};
constexpr int kMaxSorted = 1024;  // pieces that one block sorts

// Bounds of sequence n; offsets outside [0, t_total] or out of order are cut back to it.
__device__ __forceinline__ void seq_bounds(const Cut &c, int n, int *t0, int *len) {
  if (!c.cu) {
    *t0 = n * c.seq_len;
    *len = c.seq_len;
    return;
  }
  const int a = min(max(c.cu[n], 0), c.t_total), b = min(max(c.cu[n + 1], a), c.t_total);
  *t0 = a;
  *len = b - a;
}

// The last of n offsets that is not above g.
__device__ __forceinline__ int last_below(const int32_t *off, int n, int g) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= g) lo = mid; else hi = mid;
  }
  return lo;
}
// Piece s of sequence n.
__device__ __forceinline__ void fill_piece(const Cut &c, int n, int s, Piece *p) {
  int t0, len;
  seq_bounds(c, n, &t0, &len);
  const int pl = piece_len(len, c.target, c.grain);
  p->n = n;
  p->s = s;
  p->count = c.seg_off ? c.seg_off[n + 1] - c.seg_off[n] : c.per_seq;
  p->t0 = t0 + min(s * pl, len);
  p->len = min(pl, len - min(s * pl, len));
  // (offsets out of order may count more pieces than there is room for)
  p->cut = min((c.cut_off ? c.cut_off[n] : n * c.per_seq) + s, c.n_cut - 1);
}
// Piece number g; false past the last one (the grid covers an upper bound).
__device__ __forceinline__ bool find_piece(const Cut &c, int g, Piece *p) {
  if (c.seg_off) {
    if (g >= c.seg_off[c.n_seqs]) return false;
    const int n = last_below(c.seg_off, c.n_seqs, g);
    fill_piece(c, n, g - c.seg_off[n], p);
  } else {
    fill_piece(c, g / c.per_seq, g % c.per_seq, p);
  }
  return true;
}
// The same by the number among the pieces of cut sequences.
__device__ __forceinline__ bool find_cut_piece(const Cut &c, int i, Piece *p) {
  if (!c.cut_off) return find_piece(c, i, p);
  if (i >= c.cut_off[c.n_seqs]) return false;
  const int n = last_below(c.cut_off, c.n_seqs, i);
  fill_piece(c, n, i - c.cut_off[n], p);
  return true;
}

// Groups of chunks that dlog_a of the tensor-core runs is summed over, numbered from each piece's
// start.  A group ends with an exact product of the two states, in between bf16 products add up: over
// 4096 tokens dlog_a is off by 0.40% with groups of 4 chunks, 0.32% with 2 and 0.27% with 1 (0.17% is its
// own rounding), and the gradients of 8 x 4096 took 553, 553 and 613 us (now 535 to 554).  Slot of the group that starts at
// token t of piece g: pieces are in token order, so no two share one.
constexpr int kGroup = 2;
constexpr int kMarkDots = 8;  // partial products a mark, one of each state warp
__host__ __device__ inline int mark_slot(int g, int t) { return g + t / (kGroup * kChunk); }
inline size_t mark_slots(const Cut &c) { return (size_t)c.n_pieces + (size_t)(c.t_total / (kGroup * kChunk)) + 1; }

// The piece of the block's unit (a position in the order, and a head); with `cuts` one of a cut sequence.
__device__ __forceinline__ bool find_unit(const Cut &c, int block, bool cuts, Piece *p) {
  const int pos = block / c.H;
  if (cuts) {
    p->unit = 0;
    return find_cut_piece(c, pos, p);
  }
  const int g = c.order ? c.order[pos] : pos;
  p->unit = g * c.H + block % c.H;
  return g >= 0 && find_piece(c, g, p);
}
// Blocks of a run: all units, or those whose end states the others start from.
inline int64_t run_blocks(const Cut &c, int state_only) { return (int64_t)(state_only ? c.n_cut : c.n_pieces) * c.H; }

// log_a below this is a reset: e^-104 is 0 in fp32, and sums over a chunk stay finite and fine enough
// (32 resets come to 4800 in log2, a float's step there is 2^-11).
constexpr float kMinLog = -104.f;
// A piece's sum of them, in units of 2^-32, stops here: 64 bits hold 14 million resets.
constexpr long long kMinLogs = -(1ll << 60);

// One run over all (piece, head) units:
//   forward:   out_t = sum_{j <= t} e^{L_t - L_j} (x_t . y_j) z_j + e^{L_t} start^T x_t
//   backward:  out_t = sum_{j >= t} e^{L_j - L_t} (x_t . y_j) z_j + e^{L_end - L_t} start^T x_t
// with L the running sum of log_a inside the sequence (inclusive).  x, y have dy columns; z and
// out have dz.  The state sum w_j y_j z_j^T is dy x dz fp32.
struct Run {
  const void *x, *y, *z;
  int Hx, Hy, Hz;        // their heads: head h reads head h / (H / Hx) and so on
  const void *log_a;     // [T, H] of the inputs' type, or fp32 [H] with per_head
  int per_head;
  const float *start;    // [N, H, dy, dz] (or [dz, dy] with start_t), or NULL: zeros
  int start_t;
  float *fin;            // the state after the last step of the run (the same shapes), or NULL
  int fin_t;
  void *out;             // [T, H, dz]
  int out_f32;           // out is fp32 whatever the inputs' type
  int dy, dz;
  int back;              // the backward form
  // Cut sequences: the end state of every piece from a zero start, then the start of every
  // piece (natural [dy][dz] layout), and the sum of its log_a.
  float *piece_state;    // [n_cut * H][dy * dz], NULL when nothing is cut
  double *piece_log;     // [n_cut * H]
  int state_only;        // write piece_state and piece_log, no out
  // For the gradient of log_a: partial dots of every out row with the row of m (Hm heads, dz
  // columns) over the columns of one slice, [slices][T, H] (the tensor-core runs: two halves, [2][H, T]);
  // NULL: none.
  const void *m;
  int Hm;
  float *dots;
  // Tensor-core runs: marks of the state behind every group of kGroup chunks, [slots][H][dy * dz]
  // in the state warps' own order; the forward form writes them, and so does the backward form with
  // mark_dots NULL; else it multiplies its state at the same place with them into mark_dots
  // [slots][H][kMarkDots].  NULL: none.
  float *marks, *mark_dots;
  Cut cut;
  int dtype;
};

cudaError_t launch_plan(const Cut &c, int32_t *seg_off, int32_t *cut_off, int32_t *order, cudaStream_t stream);
// n runs over the same cut: the forward, or the three of the gradients in one launch.
constexpr int kMaxRuns = 3;
cudaError_t launch_join(const Run *r, int n, cudaStream_t stream);
int simt_slices(int dz);
cudaError_t launch_run_simt(const Run *r, int n, cudaStream_t stream);
// The run on the tensor cores (linattn_tc.cu): bf16, dy = dz = 128.  `terms`: bf16 values that
// stand for a weighted row of y in the state's update, 4 (26 bits) or 2 (17).
cudaError_t launch_run_tc(const Run &r, int terms, int32_t *status, cudaStream_t stream);
// The gradients' three runs in one launch, four terms each.
cudaError_t launch_grads_tc(const Run *r, int32_t *status, cudaStream_t stream);
// mark_dots of the marks that the dq and the dk run wrote in one launch.
cudaError_t launch_marks(const float *a, const float *b, float *mark_dots, const Cut &c, cudaStream_t stream);
// dlog_a of the fp32 runs: dots_q (of dq with q), dots_k (of dk with k), and <S_T, dS_T> (S_T
// may be NULL with dS_T).
cudaError_t launch_dlog_simt(const float *dots_q, int nq, const float *dots_k, int nk, const float *S_T,
                             const float *dS_T, int dk, int dv, bool no_start, const void *log_a, const Cut &c, void *dlog,
                             int dtype, cudaStream_t stream);
// dlog_a of the tensor-core runs (linattn_tc.cu).
cudaError_t launch_dlog_tc(const float *dots_q, const float *dots_k, const float *mark_dots, const void *log_a, const Cut &c,
                           bool no_start, void *dlog, cudaStream_t stream);
// out[t, g, :] = sum over the heads of group g of part[t, h, :], for n (1 or 2) of them
cudaError_t launch_group_sum(const float *const *part, void *const *out, int n, const Cut &c, int Hg, int d, int dtype,
                             cudaStream_t stream);

// The largest dynamic shared memory that any launch of a kernel asks for, set once for each device.  It
// belongs to the process: set anew for every call's own size, another thread's would come between the
// setting and the launch.
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kern, int bytes, std::atomic<uint64_t> &ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev <= 63 && (ready.load(std::memory_order_relaxed) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

struct StepProblem {
  const void *q, *k, *v, *log_a;
  float *S;
  const int32_t *state_idx;
  void *o;
  int n_slots, N, H, Hqk, dk, dv, per_head, dtype_in, dtype_out;
};
cudaError_t launch_step(const StepProblem &p, cudaStream_t stream);

}  // namespace lin

// 8-bit checkpoints (ckpt8.cu)
cudaError_t launch_ckpt8_save(const void *x, int8_t *codes, uint8_t *scales, int64_t rows, int cols, int dtype,
                              cudaStream_t stream);
cudaError_t launch_ckpt8_restore(const int8_t *codes, const uint8_t *scales, void *x, int64_t rows, int cols, int dtype,
                                 cudaStream_t stream);
}  // namespace gdn2
