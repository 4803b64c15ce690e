// linattn_api.cu -- the extern "C" entry points of linear attention with a decay per head and of
// the 8-bit checkpoints (include/gdn2.h): argument checks, workspace layout, the order of the
// runs.  Nothing here computes; every step runs in the kernels.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "linattn.cuh"

namespace {

using gdn2::lin::Cut;
using gdn2::lin::Run;

int fail(int code, const char *fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  return gdn2::set_last_error(code, text);
}
void clear_error() { gdn2::set_last_error(0, ""); }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

constexpr size_t kHeader = 256;  // [0] status word

int check_dims(const gdn2_linattn_dims *d, bool one_type) {
  if (!d) return fail(GDN2_ERR_INVALID_ARG, "dims is NULL");
  if (d->reserved != 0) return fail(GDN2_ERR_INVALID_ARG, "dims.reserved must be 0");
  if (d->n_seqs < 1 || d->seq_len < 0 || d->n_heads < 1 || d->n_qk_heads < 1 || d->d_k < 1 || d->d_v < 1)
    return fail(GDN2_ERR_INVALID_ARG, "bad dims (n_seqs=%d seq_len=%d n_heads=%d n_qk_heads=%d d_k=%d d_v=%d)",
                d->n_seqs, d->seq_len, d->n_heads, d->n_qk_heads, d->d_k, d->d_v);
  if (d->n_heads % d->n_qk_heads)
    return fail(GDN2_ERR_INVALID_ARG, "n_heads=%d is not a multiple of n_qk_heads=%d", d->n_heads, d->n_qk_heads);
  if ((d->dtype_in != GDN2_BF16 && d->dtype_in != GDN2_F32) || (d->dtype_out != GDN2_BF16 && d->dtype_out != GDN2_F32))
    return fail(GDN2_ERR_INVALID_ARG, "bad dtype_in=%d / dtype_out=%d", d->dtype_in, d->dtype_out);
  if (d->flags & ~(uint32_t)GDN2_LINATTN_HEAD_DECAY)
    return fail(GDN2_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags & ~(uint32_t)GDN2_LINATTN_HEAD_DECAY);
  if (one_type && d->dtype_in != d->dtype_out)
    return fail(GDN2_ERR_UNSUPPORTED, "dtype_out must be dtype_in here");
  if (d->d_k > 128 || d->d_v > 128)
    return fail(GDN2_ERR_UNSUPPORTED, "no kernel for d_k=%d d_v=%d (both at most 128)", d->d_k, d->d_v);
  return GDN2_OK;
}

int64_t tokens_of(const gdn2_linattn_dims *d, bool packed) {
  return packed ? (int64_t)d->seq_len : (int64_t)d->n_seqs * d->seq_len;
}

// Limits of the launches: 32-bit token numbers, (piece, head) units in one grid dimension.  Loops over
// tokens step up to 2^14 past a sequence's end before they look (the groups of dlog_a, 64 of them 256
// tokens each): the numbers must not wrap there.
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - (1 << 15);
int check_sizes(const gdn2_linattn_dims *d, bool packed) {
  if (tokens_of(d, packed) > kMaxTokens) return fail(GDN2_ERR_UNSUPPORTED, "T_tot must be at most 2^31 - 2^15");
  if ((int64_t)d->n_seqs * d->n_heads >= ((int64_t)1 << 30))
    return fail(GDN2_ERR_UNSUPPORTED, "n_seqs * n_heads must be below 2^30");
  return GDN2_OK;
}

bool tensor_core(const gdn2_linattn_dims *d) { return d->d_k == 128 && d->d_v == 128 && d->dtype_in == GDN2_BF16; }

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms = 148;
  }
  return sms;
}

constexpr int64_t kLeastTc = 512;  // tokens of the shortest pieces of the tensor-core runs

// Where the (sequence, head) units alone leave SMs idle, long sequences are cut into pieces that
// run side by side (each piece's end state first, the join, then the outputs): half as much again
// of the work, spread over all SMs.  The target is the balanced share of tokens per worker; the
// tensor-core run has one worker per SM, the fp32 run (a slice of 64 state columns each) two.
// `runs` of them share the launch.
Cut make_cut(const gdn2_linattn_dims *d, const int32_t *cu, bool packed, int runs = 1) {
  const int sms = sm_count();
  const int64_t T = tokens_of(d, packed);
  const bool tc = tensor_core(d);
  const int slices = tc ? 1 : gdn2::lin::simt_slices(d->d_k < d->d_v ? d->d_k : d->d_v);
  const int64_t workers = tc ? sms : 2 * (int64_t)sms;
  int64_t target = (T * d->n_heads * slices * runs + workers - 1) / workers;
  // Pieces no shorter than what a pass over their states costs: 512 tokens on the tensor cores; in fp32,
  // where a step of 32 tokens is long, one step (4 heads of 32 x 32, 600 tokens: 37 us, from pieces of
  // 64 on 43, of 128 on 78; 3 ragged sequences' gradients, 1201 tokens, 48 x 80: 111, 115 and 162 us).
  const int64_t least = tc ? kLeastTc : gdn2::lin::kTile32;
  if (target < least) target = least;
  Cut c;
  memset(&c, 0, sizeof(c));
  c.cu = cu;
  c.n_seqs = d->n_seqs;
  c.seq_len = d->seq_len;
  c.H = d->n_heads;
  c.t_total = (int)T;
  c.target = target < gdn2::lin::kNoCut / 2 ? (int)target : gdn2::lin::kNoCut;
  c.grain = tc ? gdn2::lin::kChunk : gdn2::lin::kTile32;
  if (packed) {
    // a cut sequence has two targets of tokens at least, and no more pieces than targets
    if (T / c.target < 2) c.target = gdn2::lin::kNoCut;
    c.per_seq = 1;
    c.n_cut = (int)(T / c.target);
    c.n_pieces = d->n_seqs + c.n_cut;
  } else {
    c.per_seq = gdn2::lin::piece_count(d->seq_len, c.target, c.grain);
    c.n_pieces = d->n_seqs * c.per_seq;
    c.n_cut = c.per_seq > 1 ? c.n_pieces : 0;
  }
  c.sorted = packed && c.n_pieces > 1 && c.n_pieces <= gdn2::lin::kMaxSorted && (int64_t)c.n_pieces * c.H * slices * runs > workers;
  return c;
}
bool has_cuts(const Cut &c) { return c.n_cut > 0; }

// The cut's part of a workspace: piece offsets (of all, and of cut sequences) and order, log sums and states.
struct CutLayout {
  size_t off_seg, off_order, off_log, off_state, end;
};
CutLayout cut_layout(const Cut &c, size_t at, size_t state, size_t runs = 1) {
  CutLayout L;
  const size_t units = (size_t)c.n_cut * c.H;
  L.off_seg = at;
  L.off_order = L.off_seg + (units ? up256(2 * ((size_t)c.n_seqs + 1) * sizeof(int32_t)) : 0);
  L.off_log = L.off_order + (c.sorted ? up256((size_t)c.n_pieces * sizeof(int32_t)) : 0);
  L.off_state = L.off_log + up256(runs * units * sizeof(double));
  L.end = L.off_state + up256(runs * units * state * sizeof(float));
  return L;
}

int check_workspace(const void *ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, 256)) return fail(GDN2_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (have < need) return fail(GDN2_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return GDN2_OK;
}

int check_tensors(int64_t tokens, const void *const *p, int n) {
  for (int i = 0; i < n; ++i) {
    if (!p[i] && tokens > 0) return fail(GDN2_ERR_INVALID_ARG, "a per-token pointer is NULL");
    if (!aligned(p[i], 16)) return fail(GDN2_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p[i]);
  }
  return GDN2_OK;
}
int check_log_a(const gdn2_linattn_dims *d, int64_t tokens, const void *log_a) {
  const bool head = (d->flags & GDN2_LINATTN_HEAD_DECAY) != 0;
  if (!log_a && (head || tokens > 0)) return fail(GDN2_ERR_INVALID_ARG, "log_a is NULL");
  if (!aligned(log_a, head || d->dtype_in == GDN2_F32 ? 4 : 2))
    return fail(GDN2_ERR_INVALID_ARG, "log_a pointer %p is misaligned", log_a);
  return GDN2_OK;
}

int cuda_fail(const char *what, cudaError_t e) { return fail(GDN2_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

// Runs over one cut, their cut sequences' piece states and join first: the forward or one of the
// gradients' on the tensor cores, all three of those there (n = 3), or any number in fp32.
// The runs whose state can be a result (the forward's, dv's) take it to the tensor cores in four bf16
// terms, whether or not this call asks for it: out must not depend on that.  The others only feed it
// to bf16 products: two terms.
cudaError_t full_runs(Run *r, int n, int terms, int32_t *status, bool tc, cudaStream_t s) {
  cudaError_t e;
  auto launch = [&](const Run *run) {
    if (!tc) return gdn2::lin::launch_run_simt(run, n, s);
    return n > 1 ? gdn2::lin::launch_grads_tc(run, status, s) : gdn2::lin::launch_run_tc(*run, terms, status, s);
  };
  if (has_cuts(r->cut)) {
    Run first[gdn2::lin::kMaxRuns];
    for (int i = 0; i < n; ++i) {
      first[i] = r[i];
      first[i].state_only = 1;
      first[i].m = nullptr;
    }
    if ((e = launch(first)) != cudaSuccess) return e;
    if ((e = gdn2::lin::launch_join(r, n, s)) != cudaSuccess) return e;
  } else {
    for (int i = 0; i < n; ++i) r[i].piece_state = nullptr;
  }
  return launch(r);
}

cudaError_t prepare(Cut &c, char *ws, const CutLayout &L, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(ws, 0, kHeader, s);
  if (e != cudaSuccess) return e;
  if (c.cu && (has_cuts(c) || c.sorted)) {
    int32_t *off = has_cuts(c) ? reinterpret_cast<int32_t *>(ws + L.off_seg) : nullptr;
    int32_t *cut_off = off ? off + c.n_seqs + 1 : nullptr;
    int32_t *order = c.sorted ? reinterpret_cast<int32_t *>(ws + L.off_order) : nullptr;
    e = gdn2::lin::launch_plan(c, off, cut_off, order, s);
    c.seg_off = off;
    c.cut_off = cut_off;
    c.order = order;
  }
  return e;
}

Run base_run(const gdn2_linattn_dims *d, const void *log_a, const Cut &c, char *ws, const CutLayout &L) {
  Run r;
  memset(&r, 0, sizeof(r));
  r.log_a = log_a;
  r.per_head = (d->flags & GDN2_LINATTN_HEAD_DECAY) != 0;
  r.cut = c;
  r.dtype = d->dtype_in;
  r.piece_log = reinterpret_cast<double *>(ws + L.off_log);
  r.piece_state = reinterpret_cast<float *>(ws + L.off_state);
  return r;
}

// The three runs of the gradients go side by side in one launch in fp32 (3 ragged sequences, 1201
// tokens, 4 heads of 48 x 80: 157 us, one after the other 312).  On the tensor cores that kernel is slower a
// chunk (four terms for all, 97 KB of code), and with gradients of log_a the second run's states are
// written and read again for the products.  It pays where a run alone leaves SMs idle or needs more cuts than
// three: with lengths that are known, where it needs cuts or has units for half of the SMs; with
// cu_seqlens, whose lengths the host does not see, up to two units an SM, since ragged ones leave many
// idle.  With gradients of log_a, only where it takes no cuts (known) or at most two of the shortest
// pieces' tokens an SM.  Times in one launch / one after the other, with gradients of log_a and without, us, 16 heads:
//   one launch taken:  1 x 4096 170/207, 119/183; 3 x 6748 430/500, 346/426; 11 ragged, 9001 tokens 250/373, 189/324;
//                      8 ragged, 8192 342/345, 218/289; 16 ragged, 32768, without 483/727
//   three taken:       8 x 4096 686/483, 516/405; 1 x 20000 593/512; 3 ragged, 20246 678/571; 11 ragged, 30000 881/722;
//                      64 ragged, 32768 875/727, 665/597
//   taken and slower:  8 x 4096 given by cu_seqlens, without gradients of log_a, 516 for 405; 16 ragged, 32768, with
//                      them, 862 for 665
struct BwdPlan {
  bool together;
  Cut cut;
};
BwdPlan plan_bwd(const gdn2_linattn_dims *d, const int32_t *cu, bool packed) {
  BwdPlan p;
  const Cut one = make_cut(d, cu, packed), three = make_cut(d, cu, packed, 3);
  const int64_t units = (int64_t)d->n_seqs * d->n_heads, sms = sm_count();
  const bool light = (d->flags & GDN2_LINATTN_HEAD_DECAY) || tokens_of(d, packed) * d->n_heads <= 2 * kLeastTc * sms;
  p.together = !tensor_core(d) || (packed ? units <= 2 * sms && light
                                          : (has_cuts(one) || 2 * units <= sms) && (light || !has_cuts(three)));
  p.cut = p.together ? three : one;
  return p;
}

// gdn2_linattn_bwd's workspace: header, the cut, for dlog_a the final state (fp32 runs) or the marks of
// one or two runs and their products (tensor-core runs), the per-head parts of dq and dk where heads
// share q and k (one buffer after the other, two together), the dots.
struct BwdLayout {
  CutLayout cut;
  size_t off_fin, off_marks[2], off_mark_dots, off_part[2], off_dq, off_dk, off_restored[3], total;
};
BwdLayout bwd_layout(const gdn2_linattn_dims *d, const BwdPlan &plan, bool ckpt8) {
  BwdLayout L;
  const Cut &c = plan.cut;
  const size_t state = (size_t)d->d_k * d->d_v, T = (size_t)c.t_total, H = d->n_heads, runs = plan.together ? 3 : 1;
  const bool dlog = !(d->flags & GDN2_LINATTN_HEAD_DECAY), tc = tensor_core(d);
  const size_t slots = dlog && tc ? gdn2::lin::mark_slots(c) * H : 0;
  L.cut = cut_layout(c, kHeader, state, runs);
  size_t at = L.cut.end;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  L.off_fin = take(dlog && !tc ? (size_t)d->n_seqs * H * state * sizeof(float) : 0);
  L.off_marks[0] = take(slots * state * sizeof(float));
  L.off_marks[1] = take(plan.together ? slots * state * sizeof(float) : 0);
  L.off_mark_dots = take(slots * gdn2::lin::kMarkDots * sizeof(float));
  const size_t part = d->n_qk_heads < d->n_heads ? T * H * d->d_k * sizeof(float) : 0;
  L.off_part[0] = take(part);
  L.off_part[1] = plan.together ? take(part) : L.off_part[0];
  const size_t dots = dlog ? T * H * (tc ? 2 : gdn2::lin::simt_slices(d->d_k)) * sizeof(float) : 0;
  L.off_dq = take(dots);
  L.off_dk = take(dots);
  const size_t es = d->dtype_in == GDN2_BF16 ? 2 : 4;
  const size_t rows[3] = {T * d->n_qk_heads * d->d_k * es, T * d->n_qk_heads * d->d_k * es, T * H * d->d_v * es};
  for (int i = 0; i < 3; ++i) L.off_restored[i] = take(ckpt8 ? rows[i] : 0);
  L.total = at;
  return L;
}

int bwd_runs(const void *q, const void *k, const void *v, const void *log_a, const float *S0,
             const void *dO, const float *dS_T, void *dq, void *dk, void *dv, void *dlog_a,
             float *dS0, const gdn2_linattn_dims *d, const BwdPlan &plan, char *ws, const BwdLayout &L, cudaStream_t s) {
  const bool tc = tensor_core(d);
  const Cut &c = plan.cut;
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  const int H = d->n_heads, Hq = d->n_qk_heads;
  const bool shared = Hq < H;
  auto floats = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
  float *part_q = floats(L.off_part[0]), *part_k = floats(L.off_part[1]);
  float *dots_q = floats(L.off_dq), *dots_k = floats(L.off_dk), *mark_dots = floats(L.off_mark_dots);
  float *fin = dlog_a && dS_T && !tc ? floats(L.off_fin) : nullptr;
  const bool marks = dlog_a && tc;
  Run runs[3];
  for (int i = 0; i < 3; ++i) {
    runs[i] = base_run(d, log_a, c, ws, L.cut);
    if (plan.together) {
      const size_t units = (size_t)c.n_cut * H;
      runs[i].piece_log += i * units;
      runs[i].piece_state += i * units * d->d_k * d->d_v;
    }
  }
  {  // dq_i = sum_{j <= i} (dO_i . v_j) k_j: the state is the forward's, transposed
    Run &r = runs[0];
    r.x = dO; r.Hx = H; r.y = v; r.Hy = H; r.z = k; r.Hz = Hq;
    r.dy = d->d_v; r.dz = d->d_k;
    r.start = S0; r.start_t = 1; r.fin = fin; r.fin_t = 1;
    r.out = shared ? part_q : dq; r.out_f32 = shared;
    if (dlog_a) { r.m = q; r.Hm = Hq; r.dots = dots_q; }
    if (marks) r.marks = floats(L.off_marks[0]);
  }
  {  // dv_j = sum_{i >= j} (k_j . q_i) dO_i: the state is dLoss/dS
    Run &r = runs[1];
    r.back = 1;
    r.x = k; r.Hx = Hq; r.y = q; r.Hy = Hq; r.z = dO; r.Hz = H;
    r.dy = d->d_k; r.dz = d->d_v;
    r.start = dS_T; r.fin = dS0;
    r.out = dv;
  }
  {  // dk_j = sum_{i >= j} (v_j . dO_i) q_i
    Run &r = runs[2];
    r.back = 1;
    r.x = v; r.Hx = H; r.y = dO; r.Hy = H; r.z = q; r.Hz = Hq;
    r.dy = d->d_v; r.dz = d->d_k;
    r.start = dS_T; r.start_t = 1;
    r.out = shared ? part_k : dk; r.out_f32 = shared;
    if (dlog_a) { r.m = k; r.Hm = Hq; r.dots = dots_k; }
    if (marks) {
      r.marks = floats(L.off_marks[plan.together ? 1 : 0]);
      if (!plan.together) r.mark_dots = mark_dots;
    }
  }
  cudaError_t e;
  const float *parts[2] = {part_q, part_k};
  void *outs[2] = {dq, dk};
  auto sum = [&](int first, int n) {
    return gdn2::lin::launch_group_sum(parts + first, outs + first, n, c, Hq, d->d_k, d->dtype_in, s);
  };
  if (plan.together) {
    if ((e = full_runs(runs, 3, 0, status, tc, s)) != cudaSuccess) return cuda_fail("linattn gradient runs", e);
    if (marks && c.t_total > 0 &&
        (e = gdn2::lin::launch_marks(floats(L.off_marks[0]), floats(L.off_marks[1]), mark_dots, c, s)) != cudaSuccess)
      return cuda_fail("linattn states' products", e);
    if (shared && (e = sum(0, 2)) != cudaSuccess) return cuda_fail("linattn head sums", e);
  } else {
    if ((e = full_runs(&runs[0], 1, 2, status, tc, s)) != cudaSuccess) return cuda_fail("linattn dq run", e);
    if (shared && (e = sum(0, 1)) != cudaSuccess) return cuda_fail("linattn dq head sum", e);
    if ((e = full_runs(&runs[1], 1, 4, status, tc, s)) != cudaSuccess) return cuda_fail("linattn dv run", e);
    if ((e = full_runs(&runs[2], 1, 2, status, tc, s)) != cudaSuccess) return cuda_fail("linattn dk run", e);
    if (shared && (e = sum(1, 1)) != cudaSuccess) return cuda_fail("linattn dk head sum", e);
  }
  if (dlog_a) {
    const int n = gdn2::lin::simt_slices(d->d_k);
    e = tc ? gdn2::lin::launch_dlog_tc(dots_q, dots_k, mark_dots, log_a, c, !S0, dlog_a, s)
           : gdn2::lin::launch_dlog_simt(dots_q, n, dots_k, n, fin, dS_T, d->d_k, d->d_v, !S0, log_a, c, dlog_a, d->dtype_in, s);
    if (e != cudaSuccess) return cuda_fail("linattn dlog_a", e);
  }
  return GDN2_OK;
}

int check_bwd(const gdn2_linattn_dims *d, const void *log_a, const float *S0, const int32_t *cu, const void *dO,
              const float *dS_T, void *dq, void *dk, void *dv, void *dlog_a, float *dS0) {
  const int64_t T = tokens_of(d, cu != nullptr);
  const void *rows[4] = {dO, dq, dk, dv};
  int rc = check_tensors(T, rows, 4);
  if (!rc) rc = check_log_a(d, T, log_a);
  if (rc) return rc;
  const bool head = (d->flags & GDN2_LINATTN_HEAD_DECAY) != 0;
  if (head && dlog_a) return fail(GDN2_ERR_INVALID_ARG, "dlog_a must be NULL with GDN2_LINATTN_HEAD_DECAY");
  if (!head && !dlog_a && T > 0) return fail(GDN2_ERR_INVALID_ARG, "dlog_a is NULL");
  if (!aligned(dlog_a, d->dtype_in == GDN2_F32 ? 4 : 2)) return fail(GDN2_ERR_INVALID_ARG, "dlog_a is misaligned");
  if (!aligned(S0, 16) || !aligned(dS_T, 16) || !aligned(dS0, 16))
    return fail(GDN2_ERR_INVALID_ARG, "S0, dS_T and dS0 must be 16-byte aligned");
  if (!aligned(cu, 4)) return fail(GDN2_ERR_INVALID_ARG, "cu_seqlens is misaligned");
  return GDN2_OK;
}

// Outputs are written while inputs are still read, and not in one order for all sizes.
int check_apart(const void *const *out, int n_out, const void *const *in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    if (!out[i]) continue;
    for (int j = 0; j < i; ++j)
      if (out[i] == out[j]) return fail(GDN2_ERR_INVALID_ARG, "two outputs share the address %p", out[i]);
    for (int j = 0; j < n_in; ++j)
      if (out[i] == in[j]) return fail(GDN2_ERR_INVALID_ARG, "an output has an input's address %p", out[i]);
  }
  return GDN2_OK;
}

int check_ckpt8(const void *x, const int8_t *codes, const uint8_t *scales, int64_t rows, int32_t cols, int32_t dtype) {
  if (rows < 0 || cols < 1) return fail(GDN2_ERR_INVALID_ARG, "bad shape (rows=%lld cols=%d)", (long long)rows, cols);
  if (dtype != GDN2_BF16 && dtype != GDN2_F32) return fail(GDN2_ERR_INVALID_ARG, "bad dtype=%d", dtype);
  if (rows > ((int64_t)1 << 33) / ((cols + 31) / 32))
    return fail(GDN2_ERR_UNSUPPORTED, "more than 2^33 blocks of 32 values");
  if (rows > 0 && (!x || !codes || !scales)) return fail(GDN2_ERR_INVALID_ARG, "x, codes and scales must be non-NULL");
  if (!aligned(x, 16) || !aligned(codes, 16))
    return fail(GDN2_ERR_INVALID_ARG, "x and codes must be 16-byte aligned");
  return GDN2_OK;
}

}  // namespace

extern "C" {

size_t gdn2_linattn_fwd_workspace_size(const gdn2_linattn_dims *dims, int32_t packed) {
  clear_error();
  if (check_dims(dims, true) || check_sizes(dims, packed != 0)) return 0;
  const Cut c = make_cut(dims, nullptr, packed != 0);
  return cut_layout(c, kHeader, (size_t)dims->d_k * dims->d_v).end;
}

int gdn2_linattn_fwd(const void *q, const void *k, const void *v, const void *log_a, const float *S0,
                     const int32_t *cu_seqlens, void *o, float *S_T, const gdn2_linattn_dims *dims, void *workspace,
                     size_t workspace_bytes, gdn2_stream_t stream) {
  clear_error();
  int rc = check_dims(dims, true);
  if (!rc) rc = check_sizes(dims, cu_seqlens != nullptr);
  if (rc) return rc;
  const int64_t T = tokens_of(dims, cu_seqlens != nullptr);
  const void *rows[4] = {q, k, v, o};
  rc = check_tensors(T, rows, 4);
  if (!rc) rc = check_log_a(dims, T, log_a);
  if (rc) return rc;
  if (!aligned(S0, 16) || !aligned(S_T, 16)) return fail(GDN2_ERR_INVALID_ARG, "S0 / S_T must be 16-byte aligned");
  if (!aligned(cu_seqlens, 4)) return fail(GDN2_ERR_INVALID_ARG, "cu_seqlens is misaligned");
  Cut c = make_cut(dims, cu_seqlens, cu_seqlens != nullptr);
  const CutLayout L = cut_layout(c, kHeader, (size_t)dims->d_k * dims->d_v);
  rc = check_workspace(workspace, workspace_bytes, L.end);
  const void *in[5] = {q, k, v, log_a, cu_seqlens}, *out[2] = {o, S_T};
  if (!rc) rc = check_apart(out, 2, in, 5);
  if (!rc) rc = check_apart(out, 1, reinterpret_cast<const void *const *>(&S0), 1);  // S_T may be S0
  if (rc) return rc;
  char *ws = static_cast<char *>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = prepare(c, ws, L, s);
  if (e != cudaSuccess) return cuda_fail("linattn workspace", e);
  Run r = base_run(dims, log_a, c, ws, L);
  r.x = q; r.Hx = dims->n_qk_heads; r.y = k; r.Hy = dims->n_qk_heads; r.z = v; r.Hz = dims->n_heads;
  r.dy = dims->d_k; r.dz = dims->d_v;
  r.start = S0; r.fin = S_T; r.out = o;
  if ((e = full_runs(&r, 1, 4, reinterpret_cast<int32_t *>(ws), tensor_core(dims), s)) != cudaSuccess) return cuda_fail("linattn run", e);
  return GDN2_OK;
}

int gdn2_linattn_step(const void *q, const void *k, const void *v, const void *log_a, float *S, int32_t n_slots,
                      const int32_t *state_idx, void *o, const gdn2_linattn_dims *dims, gdn2_stream_t stream) {
  clear_error();
  int rc = check_dims(dims, false);
  if (!rc) rc = check_sizes(dims, false);
  if (rc) return rc;
  if (dims->seq_len != 1) return fail(GDN2_ERR_INVALID_ARG, "seq_len must be 1 (got %d)", dims->seq_len);
  const void *rows[4] = {q, k, v, o};
  rc = check_tensors(1, rows, 4);
  if (!rc) rc = check_log_a(dims, 1, log_a);
  if (rc) return rc;
  if (!S || !aligned(S, 16)) return fail(GDN2_ERR_INVALID_ARG, "S must be non-NULL and 16-byte aligned");
  if (state_idx && n_slots < 1) return fail(GDN2_ERR_INVALID_ARG, "n_slots must be at least 1 (got %d)", n_slots);
  if (!aligned(state_idx, 4)) return fail(GDN2_ERR_INVALID_ARG, "state_idx is misaligned");
  const void *in[5] = {q, k, v, log_a, state_idx}, *out[2] = {o, S};
  rc = check_apart(out, 2, in, 5);
  if (rc) return rc;
  gdn2::lin::StepProblem p;
  memset(&p, 0, sizeof(p));
  p.q = q; p.k = k; p.v = v; p.log_a = log_a; p.S = S; p.state_idx = state_idx; p.o = o;
  p.n_slots = n_slots; p.N = dims->n_seqs; p.H = dims->n_heads; p.Hqk = dims->n_qk_heads;
  p.dk = dims->d_k; p.dv = dims->d_v;
  p.per_head = (dims->flags & GDN2_LINATTN_HEAD_DECAY) != 0;
  p.dtype_in = dims->dtype_in; p.dtype_out = dims->dtype_out;
  const cudaError_t e = gdn2::lin::launch_step(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail("linattn step launch", e);
  return GDN2_OK;
}

size_t gdn2_linattn_bwd_workspace_size(const gdn2_linattn_dims *dims, int32_t packed) {
  clear_error();
  if (check_dims(dims, true) || check_sizes(dims, packed != 0)) return 0;
  return bwd_layout(dims, plan_bwd(dims, nullptr, packed != 0), false).total;
}

int gdn2_linattn_bwd(const void *q, const void *k, const void *v, const void *log_a, const float *S0,
                     const int32_t *cu_seqlens, const void *dO, const float *dS_T, void *dq, void *dk, void *dv,
                     void *dlog_a, float *dS0, const gdn2_linattn_dims *dims, void *workspace, size_t workspace_bytes,
                     gdn2_stream_t stream) {
  clear_error();
  int rc = check_dims(dims, true);
  if (!rc) rc = check_sizes(dims, cu_seqlens != nullptr);
  if (rc) return rc;
  const void *rows[3] = {q, k, v};
  rc = check_tensors(tokens_of(dims, cu_seqlens != nullptr), rows, 3);
  if (!rc) rc = check_bwd(dims, log_a, S0, cu_seqlens, dO, dS_T, dq, dk, dv, dlog_a, dS0);
  if (rc) return rc;
  BwdPlan plan = plan_bwd(dims, cu_seqlens, cu_seqlens != nullptr);
  const BwdLayout L = bwd_layout(dims, plan, false);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  const void *in[8] = {q, k, v, log_a, dO, S0, dS_T, cu_seqlens}, *out[5] = {dq, dk, dv, dlog_a, dS0};
  if (!rc) rc = check_apart(out, 5, in, 8);
  if (rc) return rc;
  char *ws = static_cast<char *>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = prepare(plan.cut, ws, L.cut, s);
  if (e != cudaSuccess) return cuda_fail("linattn workspace", e);
  return bwd_runs(q, k, v, log_a, S0, dO, dS_T, dq, dk, dv, dlog_a, dS0, dims, plan, ws, L, s);
}

int gdn2_ckpt8_save(const void *x, int8_t *codes, uint8_t *scales, int64_t rows, int32_t cols, int32_t dtype,
                    gdn2_stream_t stream) {
  clear_error();
  int rc = check_ckpt8(x, codes, scales, rows, cols, dtype);
  if (rc || rows == 0) return rc;
  const void *out[2] = {codes, scales}, *in[1] = {x};
  rc = check_apart(out, 2, in, 1);
  if (rc) return rc;
  const cudaError_t e = gdn2::launch_ckpt8_save(x, codes, scales, rows, cols, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN2_OK : cuda_fail("ckpt8 save launch", e);
}

int gdn2_ckpt8_restore(const int8_t *codes, const uint8_t *scales, void *x, int64_t rows, int32_t cols, int32_t dtype,
                       gdn2_stream_t stream) {
  clear_error();
  int rc = check_ckpt8(x, codes, scales, rows, cols, dtype);
  if (rc || rows == 0) return rc;
  const void *out[1] = {x}, *in[2] = {codes, scales};
  rc = check_apart(out, 1, in, 2);
  if (rc) return rc;
  const cudaError_t e =
      gdn2::launch_ckpt8_restore(codes, scales, x, rows, cols, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN2_OK : cuda_fail("ckpt8 restore launch", e);
}

size_t gdn2_linattn_bwd_ckpt8_workspace_size(const gdn2_linattn_dims *dims, int32_t packed) {
  clear_error();
  if (check_dims(dims, true) || check_sizes(dims, packed != 0)) return 0;
  return bwd_layout(dims, plan_bwd(dims, nullptr, packed != 0), true).total;
}

int gdn2_linattn_bwd_ckpt8(const int8_t *q_codes, const uint8_t *q_scales, const int8_t *k_codes,
                           const uint8_t *k_scales, const int8_t *v_codes, const uint8_t *v_scales, const void *log_a,
                           const float *S0, const int32_t *cu_seqlens, const void *dO, const float *dS_T, void *dq,
                           void *dk, void *dv, void *dlog_a, float *dS0, const gdn2_linattn_dims *dims, void *workspace,
                           size_t workspace_bytes, gdn2_stream_t stream) {
  clear_error();
  int rc = check_dims(dims, true);
  if (!rc) rc = check_sizes(dims, cu_seqlens != nullptr);
  if (rc) return rc;
  const int64_t T = tokens_of(dims, cu_seqlens != nullptr);
  const void *rows[3] = {q_codes, k_codes, v_codes};
  rc = check_tensors(T, rows, 3);
  if (rc) return rc;
  if (T > 0 && (!q_scales || !k_scales || !v_scales)) return fail(GDN2_ERR_INVALID_ARG, "a scales pointer is NULL");
  rc = check_bwd(dims, log_a, S0, cu_seqlens, dO, dS_T, dq, dk, dv, dlog_a, dS0);
  if (rc) return rc;
  BwdPlan plan = plan_bwd(dims, cu_seqlens, cu_seqlens != nullptr);
  const BwdLayout L = bwd_layout(dims, plan, true);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  const void *in[11] = {q_codes, q_scales, k_codes, k_scales, v_codes, v_scales, log_a, dO, S0, dS_T, cu_seqlens};
  const void *out[5] = {dq, dk, dv, dlog_a, dS0};
  if (!rc) rc = check_apart(out, 5, in, 11);
  if (rc) return rc;
  char *ws = static_cast<char *>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = prepare(plan.cut, ws, L.cut, s);
  if (e != cudaSuccess) return cuda_fail("linattn workspace", e);
  const int8_t *codes[3] = {q_codes, k_codes, v_codes};
  const uint8_t *scales[3] = {q_scales, k_scales, v_scales};
  for (int i = 0; i < 3 && T > 0; ++i) {
    e = gdn2::launch_ckpt8_restore(codes[i], scales[i], ws + L.off_restored[i],
                                   T * (i < 2 ? dims->n_qk_heads : dims->n_heads), i < 2 ? dims->d_k : dims->d_v,
                                   dims->dtype_in, s);
    if (e != cudaSuccess) return cuda_fail("ckpt8 restore launch", e);
  }
  return bwd_runs(ws + L.off_restored[0], ws + L.off_restored[1], ws + L.off_restored[2], log_a, S0, dO,
                  dS_T, dq, dk, dv, dlog_a, dS0, dims, plan, ws, L, s);
}

}  // extern "C"
