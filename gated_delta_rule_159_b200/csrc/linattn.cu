// linattn.cu -- linear attention with a decay per head on the CUDA cores: the run for fp32 inputs
// and for head sizes the tensor-core run does not take, the single-token step, and the helpers
// both runs share (the cut plan, the join of the pieces, the gradient of log_a, head sums).
#include <type_traits>

#include "linattn.cuh"

namespace gdn2 {
namespace lin {
namespace {

// ---------------------------------------------------------------- plan and join
// Exclusive running count of pieces over the sequences (one block).
__global__ void __launch_bounds__(1024) plan_kernel(Cut c, int32_t *seg_off) {
  __shared__ int warp_sum[32];
  __shared__ int base;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) base = 0;
  for (int n0 = 0; n0 < c.n_seqs; n0 += 1024) {
    const int n = n0 + threadIdx.x;
    int v = 0;
    if (n < c.n_seqs) {
      int t0, len;
      seq_bounds(c, n, &t0, &len);
      v = piece_count(len, c.target);
    }
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = base;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    // n_pieces bounds the count for offsets in order; anything else is cut back to it
    if (n < c.n_seqs) seg_off[n] = min(before + incl - v, c.n_pieces);
    __syncthreads();
    if (threadIdx.x == 1023) {
      base = before + incl;
      if (n0 + 1024 >= c.n_seqs) seg_off[c.n_seqs] = min(base, c.n_pieces);
    }
    __syncthreads();
  }
}

// piece_state[s] holds the end state of piece s from zero; in its place comes the state piece s
// starts from: start_{s+1} = e^{sum log_a of s} start_s + end_s (from the last piece down in a
// backward run).  Elementwise in the state, serial over the pieces; the loads of the next piece
// do not depend on the sum, so four are kept in flight.
__global__ void __launch_bounds__(256) join_kernel(Run r) {
  const int size = r.dy * r.dz, H = r.cut.H;
  const int n = blockIdx.x / H, h = blockIdx.x % H;
  const int first = r.cut.seg_off ? r.cut.seg_off[n] : n * r.cut.per_seq;
  const int count = r.cut.seg_off ? r.cut.seg_off[n + 1] - first : r.cut.per_seq;
  if (count < 2) return;
  const int e = blockIdx.y * 256 + threadIdx.x;
  if (e >= size) return;
  float cur = 0.f;
  if (r.start) {
    const float *s0 = r.start + (size_t)(n * H + h) * size;
    cur = r.start_t ? s0[(size_t)(e % r.dz) * r.dy + e / r.dz] : s0[e];
  }
  const int64_t unit0 = (int64_t)first * H + h;
  for (int i0 = 0; i0 < count; i0 += 4) {
    float got[4], g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = r.back ? count - 1 - (i0 + j) : i0 + j;
      if (i0 + j < count - 1) {
        got[j] = r.piece_state[(unit0 + (int64_t)s * H) * size + e];
        const double l = r.piece_log[unit0 + (int64_t)s * H];
        const float hi = (float)l;
        g[j] = expf(hi) * (1.f + (float)(l - (double)hi));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i0 + j >= count) break;
      const int s = r.back ? count - 1 - (i0 + j) : i0 + j;
      r.piece_state[(unit0 + (int64_t)s * H) * size + e] = cur;
      if (i0 + j < count - 1) cur = fmaf(g[j], cur, got[j]);
    }
  }
}

// ---------------------------------------------------------------- the run, token by token in fp32
// The columns of the state do not mix: a warp owns 16 of them and all dy rows, 8 lanes x R rows
// by 4 lanes x 4 columns, in registers.  Per token a lane updates R x 4 elements and multiplies
// them by x; four shuffles sum each column over its 8 lanes.  4 dy dz FMA-class operations a token
// on the CUDA cores bound it (and the chain of tokens, where there are few units).
constexpr int TB = 32;     // tokens staged at a time
constexpr int WARPS = 2;   // warps of a block
constexpr int COLS = 16 * WARPS;

// A fixed decay's rounding is the same at every token, and a state that keeps n tokens would be off
// by n of them: the product with the state takes the decay in two parts.
__device__ __forceinline__ float2 split_exp(float la) {
  const double a = exp((double)la);
  const float hi = (float)a;
  return make_float2(hi, (float)(a - (double)hi));
}

template <int R>
__device__ __forceinline__ int row_of(int rg, int r) {
  constexpr int V = R < 4 ? R : 4;
  return (r / V) * (8 * V) + rg * V + r % V;
}

template <typename T, int R>
__global__ void __launch_bounds__(32 * WARPS) run_kernel(Run p) {
  constexpr int DP = 8 * R;
  constexpr int V = R < 4 ? R : 4;
  __shared__ __align__(16) float xs[TB][DP];
  __shared__ __align__(16) float ys[TB][DP];
  __shared__ __align__(16) float zs[TB][COLS];
  __shared__ float ms[TB][COLS];
  __shared__ float2 decay[TB];  // e^{log_a} as a sum of two floats
  __shared__ float raw[TB];
  __shared__ float part[TB][WARPS];
  const int H = p.cut.H, unit = blockIdx.x, h = unit % H;
  Piece pc;
  if (!find_piece(p.cut, unit / H, &pc)) return;
  if (p.state_only && (pc.count < 2 || pc.s == (p.back ? 0 : pc.count - 1))) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rg = lane & 7, cg = lane >> 3;
  const int col0 = blockIdx.y * COLS, wcol = warp * 16 + cg * 4;
  const T *x = static_cast<const T *>(p.x), *y = static_cast<const T *>(p.y), *z = static_cast<const T *>(p.z);
  const T *m = static_cast<const T *>(p.m);
  const int hx = h / (H / p.Hx), hy = h / (H / p.Hy), hz = h / (H / p.Hz), hm = p.m ? h / (H / p.Hm) : 0;

  float S[R][4];
  const float *start = nullptr;
  bool st = false;
  const size_t state = (size_t)p.dy * p.dz;
  if (!p.state_only) {
    if (p.piece_state && pc.count > 1) {
      start = p.piece_state + (size_t)unit * state;
    } else if (p.start) {
      start = p.start + ((size_t)pc.n * H + h) * state;
      st = p.start_t;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = row_of<R>(rg, r), col = col0 + wcol + c;
      S[r][c] = start && row < p.dy && col < p.dz ? start[st ? (size_t)col * p.dy + row : (size_t)row * p.dz + col]
                                                  : 0.f;
    }

  const float fixed = p.per_head ? static_cast<const float *>(p.log_a)[h] : 0.f;
  double logs = 0.0;
  const int tiles = (pc.len + TB - 1) / TB;
  float2 carry = make_float2(1.f, 0.f);  // backward: the decay of the token after this one, applied before its update
  for (int it = 0; it < tiles; ++it) {
    const int tile = p.back ? tiles - 1 - it : it;
    const int t0 = tile * TB, cnt = min(TB, pc.len - t0);
    __syncthreads();
    for (int i = tid; i < cnt * DP; i += 32 * WARPS) {
      const int t = i / DP, c = i % DP;
      const bool in = c < p.dy;
      const size_t tok = (size_t)(pc.t0 + t0 + t);
      if (!p.state_only) xs[t][c] = in ? to_f32<T>(x[(tok * p.Hx + hx) * p.dy + c]) : 0.f;
      ys[t][c] = in ? to_f32<T>(y[(tok * p.Hy + hy) * p.dy + c]) : 0.f;
    }
    for (int i = tid; i < cnt * COLS; i += 32 * WARPS) {
      const int t = i / COLS, c = i % COLS;
      const bool in = col0 + c < p.dz;
      const size_t tok = (size_t)(pc.t0 + t0 + t);
      zs[t][c] = in ? to_f32<T>(z[(tok * p.Hz + hz) * p.dz + col0 + c]) : 0.f;
      if (m) ms[t][c] = in ? to_f32<T>(m[(tok * p.Hm + hm) * p.dz + col0 + c]) : 0.f;
    }
    for (int t = tid; t < cnt; t += 32 * WARPS) {
      const float la = p.per_head ? fixed
                                  : to_f32<T>(static_cast<const T *>(p.log_a)[(size_t)(pc.t0 + t0 + t) * H + h]);
      raw[t] = fmaxf(la, kMinLog);
      decay[t] = split_exp(raw[t]);
    }
    __syncthreads();
    if (p.state_only && blockIdx.y == 0 && tid == 0)
      for (int t = 0; t < cnt; ++t) logs += (double)raw[t];
    for (int i = 0; i < cnt; ++i) {
      const int t = p.back ? cnt - 1 - i : i;
      const float2 mine = decay[t];
      const float2 a = p.back ? carry : mine;
      carry = mine;
      const float4 z4 = *reinterpret_cast<const float4 *>(&zs[t][wcol]);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int rv = 0; rv < R / V; ++rv) {
        float yv[V], xv[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          yv[j] = ys[t][rv * 8 * V + rg * V + j];
          xv[j] = p.state_only ? 0.f : xs[t][rv * 8 * V + rg * V + j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float(&s)[4] = S[rv * V + j];
          s[0] = fmaf(a.x, s[0], fmaf(a.y, s[0], yv[j] * z4.x));
          s[1] = fmaf(a.x, s[1], fmaf(a.y, s[1], yv[j] * z4.y));
          s[2] = fmaf(a.x, s[2], fmaf(a.y, s[2], yv[j] * z4.z));
          s[3] = fmaf(a.x, s[3], fmaf(a.y, s[3], yv[j] * z4.w));
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c] = fmaf(xv[j], s[c], acc[c]);
        }
      }
      if (p.state_only) continue;
      // sum over the 8 row lanes: each step halves the columns a lane keeps, the last joins halves
      const bool b0 = rg & 1, b1 = rg & 2;
      float k0 = b0 ? acc[2] : acc[0], k1 = b0 ? acc[3] : acc[1];
      k0 += __shfl_xor_sync(0xffffffffu, b0 ? acc[0] : acc[2], 1);
      k1 += __shfl_xor_sync(0xffffffffu, b0 ? acc[1] : acc[3], 1);
      float o = b1 ? k1 : k0;
      o += __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2);
      o += __shfl_xor_sync(0xffffffffu, o, 4);
      const int c = wcol + (b0 ? 2 : 0) + (b1 ? 1 : 0), col = col0 + c;
      if (rg < 4 && col < p.dz) {
        const size_t at = ((size_t)(pc.t0 + t0 + t) * H + h) * p.dz + col;
        if (p.out_f32) static_cast<float *>(p.out)[at] = o;
        else static_cast<T *>(p.out)[at] = from_f32<T>(o);
      }
      if (m) {
        float d = rg < 4 ? o * ms[t][c] : 0.f;
#pragma unroll
        for (int b = 16; b; b >>= 1) d += __shfl_xor_sync(0xffffffffu, d, b);
        if (lane == 0) part[t][warp] = d;
      }
    }
    if (m && !p.state_only) {
      __syncthreads();
      for (int t = tid; t < cnt; t += 32 * WARPS) {
        float d = 0.f;
        for (int w = 0; w < WARPS; ++w) d += part[t][w];
        p.dots[((size_t)blockIdx.y * p.cut.t_total + (pc.t0 + t0 + t)) * H + h] = d;
      }
    }
  }
  if (p.back)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[r][c] = fmaf(carry.x, S[r][c], carry.y * S[r][c]);

  float *dst = nullptr;
  bool dt = false;
  if (p.state_only) {
    dst = p.piece_state + (size_t)unit * state;
    if (blockIdx.y == 0 && tid == 0) p.piece_log[unit] = logs;
  } else if (p.fin && pc.s == (p.back ? 0 : pc.count - 1)) {
    dst = p.fin + ((size_t)pc.n * H + h) * state;
    dt = p.fin_t;
  }
  if (!dst) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = row_of<R>(rg, r), col = col0 + wcol + c;
      if (row < p.dy && col < p.dz) dst[dt ? (size_t)col * p.dy + row : (size_t)row * p.dz + col] = S[r][c];
    }
}

template <typename T>
cudaError_t launch_run_t(const Run &r, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)r.cut.n_pieces * r.cut.H), (unsigned)simt_slices(r.dz));
  const int R = (r.dy + 7) / 8;
  if (R <= 2) run_kernel<T, 2><<<grid, 32 * WARPS, 0, s>>>(r);
  else if (R <= 4) run_kernel<T, 4><<<grid, 32 * WARPS, 0, s>>>(r);
  else if (R <= 8) run_kernel<T, 8><<<grid, 32 * WARPS, 0, s>>>(r);
  else run_kernel<T, 16><<<grid, 32 * WARPS, 0, s>>>(r);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- gradient of log_a
// a_t stands once in every pair (i, j) with j < t <= i:
//   dlog_a_t = sum_{i >= t} (q_i . dq_i - k_i . dk_i) + <S_T, dS_T>,
// a suffix sum over the sequence, held in fp64: its terms cancel.
constexpr int kScan = 256;
template <typename T>
__global__ void __launch_bounds__(kScan) dlog_kernel(const float *dq, int nq, const float *dk, int nk,
                                                     const float *S_T, const float *dS_T, int size, Cut c, T *dlog) {
  __shared__ double sums[kScan / 32];
  const int H = c.H, n = blockIdx.x / H, h = blockIdx.x % H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int t0, len;
  seq_bounds(c, n, &t0, &len);
  double carry = 0.0;
  if (dS_T && S_T) {
    const size_t at = (size_t)blockIdx.x * size;
    double v = 0.0;
    for (int i = threadIdx.x; i < size; i += kScan) v += (double)S_T[at + i] * (double)dS_T[at + i];
    for (int b = 16; b; b >>= 1) v += __shfl_xor_sync(0xffffffffu, v, b);
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    for (int w = 0; w < kScan / 32; ++w) carry += sums[w];
  }
  for (int done = 0; done < len; done += kScan) {
    const int t = len - 1 - done - (int)threadIdx.x;  // thread 0 has the latest token
    double v = 0.0;
    const size_t at = (size_t)(t0 + t) * H + h, slice = (size_t)c.t_total * H;
    if (t >= 0) {
      for (int i = 0; i < nq; ++i) v += (double)dq[i * slice + at];
      for (int i = 0; i < nk; ++i) v -= (double)dk[i * slice + at];
    }
    double incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    double before = carry;
    for (int w = 0; w < warp; ++w) before += sums[w];
    if (t >= 0) dlog[at] = from_f32<T>((float)(before + incl));
    for (int w = 0; w < kScan / 32; ++w) carry += sums[w];
  }
}

// ---------------------------------------------------------------- heads that share q and k
// A thread sums VEC columns: 16-byte loads of the parts, which are most of what it moves.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) group_sum_kernel(const float *part, T *out, int64_t total, int share, int d,
                                                        const int32_t *cu, int n_seqs, int Hg) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;  // over [T, Hg, d]
  if (i >= total) return;
  const int64_t row = i / d, t = row / Hg;
  if (cu && (t < cu[0] || t >= cu[n_seqs])) return;  // outside every sequence: left as it was
  const float *p = part + row * share * d + (i - row * d);
  float v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = 0.f;
  for (int s = 0; s < share; ++s) {
    if constexpr (VEC == 4) {
      const float4 f = __ldcs(reinterpret_cast<const float4 *>(p + (int64_t)s * d));
      v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    } else {
      v[0] += p[(int64_t)s * d];
    }
  }
  if constexpr (VEC == 4 && sizeof(T) == 2)
    *reinterpret_cast<uint2 *>(out + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else if constexpr (VEC == 4)
    *reinterpret_cast<float4 *>(out + i) = make_float4(v[0], v[1], v[2], v[3]);
  else
    out[i] = from_f32<T>(v[0]);
}

// ---------------------------------------------------------------- single-token step
// The state is read once and written once: 8 bytes an element against 4 operations, so HBM bounds
// it.  A block per (row, head); a thread owns VEC columns and every nrg-th row, and requests eight
// rows before it uses the first, so a block keeps 32 KB and more in flight.
constexpr int kStepThreads = 256;
template <typename T, typename TO, int VEC>
__global__ void __launch_bounds__(kStepThreads) step_kernel(StepProblem p) {
  __shared__ float qs[128], ks[128];
  __shared__ float2 decay;
  __shared__ __align__(16) float red[kStepThreads * VEC];
  const int row = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x;
  TO *o = static_cast<TO *>(p.o) + (size_t)blockIdx.x * p.dv;
  const int slot = p.state_idx ? p.state_idx[row] : row;
  if (p.state_idx && (slot < 0 || slot >= p.n_slots)) {  // a padding row
    for (int c = tid; c < p.dv; c += kStepThreads) o[c] = from_f32<TO>(0.f);
    return;
  }
  const int hq = h / (p.H / p.Hqk);
  const T *q = static_cast<const T *>(p.q) + ((size_t)row * p.Hqk + hq) * p.dk;
  const T *k = static_cast<const T *>(p.k) + ((size_t)row * p.Hqk + hq) * p.dk;
  const T *v = static_cast<const T *>(p.v) + (size_t)blockIdx.x * p.dv;
  float *S = p.S + ((size_t)slot * p.H + h) * p.dk * p.dv;
  const int nc = (p.dv + VEC - 1) / VEC, nrg = kStepThreads / nc;
  const int cg = tid % nc, rg = tid / nc;
  const bool live = rg < nrg;
  float vv[VEC], acc[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    vv[c] = live ? to_f32<T>(v[cg * VEC + c]) : 0.f;
    acc[c] = 0.f;
  }
  if (tid < p.dk) {
    qs[tid] = to_f32<T>(q[tid]);
    ks[tid] = to_f32<T>(k[tid]);
  }
  if (tid == kStepThreads - 1)
    decay = split_exp(p.per_head ? static_cast<const float *>(p.log_a)[h]
                                 : to_f32<T>(static_cast<const T *>(p.log_a)[blockIdx.x]));
  __syncthreads();
  const float2 a = decay;
  if (live) {
    float *mine = S + cg * VEC;
    for (int r0 = rg; r0 < p.dk; r0 += 8 * nrg) {
      float s[8][VEC];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r0 + j * nrg;
        if (r < p.dk) {
          if constexpr (VEC == 4) {
            const float4 f = __ldcs(reinterpret_cast<const float4 *>(mine + (size_t)r * p.dv));
            s[j][0] = f.x; s[j][1] = f.y; s[j][2] = f.z; s[j][3] = f.w;
          } else {
            s[j][0] = mine[(size_t)r * p.dv];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r0 + j * nrg;
        if (r < p.dk) {
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            s[j][c] = fmaf(a.x, s[j][c], fmaf(a.y, s[j][c], ks[r] * vv[c]));
            acc[c] = fmaf(qs[r], s[j][c], acc[c]);
          }
          if constexpr (VEC == 4)
            __stcs(reinterpret_cast<float4 *>(mine + (size_t)r * p.dv), make_float4(s[j][0], s[j][1], s[j][2], s[j][3]));
          else
            mine[(size_t)r * p.dv] = s[j][0];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) red[(rg * nc + cg) * VEC + c] = acc[c];
  }
  __syncthreads();
  for (int c = tid; c < p.dv; c += kStepThreads) {
    float sum = 0.f;
    for (int g = 0; g < nrg; ++g) sum += red[g * nc * VEC + c];
    o[c] = from_f32<TO>(sum);
  }
}

template <typename T, typename TO>
cudaError_t launch_step_t(const StepProblem &p, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.N * p.H);
  if (p.dv % 4 == 0) step_kernel<T, TO, 4><<<grid, kStepThreads, 0, s>>>(p);
  else step_kernel<T, TO, 1><<<grid, kStepThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_plan(const Cut &c, int32_t *seg_off, cudaStream_t s) {
  plan_kernel<<<1, 1024, 0, s>>>(c, seg_off);
  return cudaGetLastError();
}

cudaError_t launch_join(const Run &r, cudaStream_t s) {
  const dim3 grid((unsigned)(r.cut.n_seqs * r.cut.H), (unsigned)((r.dy * r.dz + 255) / 256));
  join_kernel<<<grid, 256, 0, s>>>(r);
  return cudaGetLastError();
}

int simt_slices(int dz) { return (dz + COLS - 1) / COLS; }

cudaError_t launch_run_simt(const Run &r, cudaStream_t s) {
  return r.dtype == GDN2_BF16 ? launch_run_t<__nv_bfloat16>(r, s) : launch_run_t<float>(r, s);
}

cudaError_t launch_dlog_simt(const float *dots_q, int nq, const float *dots_k, int nk, const float *S_T,
                             const float *dS_T, int dk, int dv, const Cut &c, void *dlog, int dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)(c.n_seqs * c.H);
  if (dtype == GDN2_BF16)
    dlog_kernel<<<grid, kScan, 0, s>>>(dots_q, nq, dots_k, nk, S_T, dS_T, dk * dv, c, static_cast<__nv_bfloat16 *>(dlog));
  else
    dlog_kernel<<<grid, kScan, 0, s>>>(dots_q, nq, dots_k, nk, S_T, dS_T, dk * dv, c, static_cast<float *>(dlog));
  return cudaGetLastError();
}

cudaError_t launch_group_sum(const float *part, void *out, const Cut &c, int Hg, int d, int dtype, cudaStream_t s) {
  const int64_t total = (int64_t)c.t_total * Hg * d;
  const int share = c.H / Hg;
  if (total == 0) return cudaSuccess;
  const int vec = d % 4 == 0 ? 4 : 1;
  const unsigned grid = (unsigned)((total + 256 * vec - 1) / (256 * vec));
  auto go = [&](auto *o) {
    using T = std::remove_pointer_t<decltype(o)>;
    if (vec == 4) group_sum_kernel<T, 4><<<grid, 256, 0, s>>>(part, o, total, share, d, c.cu, c.n_seqs, Hg);
    else group_sum_kernel<T, 1><<<grid, 256, 0, s>>>(part, o, total, share, d, c.cu, c.n_seqs, Hg);
  };
  if (dtype == GDN2_BF16) go(static_cast<__nv_bfloat16 *>(out));
  else go(static_cast<float *>(out));
  return cudaGetLastError();
}

cudaError_t launch_step(const StepProblem &p, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.dtype_in == GDN2_BF16)
    return p.dtype_out == GDN2_BF16 ? launch_step_t<B, B>(p, s) : launch_step_t<B, float>(p, s);
  return p.dtype_out == GDN2_BF16 ? launch_step_t<float, B>(p, s) : launch_step_t<float, float>(p, s);
}

}  // namespace lin
}  // namespace gdn2
