// linattn.cu -- linear attention with a decay per head on the CUDA cores: the run for fp32 inputs
// and for head sizes the tensor-core run does not take, the single-token step, and the helpers
// both runs share (the cut plan, the join of the pieces, the gradient of log_a, head sums).
#include <cmath>
#include <type_traits>

#include "linattn.cuh"

namespace gdn2 {
namespace lin {
namespace {

// ---------------------------------------------------------------- plan and join
// Exclusive running counts over the sequences (one block) of their pieces into seg_off and of those of cut
// sequences into cut_off, and the pieces' numbers from the longest down into order; the first two or the
// last may be NULL.
__global__ void __launch_bounds__(1024) plan_kernel(Cut c, int32_t *seg_off, int32_t *cut_off, int32_t *order) {
  __shared__ long long warp_sum[32];  // cut sequences' pieces above bit 32
  __shared__ long long base;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) base = 0;
  for (int n0 = 0; seg_off && n0 < c.n_seqs; n0 += 1024) {
    const int n = n0 + threadIdx.x;
    long long v = 0;
    if (n < c.n_seqs) {
      int t0, len;
      seq_bounds(c, n, &t0, &len);
      v = piece_count(len, c.target, c.grain);
      if (v > 1) v |= v << 32;
    }
    long long incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = base;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    // n_pieces and n_cut bound the counts for offsets in order; anything else is cut back to them
    auto put = [&](int at, long long sum) {
      seg_off[at] = (int)min(sum & 0xffffffffll, (long long)c.n_pieces);
      cut_off[at] = (int)min(sum >> 32, (long long)c.n_cut);
    };
    if (n < c.n_seqs) put(n, before + incl - v);
    __syncthreads();
    if (threadIdx.x == 1023) {
      const long long sum = before + incl;
      base = min(sum & 0xffffffffll, (long long)c.n_pieces) | min(sum >> 32, (long long)c.n_cut) << 32;
      if (n0 + 1024 >= c.n_seqs) put(c.n_seqs, base);
    }
    __syncthreads();
  }
  if (!order) return;
  __syncthreads();
  // keys: chunks, then the lower number first; 0 is no piece.  A bitonic sort, largest first.
  __shared__ uint32_t key[kMaxSorted];
  c.seg_off = seg_off;
  c.cut_off = cut_off;
  const int i = threadIdx.x;
  Piece p;
  key[i] = i < c.n_pieces && find_piece(c, i, &p)
               ? (uint32_t)min(p.len / kChunk + 1, (1 << 21) - 1) << 10 | (uint32_t)(kMaxSorted - 1 - i)
               : 0u;
  for (int size = 2; size <= kMaxSorted; size *= 2)
    for (int step = size / 2; step; step /= 2) {
      __syncthreads();
      const int j = i ^ step;
      if (j > i) {
        const uint32_t a = key[i], b = key[j];
        if ((a < b) == ((i & size) == 0)) {
          key[i] = b;
          key[j] = a;
        }
      }
    }
  __syncthreads();
  if (i < c.n_pieces) order[i] = key[i] ? kMaxSorted - 1 - (int)(key[i] & (kMaxSorted - 1)) : -1;
}

// piece_state[s] holds the end state of piece s from zero; in its place comes the state piece s
// starts from: start_{s+1} = e^{sum log_a of s} start_s + end_s (from the last piece down in a
// backward run).  Elementwise in the state, serial over the pieces; the loads of the next piece
// do not depend on the sum, so four are kept in flight.
struct Runs {
  Run run[kMaxRuns];
};
// A block for a sequence, or, of many sequences, for a piece of a cut one (its first works).
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Runs P, int by_seq) {
  const Run &r = P.run[blockIdx.z];
  const int size = r.dy * r.dz, H = r.cut.H;
  const int h = blockIdx.x % H;
  Piece pc;  // the first of a cut sequence
  if (by_seq) fill_piece(r.cut, blockIdx.x / H, 0, &pc);
  else if (!find_cut_piece(r.cut, blockIdx.x / H, &pc)) return;
  if (pc.count < 2 || pc.s) return;
  const int n = pc.n, count = min(pc.count, r.cut.n_cut - pc.cut);
  const int e = blockIdx.y * 256 + threadIdx.x;
  if (e >= size) return;
  float cur = 0.f;
  if (r.start) {
    const float *s0 = r.start + (size_t)(n * H + h) * size;
    cur = r.start_t ? s0[(size_t)(e % r.dz) * r.dy + e / r.dz] : s0[e];
  }
  const int64_t unit0 = (int64_t)pc.cut * H + h;
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

// ---------------------------------------------------------------- the run in fp32
// Tiles of 32 tokens: G = X Y^T, P = G o D, out = P Z + f o (X S), S <- g S + (w o Y)^T Z, all in fp32 on
// the CUDA cores.  A block takes a (piece, head) and 64 of the state's columns, which do not mix.
// Per tile and token a block does 64 (2 dy + 32) + 32 dy multiply-adds; shared memory, read by 16
// bytes, bounds it (79% of its rate with two blocks on an SM, now 70%).  So a thread takes 2 x 4 of P and 4 x 4 of
// out, over half of the sums each, which a shuffle joins: 8 x 2048 tokens' gradients of 16 heads of
// 64 x 64 took 1580 us with 1 x 4 and 2 x 4 over whole sums, then 1200, and with two multiply-adds an
// instruction 1126.  (Token by token, a chain of
// shuffles and dependent sums for each, it took 54 us for 32 tokens.)  The decays are summed in whole
// numbers of 2^-32: a tile may hold resets beside weak decays, and differences of their sums have to
// stay exact.
constexpr int TB = kTile32;
constexpr int COLS = 64;
constexpr int kRunThreads = 256;

struct RunSmem {
  int ys;  // floats a row of X and Y (4 banks further on each row)
  int off_y, off_z, off_s, off_m, total;
  __host__ __device__ RunSmem(int dy, bool dots) {
    const int dyp = (dy + 7) / 8 * 8;
    ys = dyp + 4;
    off_y = TB * ys;
    off_z = off_y + TB * ys;
    off_s = off_z + TB * COLS;
    off_m = off_s + dyp * COLS;
    total = off_m + (dots ? TB * COLS : 0);
  }
};

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float part4(const float4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ void fma4(float (&acc)[4], float a, const float4 &b) {
  const float2 aa = make_float2(a, a);
  const float2 lo = __ffma2_rn(aa, make_float2(b.x, b.y), make_float2(acc[0], acc[1]));
  const float2 hi = __ffma2_rn(aa, make_float2(b.z, b.w), make_float2(acc[2], acc[3]));
  acc[0] = lo.x; acc[1] = lo.y; acc[2] = hi.x; acc[3] = hi.y;
}

// ROWS rows of out a thread: 2 where the slice has at most 32 columns, else 4.
template <typename T, int ROWS>
__global__ void __launch_bounds__(kRunThreads, 2) run_kernel(const __grid_constant__ Runs P) {
  const Run &p = P.run[blockIdx.z];
  extern __shared__ __align__(16) float sm[];
  __shared__ __align__(16) float ps[TB][TB + 4];
  __shared__ float dot[TB][COLS / 4 + 1];
  __shared__ long long cum[TB];  // sums of log_a from the tile's first token, inclusive
  __shared__ float fs[TB], ws[TB], tile_g;
  const int H = p.cut.H, tid = threadIdx.x;
  Piece pc;
  if (blockIdx.y * COLS >= p.dz || !find_unit(p.cut, blockIdx.x, p.state_only, &pc)) return;
  const int h = blockIdx.x % H;
  const size_t cut_unit = (size_t)pc.cut * H + h;
  if (p.state_only && (pc.count < 2 || pc.s == (p.back ? 0 : pc.count - 1))) return;
  const RunSmem L(p.dy, p.m != nullptr);
  float *xs = sm, *yv = sm + L.off_y, *zs = sm + L.off_z, *ss = sm + L.off_s, *ms = sm + L.off_m;
  const int dyp = L.ys - 4, col0 = blockIdx.y * COLS, width = min(COLS, p.dz - col0), groups = (width + 3) / 4;
  const T *x = static_cast<const T *>(p.x), *y = static_cast<const T *>(p.y), *z = static_cast<const T *>(p.z);
  const T *m = static_cast<const T *>(p.m);
  const int hx = h / (H / p.Hx), hy = h / (H / p.Hy), hz = h / (H / p.Hz), hm = p.m ? h / (H / p.Hm) : 0;

  // this thread's part of the state: 8 rows by 4 columns
  const int cg = tid % groups, yg = tid / groups;
  const bool owner = yg * 8 < p.dy;
  float S[8][4];
  const size_t state = (size_t)p.dy * p.dz;
  const float *start = nullptr;
  bool st = false;
  if (!p.state_only) {
    if (p.piece_state && pc.count > 1) {
      start = p.piece_state + cut_unit * state;
    } else if (p.start) {
      start = p.start + ((size_t)pc.n * H + h) * state;
      st = p.start_t;
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = yg * 8 + r, col = col0 + cg * 4 + c;
      S[r][c] = start && row < p.dy && col < p.dz ? start[st ? (size_t)col * p.dy + row : (size_t)row * p.dz + col] : 0.f;
    }

  const float fixed = p.per_head ? static_cast<const float *>(p.log_a)[h] : 0.f;
  long long logs = 0;
  bool lost = false;  // a NaN was among the log_a
  const int tiles = (pc.len + TB - 1) / TB;
  for (int it = 0; it < tiles; ++it) {
    const int t0 = (p.back ? tiles - 1 - it : it) * TB, cnt = min(TB, pc.len - t0);
    const size_t tok0 = (size_t)(pc.t0 + t0);
    __syncthreads();
    {  // 8 threads a token, every eighth column each: all of a round's loads before the first store
      const int t = tid >> 3, l = tid & 7;
      const bool in = t < cnt;
      const T *px = p.state_only ? nullptr : x + ((tok0 + t) * p.Hx + hx) * p.dy;
      const T *py = y + ((tok0 + t) * p.Hy + hy) * p.dy, *pz = z + ((tok0 + t) * p.Hz + hz) * p.dz + col0;
      const T *pm = m ? m + ((tok0 + t) * p.Hm + hm) * p.dz + col0 : nullptr;
      for (int c0 = l; c0 < dyp || c0 < COLS; c0 += 64) {
        float vx[8], vy[8], vz[8], vm[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = c0 + 8 * j;
          vx[j] = in && px && c < p.dy ? to_f32<T>(px[c]) : 0.f;
          vy[j] = in && c < p.dy ? to_f32<T>(py[c]) : 0.f;
          vz[j] = in && c < width ? to_f32<T>(pz[c]) : 0.f;
          vm[j] = in && pm && c < width ? to_f32<T>(pm[c]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = c0 + 8 * j;
          if (c < dyp) {
            xs[t * L.ys + c] = vx[j];
            yv[t * L.ys + c] = vy[j];
          }
          if (c < COLS) {
            zs[t * COLS + c] = vz[j];
            if (m) ms[t * COLS + c] = vm[j];
          }
        }
      }
    }
    if (owner && !p.state_only)
#pragma unroll
      for (int r = 0; r < 8; ++r)
        *reinterpret_cast<float4 *>(ss + (yg * 8 + r) * COLS + cg * 4) = make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
    if (tid < TB) {
      float la = 0.f;
      if (tid < cnt) la = p.per_head ? fixed : to_f32<T>(static_cast<const T *>(p.log_a)[(tok0 + tid) * H + h]);
      long long sum = __float2ll_rn(fmaxf(la, kMinLog) * 0x1p32f);
#pragma unroll
      for (int d = 1; d < TB; d <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, d);
        if (tid >= d) sum += up;
      }
      const long long all = __shfl_sync(0xffffffffu, sum, TB - 1);
      cum[tid] = sum;
      const float here = expf(__ll2float_rn(sum) * 0x1p-32f), rest = expf(__ll2float_rn(all - sum) * 0x1p-32f);
      // a NaN among them: what the state reaches through it, and the state
      const uint32_t nans = __ballot_sync(0xffffffffu, isnan(la));
      const bool hit = (p.back ? nans >> tid >> 1 : nans & (0xffffffffu >> (31 - tid))) != 0;
      lost |= nans != 0;
      fs[tid] = hit ? NAN : p.back ? rest : here;
      ws[tid] = p.back ? here : rest;
      if (tid == TB - 1) tile_g = nans ? NAN : here;
      logs = max(logs + all, kMinLogs);
    }
    __syncthreads();
    const float g = tile_g;

    if (!p.state_only) {
      {  // P: rows i, i + 1 and columns j = c + 8 q, half of the sum over k a thread
        const int c = tid & 7, kh = tid >> 3 & 1, i0 = tid >> 4 << 1, k0 = kh * (dyp / 2);
        float acc[2][4] = {};
#pragma unroll 2
        for (int k = k0; k < k0 + dyp / 2; k += 4) {
          const float4 a0 = ld4(xs + i0 * L.ys + k), a1 = ld4(xs + (i0 + 1) * L.ys + k);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 b = ld4(yv + (c + 8 * q) * L.ys + k);
            acc[0][q] = fmaf(a0.x, b.x, fmaf(a0.y, b.y, fmaf(a0.z, b.z, fmaf(a0.w, b.w, acc[0][q]))));
            acc[1][q] = fmaf(a1.x, b.x, fmaf(a1.y, b.y, fmaf(a1.z, b.z, fmaf(a1.w, b.w, acc[1][q]))));
          }
        }
        const int i = i0 + kh;  // the row that this thread adds up
        const long long mine = cum[i];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float other = __shfl_xor_sync(0xffffffffu, kh ? acc[0][q] : acc[1][q], 8);
          const float sum = (kh ? acc[1][q] : acc[0][q]) + other;
          const int j = c + 8 * q;
          const bool in = (p.back ? j >= i : j <= i) && j < cnt;
          const long long d = p.back ? cum[j] - mine : mine - cum[j];
          ps[i][j] = in ? sum * expf(__ll2float_rn(d) * 0x1p-32f) : 0.f;
        }
      }
      __syncthreads();
      {  // out: ROWS rows by 4 columns, half of the sums over k a thread
        const int lane = tid & 31, half = tid >> 5 << 4 | (lane & 15), kh = lane >> 4;
        const int oc = half % groups, og = half / groups, r0 = min(og * ROWS, TB - ROWS);
        float acc[ROWS][4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;
#pragma unroll 2
        for (int k = kh * (dyp / 2); k < (kh + 1) * (dyp / 2); k += 4) {
          float4 a[ROWS];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) a[r] = ld4(xs + (r0 + r) * L.ys + k);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 b = ld4(ss + (k + q) * COLS + oc * 4);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) fma4(acc[r], part4(a[r], q), b);
          }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float f = fs[r0 + r];
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[r][c] *= f;
        }
#pragma unroll 2
        for (int k = kh * (TB / 2); k < (kh + 1) * (TB / 2); k += 4) {
          float4 a[ROWS];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) a[r] = ld4(&ps[r0 + r][k]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 b = ld4(zs + (k + q) * COLS + oc * 4);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) fma4(acc[r], part4(a[r], q), b);
          }
        }
#pragma unroll
        for (int r = 0; r < ROWS / 2; ++r) {
          float o[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float other = __shfl_xor_sync(0xffffffffu, kh ? acc[r][c] : acc[r + ROWS / 2][c], 16);
            o[c] = (kh ? acc[r + ROWS / 2][c] : acc[r][c]) + other;
          }
          const int t = r0 + kh * (ROWS / 2) + r;
          if (og * ROWS >= TB) continue;  // the last threads of widths that do not divide them evenly
          if (m) {
            const float4 b = ld4(ms + t * COLS + oc * 4);
            dot[t][oc] = fmaf(o[0], b.x, fmaf(o[1], b.y, fmaf(o[2], b.z, o[3] * b.w)));
          }
          if (t >= cnt) continue;
          const size_t at = ((tok0 + t) * H + h) * p.dz + col0 + oc * 4;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (oc * 4 + c < width) {
              if (p.out_f32) static_cast<float *>(p.out)[at + c] = o[c];
              else static_cast<T *>(p.out)[at + c] = from_f32<T>(o[c]);
            }
        }
      }
      if (m) {
        __syncthreads();
        if (tid < cnt) {
          float d = 0.f;
          for (int c = 0; c < groups; ++c) d += dot[tid][c];
          p.dots[((size_t)blockIdx.y * p.cut.t_total + tok0 + tid) * H + h] = d;
        }
      }
    }
    if (owner) {
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) S[r][c] *= g;
#pragma unroll 4
      for (int t = 0; t < TB; ++t) {  // zeros behind the sequence
        const float w = ws[t];
        const float4 a = ld4(yv + t * L.ys + yg * 8), b = ld4(yv + t * L.ys + yg * 8 + 4), v = ld4(zs + t * COLS + cg * 4);
#pragma unroll
        for (int r = 0; r < 8; ++r) fma4(S[r], w * part4(r < 4 ? a : b, r & 3), v);
      }
    }
  }

  float *dst = nullptr;
  bool dt = false;
  if (p.state_only) {
    dst = p.piece_state + cut_unit * state;
    if (blockIdx.y == 0 && tid == 0) p.piece_log[cut_unit] = lost ? (double)NAN : (double)logs * 0x1p-32;
  } else if (p.fin && pc.s == (p.back ? 0 : pc.count - 1)) {
    dst = p.fin + ((size_t)pc.n * H + h) * state;
    dt = p.fin_t;
  }
  if (!dst || !owner) return;
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = yg * 8 + r, col = col0 + cg * 4 + c;
      if (row < p.dy && col < p.dz) dst[dt ? (size_t)col * p.dy + row : (size_t)row * p.dz + col] = S[r][c];
    }
}

template <typename T, int ROWS>
cudaError_t launch_run_t(const Run *r, int n, int widest, cudaStream_t s) {
  Runs P;
  int bytes = 0;
  for (int i = 0; i < n; ++i) {
    P.run[i] = r[i];
    const int mine = RunSmem(r[i].dy, r[i].m != nullptr).total * (int)sizeof(float);
    if (mine > bytes) bytes = mine;
  }
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = prepare_kernel(run_kernel<T, ROWS>, RunSmem(128, true).total * (int)sizeof(float), ready);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)run_blocks(r->cut, r->state_only), (unsigned)simt_slices(widest), (unsigned)n);
  run_kernel<T, ROWS><<<grid, kRunThreads, bytes, s>>>(P);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- gradient of log_a
// a_t stands once in every pair (i, j) with j < t <= i:
//   dlog_a_t = sum_{i >= t} (q_i . dq_i - k_i . dk_i) + <S_T, dS_T>,
// a suffix sum over the sequence, held in fp64: its terms cancel.  At a reset they do so wholly (a_t = 0), but for
// their roundings: 0 is written there.
constexpr int kScan = 256;
template <typename T>
__global__ void __launch_bounds__(kScan) dlog_kernel(const float *dq, int nq, const float *dk, int nk,
                                                     const float *S_T, const float *dS_T, int size, int no_start,
                                                     const T *log_a, Cut c, T *dlog) {
  __shared__ double sums[kScan / 32];
  const int H = c.H, n = blockIdx.x / H, h = blockIdx.x % H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int t0, len;
  seq_bounds(c, n, &t0, &len);
  double carry = 0.0;
  if (dS_T && S_T) {
    const size_t at = (size_t)blockIdx.x * size;
    double v = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < size; i += kScan) v += (double)S_T[at + i] * (double)dS_T[at + i];
    for (int b = 16; b; b >>= 1) v += __shfl_xor_sync(0xffffffffu, v, b);
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    for (int w = 0; w < kScan / 32; ++w) carry += sums[w];
  }
  for (int done = 0; done < len; done += kScan) {
    const int t = len - 1 - done - (int)threadIdx.x;  // thread 0 has the latest token
    double v = 0.0;
    float la = 0.f;
    const size_t at = (size_t)(t0 + t) * H + h, slice = (size_t)c.t_total * H;
    if (t >= 0) {
      la = to_f32<T>(log_a[at]);
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
    // the first token decays nothing where no state comes in
    if (t >= 0)
      dlog[at] = from_f32<T>((no_start && t == 0) || la <= kMinLog ? 0.f : (float)(before + incl));
    for (int w = 0; w < kScan / 32; ++w) carry += sums[w];
  }
}

// ---------------------------------------------------------------- heads that share q and k
// A thread sums VEC columns: 16-byte loads of the parts, which are most of what it moves.
struct Sums {
  const float *part[2];
  void *out[2];
};
template <typename T, int VEC>
__global__ void __launch_bounds__(256) group_sum_kernel(const __grid_constant__ Sums P, int64_t total, int share, int d,
                                                        const int32_t *cu, int n_seqs, int Hg) {
  const float *part = P.part[blockIdx.y];
  T *out = static_cast<T *>(P.out[blockIdx.y]);
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
// e^la as the sum of two floats: a fixed decay's rounding is the same at every token, and a state that
// keeps n of them would be off by n.  la = n ln 2 + r (Cody and Waite's two-part ln 2), then the
// Taylor series of e^r, its terms from r^2 / 2 on in one float: off by about r^2 2^-23, 2^-25 at most, and by far
// less for the weak decays that are remembered long.
__device__ __forceinline__ float2 split_exp(float la) {
  if (la <= kMinLog) return make_float2(0.f, 0.f);
  const float n = rintf(la * 1.44269504f);
  const float big = fmaf(n, -0.693359375f, la);         // exact
  const float r = fmaf(n, 2.12194440e-4f, big), r_lo = fmaf(n, 2.12194440e-4f, big - r);
  float e = 1.f / 40320.f;
  e = fmaf(e, r, 1.f / 5040.f);
  e = fmaf(e, r, 1.f / 720.f);
  e = fmaf(e, r, 1.f / 120.f);
  e = fmaf(e, r, 1.f / 24.f);
  e = fmaf(e, r, 1.f / 6.f);
  e = fmaf(e, r, 0.5f);
  const float rest = fmaf(e * r, r, r_lo);
  const float a = 1.f + r, b = r - (a - 1.f);            // 1 + r
  const float hi = a + (rest + b), lo = (rest + b) - (hi - a);
  return make_float2(ldexpf(hi, (int)n), ldexpf(lo, (int)n));
}
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

cudaError_t launch_plan(const Cut &c, int32_t *seg_off, int32_t *cut_off, int32_t *order, cudaStream_t s) {
  plan_kernel<<<1, 1024, 0, s>>>(c, seg_off, cut_off, order);
  return cudaGetLastError();
}

cudaError_t launch_join(const Run *r, int n, cudaStream_t s) {
  Runs P;
  for (int i = 0; i < n; ++i) P.run[i] = r[i];
  const int by_seq = r->cut.n_seqs <= r->cut.n_cut;
  const dim3 grid((unsigned)((by_seq ? r->cut.n_seqs : r->cut.n_cut) * r->cut.H), (unsigned)((r->dy * r->dz + 255) / 256),
                  (unsigned)n);
  join_kernel<<<grid, 256, 0, s>>>(P, by_seq);
  return cudaGetLastError();
}

int simt_slices(int dz) { return (dz + COLS - 1) / COLS; }

cudaError_t launch_run_simt(const Run *r, int n, cudaStream_t s) {
  int widest = 0;
  for (int i = 0; i < n; ++i)
    if (r[i].dz > widest) widest = r[i].dz;
  const bool bf16 = r->dtype == GDN2_BF16;
  if (widest <= 32)
    return bf16 ? launch_run_t<__nv_bfloat16, 2>(r, n, widest, s) : launch_run_t<float, 2>(r, n, widest, s);
  return bf16 ? launch_run_t<__nv_bfloat16, 4>(r, n, widest, s) : launch_run_t<float, 4>(r, n, widest, s);
}

cudaError_t launch_dlog_simt(const float *dots_q, int nq, const float *dots_k, int nk, const float *S_T,
                             const float *dS_T, int dk, int dv, bool no_start, const void *log_a, const Cut &c, void *dlog,
                             int dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)(c.n_seqs * c.H);
  if (dtype == GDN2_BF16)
    dlog_kernel<<<grid, kScan, 0, s>>>(dots_q, nq, dots_k, nk, S_T, dS_T, dk * dv, no_start,
                                       static_cast<const __nv_bfloat16 *>(log_a), c, static_cast<__nv_bfloat16 *>(dlog));
  else
    dlog_kernel<<<grid, kScan, 0, s>>>(dots_q, nq, dots_k, nk, S_T, dS_T, dk * dv, no_start,
                                       static_cast<const float *>(log_a), c, static_cast<float *>(dlog));
  return cudaGetLastError();
}

cudaError_t launch_group_sum(const float *const *part, void *const *out, int n, const Cut &c, int Hg, int d, int dtype,
                             cudaStream_t s) {
  const int64_t total = (int64_t)c.t_total * Hg * d;
  const int share = c.H / Hg;
  if (total == 0) return cudaSuccess;
  Sums P;
  for (int i = 0; i < 2; ++i) {
    P.part[i] = part[i < n ? i : 0];
    P.out[i] = out[i < n ? i : 0];
  }
  const int vec = d % 4 == 0 ? 4 : 1;
  const dim3 grid((unsigned)((total + 256 * vec - 1) / (256 * vec)), (unsigned)n);
  auto go = [&](auto zero) {
    using T = decltype(zero);
    if (vec == 4) group_sum_kernel<T, 4><<<grid, 256, 0, s>>>(P, total, share, d, c.cu, c.n_seqs, Hg);
    else group_sum_kernel<T, 1><<<grid, 256, 0, s>>>(P, total, share, d, c.cu, c.n_seqs, Hg);
  };
  if (dtype == GDN2_BF16) go(__nv_bfloat16());
  else go(0.f);
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
