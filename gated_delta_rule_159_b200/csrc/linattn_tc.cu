// linattn_tc.cu -- one run of linear attention with a decay per head on the tensor cores
// (d_k = d_v = 128, bf16): out_t = sum_j e^{|L_t - L_j|..} (x_t . y_j) z_j + (state part), chunks of
// 128 tokens, a CTA per (piece, head) that walks its chunks in order (last first when BACK).
//
// Per chunk, with D the matrix of decays inside the chunk (0 outside the triangle), w_j the decay
// from token j to the chunk's far end, f_i the decay from its near end to token i, g the chunk's:
//   G = X Y^T,  P = bf16(G o D)           (rows = tokens; P becomes a TMEM operand)
//   out = P Z + f o (X S)                 (two accumulators, joined in fp32 by the epilogue)
//   S <- g S + (w o Y)^T Z                (S in fp32 registers; the increment in TMEM)
// The state is exact to fp32: w o Y goes to the tensor cores as a sum of NT bf16 values (3 give 24
// bits, 2 give 16, for runs whose state only feeds bf16 products), Z is bf16 already.
//
// Memory is what bounds it: 4 tiles of 32 KB a chunk, 128 KB against 2.9 us of 6.6 TB/s / 148 SMs;
// the products take 6 x 512 tensor cycles.  One chain runs through the chunks: the state and its
// update; everything else runs beside it.  Roles: warp 0 loads; warp 1 issues the state's products
// (X S, the update), warp 3 the rows' (G, P Z); warp 2 sums the decays; warps 4-7 own a token row a
// thread (P, out); warps 8-15 own the state and weight Y.  What fits two stages of Y and Z into shared memory: X has one, the first bf16 term of w o Y
// overwrites Y once X Y^T is done, the other terms pass through a ring of 32-token slices, and
// out is staged in Y's place after the update.
// Instruction issue comes next: the loops stay rolled (unrolled, the roles together ran out of the
// instruction cache) and the fp32 arithmetic goes by pairs.
#include <cstring>

#include "linattn.cuh"
#include "tc_util.cuh"

namespace gdn2 {
namespace lin {
namespace {

using namespace gdn2::tc;

constexpr int D = 128;
constexpr int C = kChunk;
constexpr int kThreads = 512;
constexpr uint32_t kTile = C * D * 2;       // 32 KB, two column blocks of 64
constexpr uint32_t kBlock = kTile / 2;
constexpr int kSlice = 32;                  // tokens of a slice of w o Y
constexpr uint32_t kSliceTile = kSlice * D * 2, kSliceBlock = kSliceTile / 2;
constexpr uint32_t OFF_X = 0, OFF_Y = kTile, OFF_Z = 3 * kTile;  // Y, Z: two stages
constexpr uint32_t OFF_S = 5 * kTile;       // the bf16 state, [dz][dy]
constexpr uint32_t OFF_W = 6 * kTile;       // the ring
constexpr uint32_t OFF_MISC = 7 * kTile;
// per stage: the decay from each token to the edge of its 32-token block (log2, as a float and its
// bf16 remainder), 2^(block total - that), the four block totals
constexpr uint32_t DEC_HI = 0, DEC_LO = 512, DEC_BETA = 768, DEC_TOT = 1280, DEC_BYTES = 1296;
constexpr uint32_t MISC_BAR = 2 * DEC_BYTES;
enum {
  BAR_Y = 0,        // + stage: Y loaded
  BAR_Z = 2,        // + stage: Z loaded
  BAR_DEC = 4,      // + stage: decays summed
  BAR_FREE = 6,     // + stage: nothing uses Y, Z and the decays any more
  BAR_G = 8,        // + stage: X Y^T done (two: the next may be done before the state warps look)
  BAR_STAGED = 10,  // + stage: out tile staged (two: the next may be staged before the storing warp looks)
  BAR_FULL = 12,    // + slot: a slice of w o Y written
  BAR_EMPTY = 16,   // + slot: its products done
  BAR_X = 20,       // X loaded
  BAR_XFREE,        // X Y^T and X S done
  BAR_XS,           // X S done
  BAR_P,            // P written
  BAR_PZ,           // P Z done
  BAR_U,            // increment done
  BAR_S,            // bf16 state written
  BAR_OREAD,        // X S and P Z read
  BAR_CLEAN,        // Y's and Z's rows behind the sequence cleared
  BAR_DRAIN,        // + 0, 1
  N_BARS = BAR_DRAIN + 2
};
constexpr uint32_t MISC_TMEM = MISC_BAR + N_BARS * 8, MISC_ABORT = MISC_TMEM + 4;
constexpr uint32_t MISC_BYTES = MISC_ABORT + 4;
constexpr uint32_t kSmemBytes = OFF_MISC + MISC_BYTES;
static_assert(kSmemBytes <= 232448, "shared memory over the sm_100 limit per CTA");
constexpr uint32_t TM_G = 0, TM_PZ = 128, TM_XS = 256, TM_U = 384;  // TMEM columns; P overwrites G
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint32_t kSleepNs = 20000;  // between two looks at the clock: busy waits take issue slots from the workers
constexpr float kLog2 = 1.4426950408889634f;

struct TcRun {
  Run r;
  CUtensorMap tm_x, tm_y, tm_z, tm_o;
  int32_t *status;
  uint64_t wait_ns;
  int dbg_skip;
};

// Tiles of two column blocks as operands: rows x K (kmaj), K x rows (mnmaj), and the steps from one
// K = 16 product to the next, in the descriptors' 16-byte units.
__device__ __forceinline__ uint64_t kmaj(uint32_t base) { return ptx::sdesc_sw128(base, 16, 1024); }
__device__ __forceinline__ uint64_t mnmaj(uint32_t base, uint32_t block = kBlock) {
  return ptx::sdesc_sw128(base, block, 1024);
}
__device__ __forceinline__ uint64_t k_step(int kk) { return (uint64_t)((kk >> 2) * (kBlock >> 4) + (kk & 3) * 2); }
constexpr uint64_t kMnStep = 2048 >> 4;
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
// The two fp32 values cut (not rounded) to bf16, in place and packed.
__device__ __forceinline__ float2 cut2(float2 v) {
  return pair(__float_as_uint(v.x) & 0xffff0000u, __float_as_uint(v.y) & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_cut(float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); }
// One copy of the waiting loop for all waits: some thirty inlined ones filled the instruction cache.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status,
                                       uint64_t limit_ns) {
  if (*abort_flag) return false;
  const uint64_t t0 = global_timer_ns();
  while (!ptx::mbar_try_wait_for(bar, parity, kSleepNs)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicExch(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

template <bool BACK, int NT>
__global__ void __launch_bounds__(kThreads, 1) run_tc_kernel(const __grid_constant__ TcRun P) {
  constexpr int SLOTS = NT == 3 ? 2 : 4;  // of the ring: NT - 1 slice tiles each
  extern __shared__ __align__(1024) uint8_t smem[];
  const Run &r = P.r;
  const uint32_t sb = ptx::smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int H = r.cut.H, unit = blockIdx.x, h = unit % H;
  Piece pc;
  if (!find_piece(r.cut, unit / H, &pc)) return;
  const bool only = r.state_only != 0;
  if (only && (pc.count < 2 || pc.s == (BACK ? 0 : pc.count - 1))) return;
  if (sb & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts on it
    if (tid == 0) atomicExch(P.status, kStatusTimeout);
    return;
  }
  const int nch = (pc.len + C - 1) / C;
  auto bar = [&](int b) { return sb + OFF_MISC + MISC_BAR + 8u * (uint32_t)b; };
  auto dec = [&](int s) { return sb + OFF_MISC + (uint32_t)s * DEC_BYTES; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + OFF_MISC + MISC_ABORT);
  auto wait = [&](int b, uint32_t parity) {
    return ptx::mbar_try_wait(bar(b), parity & 1u) || wait_long(bar(b), parity & 1u, abort_flag, P.status, P.wait_ns);
  };
  // the same for whole warps, which stay together whether or not it gives up
  auto wait_warp = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar(b), parity & 1u)) ||
           __all_sync(0xffffffffu, wait_long(bar(b), parity & 1u, abort_flag, P.status, P.wait_ns));
  };
  // tokens of the k-th chunk walked: its number and how many rows it has
  auto chunk_no = [&](int k) { return BACK ? nch - 1 - k : k; };
  auto rows_of = [&](int k) { return min(C, pc.len - chunk_no(k) * C); };

  if (tid == 0) {
    *abort_flag = 0;
    for (int b = 0; b < N_BARS; ++b) {
      const bool rows = b == BAR_P || b == BAR_OREAD || b == BAR_STAGED || b == BAR_STAGED + 1;
      const bool state = b == BAR_S || b == BAR_CLEAN || (b >= BAR_FULL && b < BAR_EMPTY);
      ptx::mbar_init(bar(b), rows ? 4 : state ? 8 : b == BAR_XFREE ? 2 : 1);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(sb + OFF_MISC + MISC_TMEM, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(smem + OFF_MISC + MISC_TMEM), 0);

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      const int hx = h / (H / r.Hx), hy = h / (H / r.Hy), hz = h / (H / r.Hz);
      const bool skip = P.dbg_skip && blockIdx.x == 0;
      int k_yz = 0, k_x = 0;  // loads asked for
      for (int k = 0; k < nch; ++k) {
        const int s = k & 1, t0 = pc.t0 + chunk_no(k) * C;
        if (k >= 2 && !wait(BAR_FREE + s, (uint32_t)(k >> 1) + 1u)) break;
        ptx::mbar_arrive_expect_tx(bar(BAR_Y + s), kTile);
        k_yz = k + 1;
        if (skip) break;
        for (int b = 0; b < 2; ++b)
          ptx::tma_load_3d(sb + OFF_Y + s * kTile + b * kBlock, &P.tm_y, b * 64, hy, t0, bar(BAR_Y + s));
        ptx::mbar_arrive_expect_tx(bar(BAR_Z + s), kTile);
        for (int b = 0; b < 2; ++b)
          ptx::tma_load_3d(sb + OFF_Z + s * kTile + b * kBlock, &P.tm_z, b * 64, hz, t0, bar(BAR_Z + s));
        if (only) continue;
        if (k >= 1 && !wait(BAR_XFREE, (uint32_t)k + 1u)) break;
        ptx::mbar_arrive_expect_tx(bar(BAR_X), kTile);
        k_x = k + 1;
        for (int b = 0; b < 2; ++b) ptx::tma_load_3d(sb + OFF_X + b * kBlock, &P.tm_x, b * 64, hx, t0, bar(BAR_X));
        if (k + 1 < nch)
          for (int b = 0; b < 2; ++b) ptx::tma_prefetch_3d(&P.tm_x, b * 64, hx, pc.t0 + chunk_no(k + 1) * C);
      }
      // every load has to land before the CTA leaves, whether or not somebody waited for it
      for (int k = max(0, k_yz - 2); k < k_yz; ++k) {
        drain_bar(bar(BAR_Y + (k & 1)), (uint32_t)(k >> 1) & 1u, P.wait_ns);
        if (!skip) drain_bar(bar(BAR_Z + (k & 1)), (uint32_t)(k >> 1) & 1u, P.wait_ns);
      }
      if (k_x) drain_bar(bar(BAR_X), (uint32_t)(k_x - 1) & 1u, P.wait_ns);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- the state's products
    {
      const bool lead = ptx::elect_one();
      constexpr uint32_t idKK = ptx::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idNN = ptx::idesc_bf16(128, 128, true, true);
      bool ok = true;
      for (int k = 0; k < nch && ok; ++k) {
        const int s = k & 1;
        const uint32_t y = sb + OFF_Y + (uint32_t)s * kTile, z = sb + OFF_Z + (uint32_t)s * kTile;
        if (!only) {
          // the state's copy, and the last X S read
          if (!wait_warp(BAR_X, (uint32_t)k) || !wait_warp(BAR_S, (uint32_t)k) || (k && !wait_warp(BAR_OREAD, (uint32_t)k + 1u))) break;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int kk = 0; kk < 8; ++kk)
            ptx::umma_bf16_if(lead, tm + TM_XS, kmaj(sb + OFF_X) + k_step(kk), kmaj(sb + OFF_S) + k_step(kk), idKK, kk > 0);
          ptx::umma_commit_if(lead, bar(BAR_XS));
          ptx::umma_commit_if(lead, bar(BAR_XFREE));
        }
        if (!wait_warp(BAR_Z + s, (uint32_t)(k >> 1))) break;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int n = 4 * k + i, slot = n % SLOTS, b = BACK ? i : 3 - i;
          ok = wait_warp(BAR_FULL + slot, (uint32_t)(n / SLOTS));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t zd = mnmaj(z + (uint32_t)b * (kSlice * 128)), yd = mnmaj(y + (uint32_t)b * (kSlice * 128));
          const uint64_t wd = mnmaj(sb + OFF_W + (uint32_t)(slot * (NT - 1)) * kSliceTile, kSliceBlock);
#pragma unroll
          for (int part = 0; part < NT; ++part)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
              ptx::umma_bf16_if(lead, tm + TM_U, zd + kk * kMnStep,
                             (part == 0 ? yd : wd + (uint64_t)(part - 1) * (kSliceTile >> 4)) + kk * kMnStep, idNN,
                             (i > 0) | (part + kk > 0));
          ptx::umma_commit_if(lead, bar(BAR_EMPTY + slot));
        }
        if (!ok) break;
        ptx::umma_commit_if(lead, bar(BAR_U));
        if (only) ptx::umma_commit_if(lead, bar(BAR_FREE + s));
      }
      ptx::umma_commit_if(lead, bar(BAR_DRAIN));  // all products, before the tensor memory is freed
      drain_bar(bar(BAR_DRAIN), 0u, P.wait_ns);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- the rows' products
    if (!only) {
      const bool lead = ptx::elect_one();
      constexpr uint32_t idKK = ptx::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idKN = ptx::idesc_bf16(128, 128, false, true);
      for (int k = 0; k < nch; ++k) {
        const int s = k & 1;
        const uint32_t y = sb + OFF_Y + (uint32_t)s * kTile, z = sb + OFF_Z + (uint32_t)s * kTile;
        if (!wait_warp(BAR_X, (uint32_t)k) || !wait_warp(BAR_Y + s, (uint32_t)(k >> 1))) break;
        if (rows_of(k) < C && !wait_warp(BAR_CLEAN, 0u)) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < 8; ++kk)
          ptx::umma_bf16_if(lead, tm + TM_G, kmaj(sb + OFF_X) + k_step(kk), kmaj(y) + k_step(kk), idKK, kk > 0);
        ptx::umma_commit_if(lead, bar(BAR_G + s));
        ptx::umma_commit_if(lead, bar(BAR_XFREE));
        if (!wait_warp(BAR_Z + s, (uint32_t)(k >> 1)) || !wait_warp(BAR_P, (uint32_t)k)) break;
        if (k && !wait_warp(BAR_OREAD, (uint32_t)k + 1u)) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < 8; ++kk)
          ptx::umma_bf16_ts_if(lead, tm + TM_PZ, tm + TM_G + kk * 8, mnmaj(z) + kk * kMnStep, idKN, kk > 0);
        ptx::umma_commit_if(lead, bar(BAR_PZ));
      }
      ptx::umma_commit_if(lead, bar(BAR_DRAIN + 1));
      drain_bar(bar(BAR_DRAIN + 1), 0u, P.wait_ns);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- decays and stores
    // Lane l sums tokens 4 l .. 4 l + 3 in fp64 (a chunk may hold resets beside weak decays); 8
    // lanes are a block of 32 tokens.  Forward, `edge` of token i is the log2 decay from its
    // block's start to it, itself included; backward, from it to the block's end, itself not.
    const float fixed = r.per_head ? static_cast<const float *>(r.log_a)[h] : 0.f;
    const __nv_bfloat16 *la = static_cast<const __nv_bfloat16 *>(r.log_a);
    auto load = [&](int k, float (&a)[4]) {
      const int c0 = chunk_no(k) * C, rows = rows_of(k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * lane + j;
        a[j] = i >= rows ? 0.f : r.per_head ? fixed : __bfloat162float(la[(size_t)(pc.t0 + c0 + i) * H + h]);
      }
    };
    // chunk k's out tile; the stage is free once it has been read
    auto store = [&](int k) {
      if (only) return wait_warp(BAR_FREE + (k & 1), (uint32_t)(k >> 1));
      if (!wait_warp(BAR_STAGED + (k & 1), (uint32_t)(k >> 1))) return false;
      if (lane == 0) {
        if (!r.out_f32 && rows_of(k) == C) {
          const uint32_t src = sb + OFF_Y + (uint32_t)(k & 1) * kTile;
          const int t0 = pc.t0 + chunk_no(k) * C;
          for (int b = 0; b < 2; ++b) ptx::tma_store_3d(&P.tm_o, src + b * kBlock, b * 64, h, t0);
          ptx::bulk_commit_group();
          ptx::bulk_wait_group_read0();
        }
        ptx::mbar_arrive(bar(BAR_FREE + (k & 1)));
      }
      return true;
    };
    double logs = 0.0;
    float a[4];
    if (nch > 0) load(0, a);
    bool ok = true;
    // the last two rounds only store
    for (int k = 0; k < (only ? nch : nch + 2) && ok; ++k) {
      if (k >= nch) {
        if (k >= 2) ok = store(k - 2);
        continue;
      }
      double own[4];  // inclusive sums inside the lane
#pragma unroll
      for (int j = 0; j < 4; ++j) own[j] = (double)fmaxf(a[j], kMinLog) + (j ? own[j - 1] : 0.0);
      if (k + 1 < nch) load(k + 1, a);
      double incl = own[3];
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, incl, d, 8);
        if ((lane & 7) >= d) incl += up;
      }
      const double total = __shfl_sync(0xffffffffu, incl, 7, 8), before = incl - own[3];
      float hi[4], beta[4];
      uint32_t lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double in = before + own[j];
        const double edge = (BACK ? total - in : in) * (double)kLog2, rest = (BACK ? in : total - in) * (double)kLog2;
        hi[j] = (float)edge;
        lo[j] = bf16_bits((float)(edge - (double)hi[j]));
        beta[j] = ptx::ex2((float)rest);
      }
      if (k >= 2) ok = store(k - 2);
      if (!ok) break;
      const uint32_t at = dec(k & 1);
      sts_v4(at + DEC_HI + 16 * lane, make_uint4(__float_as_uint(hi[0]), __float_as_uint(hi[1]), __float_as_uint(hi[2]),
                                                 __float_as_uint(hi[3])));
      sts_v2(at + DEC_LO + 8 * lane, make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16));
      sts_v4(at + DEC_BETA + 16 * lane, make_uint4(__float_as_uint(beta[0]), __float_as_uint(beta[1]),
                                                   __float_as_uint(beta[2]), __float_as_uint(beta[3])));
      if ((lane & 7) == 0) sts_f32(at + DEC_TOT + (lane >> 3) * 4, (float)(total * (double)kLog2));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(BAR_DEC + (k & 1)));
      if (only) {
        logs += __shfl_sync(0xffffffffu, total, 0) + __shfl_sync(0xffffffffu, total, 8) +
                __shfl_sync(0xffffffffu, total, 16) + __shfl_sync(0xffffffffu, total, 24);
      }
    }
    if (only && lane == 0) r.piece_log[unit] = logs;
    if (!only && lane == 0) ptx::bulk_wait_group0();
  } else if (warp < 8) {
    // ---------------------------------------------------------------- P and out: a token row a thread
    if (!only) {
      const int wq = warp & 3, row = wq * 32 + lane;
      const uint32_t lanes = tm + ((uint32_t)(wq * 32) << 16);
      for (int k = 0; k < nch; ++k) {
        const int s = k & 1;
        const uint32_t at = dec(s);
        const bool in = row < rows_of(k);
        const size_t tok = (size_t)pc.t0 + (size_t)chunk_no(k) * C + row;
        const __nv_bfloat16 *m = nullptr;
        if (r.m && in) {
          m = static_cast<const __nv_bfloat16 *>(r.m) + (tok * r.Hm + h / (H / r.Hm)) * D;
          prefetch_l2(m);
          prefetch_l2(m + 64);
        }
        if (!wait_warp(BAR_DEC + s, (uint32_t)(k >> 1))) break;
        const float edge = lds_f32(at + DEC_HI + row * 4), edge_lo = bf16_value(lds_u16(at + DEC_LO + row * 2));
        float near = edge;  // log2 f_i: to the chunk's near end
        for (int b = BACK ? wq + 1 : 0; b < (BACK ? 4 : wq); ++b) near += lds_f32(at + DEC_TOT + b * 4);
        const float f = ptx::ex2(near);
        if (!wait_warp(BAR_G + s, (uint32_t)(k >> 1))) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int cb = 0; cb < 4; ++cb) {
          uint32_t out[16];
          if (BACK ? cb < wq : cb > wq) {
#pragma unroll
            for (int j = 0; j < 16; ++j) out[j] = 0u;
          } else {
            uint32_t g[32];
            ptx::tmem_ld32(lanes + TM_G + cb * 32, g);
            if (cb == wq) {
              // both tokens in one block: the decay between them, pair by pair
              const float2 minus = make_float2(-1.f, -1.f), e2 = make_float2(edge, edge);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j4 = 0; j4 < 8; ++j4) {
                const float4 e = lds_f4(at + DEC_HI + cb * 128 + j4 * 16);
                const uint2 l = lds_v2(at + DEC_LO + cb * 64 + j4 * 8);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int j = j4 * 4 + 2 * i;
                  const uint32_t lw = i ? l.y : l.x;
                  const float2 eh = i ? make_float2(e.z, e.w) : make_float2(e.x, e.y);
                  const float2 d = fma2(eh, minus, e2);
                  const float2 w = make_float2(ptx::ex2(d.x + (edge_lo - __uint_as_float(lw << 16))),
                                               ptx::ex2(d.y + (edge_lo - __uint_as_float(lw & 0xffff0000u))));
                  const float2 v = mul2(w, pair(g[j], g[j + 1]));
                  out[2 * j4 + i] = pack_bf16x2((BACK ? j >= lane : j <= lane) ? v.x : 0.f,
                                                (BACK ? j + 1 >= lane : j + 1 <= lane) ? v.y : 0.f);
                }
              }
            } else {
              // through the edges of the two blocks: a row factor times a column factor, both <= 1
              float between = edge;
              for (int b = BACK ? wq + 1 : cb + 1; b < (BACK ? cb : wq); ++b) between += lds_f32(at + DEC_TOT + b * 4);
              const float alpha = ptx::ex2(between);
              const float2 a2 = make_float2(alpha, alpha);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j4 = 0; j4 < 8; ++j4) {
                const float4 be = lds_f4(at + DEC_BETA + cb * 128 + j4 * 16);
                const float2 v = mul2(mul2(a2, make_float2(be.x, be.y)), pair(g[4 * j4], g[4 * j4 + 1]));
                const float2 u = mul2(mul2(a2, make_float2(be.z, be.w)), pair(g[4 * j4 + 2], g[4 * j4 + 3]));
                out[2 * j4] = pack_bf16x2(v.x, v.y);
                out[2 * j4 + 1] = pack_bf16x2(u.x, u.y);
              }
            }
          }
          // columns 16 cb .. are G columns of block cb / 2, read already
          ptx::tmem_st16(lanes + TM_G + cb * 16, out);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_P));
        const float2 f2 = make_float2(f, f);
        float2 dot = make_float2(0.f, 0.f);
        const bool whole = rows_of(k) == C && !r.out_f32;
        const uint32_t dst = sb + OFF_Y + (uint32_t)s * kTile;
        if (!wait_warp(BAR_XS, (uint32_t)k) || !wait_warp(BAR_PZ, (uint32_t)k) || !wait_warp(BAR_U, (uint32_t)k)) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int cb = 0; cb < 8; ++cb) {
          uint4 mw[2];
          if (m)
#pragma unroll
            for (int j = 0; j < 2; ++j) mw[j] = *reinterpret_cast<const uint4 *>(m + cb * 16 + 8 * j);
          uint32_t u[16], v[16];
          ptx::tmem_ld16(lanes + TM_PZ + cb * 16, u);
          ptx::tmem_ld16(lanes + TM_XS + cb * 16, v);
          ptx::tmem_wait_ld();
          if (cb == 7) {  // the accumulators are in registers
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BAR_OREAD));
          }
          float2 o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = fma2(f2, pair(v[2 * j], v[2 * j + 1]), pair(u[2 * j], u[2 * j + 1]));
          if (m)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w[4] = {mw[j].x, mw[j].y, mw[j].z, mw[j].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) dot = fma2(pair(w[i] << 16, w[i] & 0xffff0000u), o[4 * j + i], dot);
            }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 w = make_uint4(pack_bf16x2(o[4 * j].x, o[4 * j].y), pack_bf16x2(o[4 * j + 1].x, o[4 * j + 1].y),
                                       pack_bf16x2(o[4 * j + 2].x, o[4 * j + 2].y),
                                       pack_bf16x2(o[4 * j + 3].x, o[4 * j + 3].y));
            const size_t at_out = (tok * H + h) * D + cb * 16 + 8 * j;
            if (whole) {
              sts_v4(dst + (uint32_t)(cb >> 2) * kBlock + swz(row, (uint32_t)((cb & 3) * 2 + j)), w);
            } else if (in && r.out_f32) {
              float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(r.out) + at_out);
              p[0] = make_float4(o[4 * j].x, o[4 * j].y, o[4 * j + 1].x, o[4 * j + 1].y);
              p[1] = make_float4(o[4 * j + 2].x, o[4 * j + 2].y, o[4 * j + 3].x, o[4 * j + 3].y);
            } else if (in) {
              *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(r.out) + at_out) = w;
            }
          }
          __syncwarp();
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_STAGED + s));
        if (m) r.dots[tok * H + h] = dot.x + dot.y;
      }
    }
  } else {
    // ---------------------------------------------------------------- state: warp -> 32 z rows x 64 y columns
    const int wq = warp & 3, half = (warp - 8) >> 2, zrow = wq * 32 + lane;
    const int stid = tid - 256;
    const uint32_t lanes = tm + ((uint32_t)(wq * 32) << 16) + TM_U + half * 64;
    float S[64];
    {
      const float *start = nullptr;
      bool st = false;
      if (!only) {
        if (r.piece_state && pc.count > 1) {
          start = r.piece_state + (size_t)unit * D * D;
        } else if (r.start) {
          start = r.start + ((size_t)pc.n * H + h) * D * D;
          st = r.start_t;
        }
      }
      if (!start) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = 0.f;
      } else if (!st) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = start[(half * 64 + j) * D + zrow];
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float4 v = *reinterpret_cast<const float4 *>(start + zrow * D + half * 64 + 4 * j);
          S[4 * j] = v.x; S[4 * j + 1] = v.y; S[4 * j + 2] = v.z; S[4 * j + 3] = v.w;
        }
      }
    }
    auto write_state = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j) sts_v4(sb + OFF_S + half * kBlock + swz(zrow, (uint32_t)j), pack8(S + 8 * j, 1.f));
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(BAR_S));
    };
    // marks of this thread's part of the state at the end of group `g` of chunks
    auto mark_unit = [&](int g) { return (size_t)mark_slot(unit / H, pc.t0 + g * kGroup * C) * H + h; };
    auto ends_group = [&](int no) { return (no + 1) % kGroup == 0 || no == nch - 1; };
    if (!only && nch > 0) write_state();
    bool ok = true;
    for (int k = 0; k < nch && ok; ++k) {
      const int s = k & 1, rows = rows_of(k);
      if (BACK && r.mark_dots && !only) {
        const int no = chunk_no(k);
        if (ends_group(no)) {
          const size_t mu = mark_unit(no / kGroup);
          const float4 *mark = reinterpret_cast<const float4 *>(r.marks + mu * (D * D)) + stid;
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float4 v = mark[j * 256];
            dot = fmaf(v.x, S[4 * j], fmaf(v.y, S[4 * j + 1], fmaf(v.z, S[4 * j + 2], fmaf(v.w, S[4 * j + 3], dot))));
          }
#pragma unroll
          for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
          if (lane == 0) r.mark_dots[mu * 8 + (warp - 8)] = dot;
        }
        if (no % kGroup == 1 && no > kGroup) {  // the next group's mark, two chunks ahead
          const char *next = reinterpret_cast<const char *>(r.marks + mark_unit(no / kGroup - 1) * (D * D)) + stid * 256;
          prefetch_l2(next);
          prefetch_l2(next + 128);
        }
      }
      const uint32_t y = sb + OFF_Y + (uint32_t)s * kTile, par = (uint32_t)(k >> 1);
      ok = wait_warp(BAR_DEC + s, par) && wait_warp(BAR_Y + s, par) && (rows == C || wait_warp(BAR_Z + s, par));
      if (ok && rows < C) {
        // rows behind the sequence meet zero weights, which a NaN would outlive
        for (int t = stid >> 4; t < C; t += 16)
          if (t >= rows) {
            const uint32_t to = y + (uint32_t)(stid >> 3 & 1) * kBlock + swz(t, (uint32_t)(stid & 7));
            sts_v4(to, make_uint4(0u, 0u, 0u, 0u));
            sts_v4(to + (OFF_Z - OFF_Y), make_uint4(0u, 0u, 0u, 0u));
          }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_CLEAN));
      }
      if (ok && !only) ok = wait_warp(BAR_G + s, (uint32_t)(k >> 1));  // Y may be overwritten
      if (!ok) break;
      const float4 tot = lds_f4(dec(s) + DEC_TOT);
      const float g = ptx::ex2((tot.x + tot.y) + (tot.z + tot.w));
      float far = 0.f;  // from the edge of the tokens' block to the chunk's far end
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int b = BACK ? i : 3 - i, n = 4 * k + i, slot = n % SLOTS;
        const float wb = ptx::ex2(far);
        far += lds_f32(dec(s) + DEC_TOT + b * 4);
        const int t = stid >> 4;  // rows t and t + 16 of the slice
        const uint32_t c = (uint32_t)(stid & 15), in_row = swz(t, c & 7u);
        const uint32_t to = y + (c >> 3) * kBlock + (uint32_t)b * (kSlice * 128) + in_row;
        const uint32_t ring = sb + OFF_W + (uint32_t)slot * (NT - 1) * kSliceTile + (c >> 3) * kSliceBlock + in_row;
        const uint4 yv[2] = {lds_v4(to), lds_v4(to + 2048)};
        const uint32_t be = dec(s) + DEC_BETA + (b * kSlice + t) * 4;
        const float w[2] = {wb * lds_f32(be), wb * lds_f32(be + 64)};
        if (n >= SLOTS) ok = wait_warp(BAR_EMPTY + slot, (uint32_t)(n / SLOTS) + 1u);
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t yw[4] = {yv[q].x, yv[q].y, yv[q].z, yv[q].w};
          const float2 w2 = make_float2(w[q], w[q]), minus = make_float2(-1.f, -1.f);
          uint32_t part[3][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // the first terms are cut, the last rounded: 8 bits each, the signs all the same
            float2 v = mul2(pair(yw[j] << 16, yw[j] & 0xffff0000u), w2);
#pragma unroll
            for (int p = 0; p < NT; ++p) {
              part[p][j] = p + 1 < NT ? pack_cut(v) : pack_bf16x2(v.x, v.y);
              if (p + 1 < NT) v = fma2(cut2(v), minus, v);
            }
          }
          sts_v4(to + q * 2048, make_uint4(part[0][0], part[0][1], part[0][2], part[0][3]));
#pragma unroll
          for (int p = 1; p < NT; ++p)
            sts_v4(ring + (p - 1) * kSliceTile + q * 2048, make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]));
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_FULL + slot));
      }
      if (!ok) break;
      ok = wait_warp(BAR_U, (uint32_t)k);
      if (!ok) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t u[32];
        ptx::tmem_ld32(lanes + c * 32, u);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float *p = S + c * 32 + 2 * j;
          const float2 v = fma2(make_float2(g, g), make_float2(p[0], p[1]), pair(u[2 * j], u[2 * j + 1]));
          p[0] = v.x;
          p[1] = v.y;
        }
      }
      ptx::tc_fence_before();
      if (!only && k + 1 < nch) {
        ok = wait_warp(BAR_XS, (uint32_t)k);  // the last copy has been read
        if (!ok) break;
        write_state();
      }
      if (!BACK && r.marks && !only && ends_group(k)) {
        float4 *mark = reinterpret_cast<float4 *>(r.marks + mark_unit(k / kGroup) * (D * D)) + stid;
#pragma unroll
        for (int j = 0; j < 16; ++j) mark[j * 256] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
      }
    }
    float *dst = nullptr;
    bool dt = false;
    if (only) {
      dst = r.piece_state + (size_t)unit * D * D;
    } else if (r.fin && pc.s == (BACK ? 0 : pc.count - 1)) {
      dst = r.fin + ((size_t)pc.n * H + h) * D * D;
      dt = r.fin_t;
    }
    if (dst && ok) {
      if (!dt) {
#pragma unroll
        for (int j = 0; j < 64; ++j) dst[(half * 64 + j) * D + zrow] = S[j];
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          *reinterpret_cast<float4 *>(dst + zrow * D + half * 64 + 4 * j) =
              make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tm, 512);
  }
}

// dlog_a_t = sum_{t <= i in the group} (q_i . dq_i - k_i . dk_i) + <S, dLoss/dS> behind the group.  The dots carry
// bf16 products whose errors would add up along a sequence; the marks' product starts each group afresh.
// A warp per group of kGroup chunks, 16 tokens a lane.
constexpr int kDlogWarps = 4;
__global__ void __launch_bounds__(32 * kDlogWarps) dlog_tc_kernel(const float *dots_q, const float *dots_k,
                                                                  const float *mark_dots, Cut c, __nv_bfloat16 *dlog) {
  constexpr int kTokens = kGroup * C, kEach = kTokens / 32;
  const int H = c.H, unit = blockIdx.x, h = unit % H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Piece pc;
  if (!find_piece(c, unit / H, &pc)) return;
  for (int g = blockIdx.y * kDlogWarps + warp; g * kTokens < pc.len; g += gridDim.y * kDlogWarps) {
    const size_t t0 = (size_t)pc.t0 + (size_t)g * kTokens;
    const int cnt = min(kTokens, pc.len - g * kTokens), first = lane * kEach;
    float v[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const size_t at = (t0 + first + j) * H + h;
      v[j] = first + j < cnt ? dots_q[at] - dots_k[at] : 0.f;
    }
#pragma unroll
    for (int j = kEach - 2; j >= 0; --j) v[j] += v[j + 1];
    const float own = v[0];
    float incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float down = __shfl_down_sync(0xffffffffu, incl, d);
      if (lane + d < 32) incl += down;
    }
    const float *end = mark_dots + ((size_t)mark_slot(unit / H, (int)t0) * H + h) * 8;
    float behind = incl - own;
#pragma unroll
    for (int w = 0; w < 8; ++w) behind += end[w];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (first + j < cnt) dlog[(t0 + first + j) * H + h] = __float2bfloat16_rn(v[j] + behind);
  }
}

template <bool BACK, int NT>
cudaError_t launch_t(const TcRun &P, cudaStream_t s) {
  auto kern = run_tc_kernel<BACK, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((int64_t)P.r.cut.n_pieces * P.r.cut.H), kThreads, kSmemBytes, s>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_run_tc(const Run &r, int terms, int32_t *status, cudaStream_t s) {
  TcRun P;
  memset(&P, 0, sizeof(P));
  P.r = r;
  P.status = status;
  P.wait_ns = kWaitNs;
  const int64_t T = r.cut.t_total;
  if (T > 0) {
    bool ok = make_row_tile_map(&P.tm_y, r.y, T, r.Hy, C) && make_row_tile_map(&P.tm_z, r.z, T, r.Hz, C);
    if (ok && !r.state_only) ok = make_row_tile_map(&P.tm_x, r.x, T, r.Hx, C);
    if (ok && !r.state_only && !r.out_f32) ok = make_row_tile_map(&P.tm_o, r.out, T, r.cut.H, C);
    if (!ok) return cudaErrorInvalidValue;
  }
  uint64_t hook_ns = 0;
  if (take_debug_timeout(GDN2_DEBUG_LINATTN, &hook_ns)) {
    P.dbg_skip = 1;
    P.wait_ns = hook_ns;
  }
  if (r.back) return terms == 3 ? launch_t<true, 3>(P, s) : launch_t<true, 2>(P, s);
  return terms == 3 ? launch_t<false, 3>(P, s) : launch_t<false, 2>(P, s);
}

cudaError_t launch_dlog_tc(const float *dots_q, const float *dots_k, const float *mark_dots, const Cut &c, void *dlog,
                           cudaStream_t s) {
  if (c.t_total == 0) return cudaSuccess;
  const int64_t groups = (int64_t)c.t_total / (kGroup * C * kDlogWarps) + 1;  // of the longest piece, at most
  const dim3 grid((unsigned)((int64_t)c.n_pieces * c.H), (unsigned)(groups < 16 ? groups : 16));
  dlog_tc_kernel<<<grid, 32 * kDlogWarps, 0, s>>>(dots_q, dots_k, mark_dots, c, static_cast<__nv_bfloat16 *>(dlog));
  return cudaGetLastError();
}

}  // namespace lin
}  // namespace gdn2
