// linattn_tc.cu -- one run of linear attention with a decay per head on the tensor cores
// (d_k = d_v = 128, bf16): out_t = sum_j e^{|L_t - L_j|..} (x_t . y_j) z_j + (state part), chunks of
// 128 tokens, a CTA per (piece, head) that walks its chunks in order (last first when BACK).
//
// Per chunk, with D the matrix of decays inside the chunk (0 outside the triangle), w_j the decay
// from token j to the chunk's far end, f_i the decay from its near end to token i, g the chunk's:
//   G = X Y^T,  P = bf16(G o D)           (rows = tokens; P becomes a TMEM operand)
//   out = P Z + f o (X S)
//   U = (w o Y)^T Z,  S <- g S + U        (fp32, rounded to nearest)
// Where the chunk's decay stays above 2^-32, D_ij = f_i / f_j is not needed: out = f o (X S + P' Z)
// with P' = bf16(G_ij / f_j), one accumulator and one product a weight.  (Not where the rows' dots with
// m are asked for: dlog_a is a difference of the dots of two runs, and the same P, rounded the same
// way in both, falls out of it; with P' it was off by 1% over 4096 tokens.)  Chunks of stronger decay
// (resets) take D block by block.
// The state is held in fp32: w o Y goes to the tensor cores as a sum of NT bf16 values (4 give 26
// bits, 2 give 17, for runs whose state only feeds bf16 products), Z is bf16 already, and g is a sum of two
// floats.  The tensor cores cut sums toward zero.  With S as the accumulator itself that loss added up
// over the chunks, by an amount that depends on the inputs; giving its average back left 8e-6 at 65000 tokens
// without a decay, and states that nothing was written to grew by it.  So every chunk's sum starts from
// zero and is added to S on the CUDA cores: S is off by what one chunk's products lose, at most 6e-7 in
// the norm (100 to 65000 tokens), and a chunk that writes nothing leaves it as it was.
//
// Memory is its floor: 4 tiles of 32 KB a chunk, 128 KB against 2.9 us of 6.6 TB/s / 148 SMs; the products
// take 5 x 512 (NT = 2) or 7 x 512 tensor cycles.  What a chunk takes is one round of its chain, 7100 cycles in
// the forward: G (570 until it is seen), P's warps read it (1050), U (3000: a slice waits for its slot of tensor
// memory, which is full), U is added to S (1050 and 550 to see it), then the next G.  The other steps run beside it,
// each in a group of warps of its own: warp 0 loads; warp 1 issues the state's products, warp 3 the rows' (G,
// X S, P Z); warp 2 sums the decays; warps 4-11 write P, half a token row a thread, and warps 12-19 out;
// warps 20-27 add U to the state, copy it to bf16 for X S and weight Y, transposed into tensor memory: with
// w o Y in shared memory (every term written, and read with Z) that memory's 128 bytes a cycle were short,
// and they still are what the CUDA cores wait for while products run.  X has one tile, Y and Z two stages.
// The loops stay rolled, and what few calls need stands outside them or is compiled out: unrolled, or with such
// code to jump over, the roles ran out of the instruction cache (8 x 4096 tokens: 182 us for 162).
#include <cmath>
#include <cstring>

#include "linattn.cuh"
#include "tc_util.cuh"

namespace gdn2 {
namespace lin {
namespace {

using namespace gdn2::tc;

constexpr int D = 128;
constexpr int C = kChunk;
constexpr int kRows0 = 4, kOut0 = 12, kState0 = 20;  // first warps of the groups of 8
constexpr int kThreads = 32 * 28;
constexpr uint32_t kTile = C * D * 2;       // 32 KB, two column blocks of 64
constexpr uint32_t kBlock = kTile / 2;
constexpr uint32_t OFF_X = 0, OFF_Y = kTile, OFF_Z = 3 * kTile;  // Y, Z: two stages
constexpr uint32_t OFF_S = 5 * kTile;       // the bf16 state, [dy][dz]
constexpr uint32_t OFF_O = 6 * kTile;       // out
constexpr uint32_t OFF_MISC = 7 * kTile;
// For the rows, mild chunks: f and 1 / f of each token, and 1; others: the decay from each token to
// the edge of its 32-token block (log2), 2^(block total - that), the four block totals (not above
// 0).  For the state (two stages): for each pair of tokens their weights as three bf16 pairs, then the
// chunk's decay as a sum of two floats.
constexpr uint32_t DEC_EDGE = 0, DEC_BETA = 512, DEC_TOT = 1024, DEC_W = 1040, DEC_G = 64 * 12, DEC_STAGE = 64 * 12 + 16;
constexpr uint32_t MISC_BAR = DEC_W + 2 * DEC_STAGE;
constexpr long long kMild = 32ll << 32;  // 2^-32, in the decays' units
// A waiter must not look so late that the phase after next is over: where nothing else keeps it, a
// barrier of each parity of the chunk does.
enum {
  BAR_Y = 0,        // + stage: Y loaded
  BAR_Z = 2,        // + stage: Z loaded
  BAR_FREE = 4,     // + stage: nothing uses Y and Z any more
  BAR_DEC = 6,      // + stage: the state's weights there
  BAR_WFREE = 8,    // + stage: and used
  BAR_FULL = 10,    // + slot: a slice of w o Y written
  BAR_EMPTY = 12,   // + slot: its products done
  BAR_U = 14,       // + parity: U done
  BAR_UREAD = 16,   // + parity: and read
  BAR_ROWDEC = 18,  // the rows' decays there
  BAR_ROWFREE,      // and used
  BAR_X,            // X loaded
  BAR_XS,           // X S done, X and the state's copy free
  BAR_G,            // X Y^T done
  BAR_GREAD,        // and read
  BAR_P,            // P written, and X S scaled where it has to be
  BAR_PZ,           // P Z done
  BAR_OREAD,        // out read
  BAR_S,            // the state's copy written
  BAR_CLEAN,        // Y's and Z's rows behind the sequence cleared
  BAR_DRAIN,        // + 0, 1
  N_BARS = BAR_DRAIN + 2
};
constexpr uint32_t MISC_TMEM = MISC_BAR + N_BARS * 8, MISC_ABORT = MISC_TMEM + 4;
constexpr uint32_t MISC_BYTES = MISC_ABORT + 4;
constexpr uint32_t kSmemBytes = OFF_MISC + MISC_BYTES;
static_assert(kSmemBytes <= 232448, "shared memory over the sm_100 limit per CTA");
// TMEM columns.  U takes G's place once P's warps have read G (all 512 are taken); runs without rows have
// it there and in out's place in turn.  TM_W: two slices of w o Y.
constexpr uint32_t TM_G = 0, TM_OUT = 128, TM_S = 256, TM_P = 384, TM_W = 448;
constexpr uint32_t kSlot = 32;
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
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t *>(&v); }
// bf16 pairs whose sum is (w0 + w1 + w2) y to 26 bits (NT = 4) or (w0 + w1) y to 17 (NT = 2): the
// product of two bf16 is the rounded one and a remainder that bf16 holds exactly.  Joining the
// remainder and the next product in one term takes seven more operations than a fourth product on
// the tensor cores, which have the time.
template <int NT>
__device__ __forceinline__ void weigh(__nv_bfloat162 y, __nv_bfloat162 w0, __nv_bfloat162 w1, __nv_bfloat162 w2,
                                      uint32_t (&part)[NT]) {
  const __nv_bfloat162 hi = __hmul2_rn(w0, y), lo = __hfma2(w0, y, __hneg2(hi));
  part[0] = bits(hi);
  if constexpr (NT == 2) {
    part[1] = bits(__hfma2(w1, y, lo));
  } else {
    const __nv_bfloat162 q = __hmul2_rn(w1, y);
    part[1] = bits(lo);
    part[2] = bits(q);
    part[3] = bits(__hfma2(w2, y, __hfma2(w1, y, __hneg2(q))));
  }
}
// 2^x for x <= 0 in units of 2^-32, as a sum of two floats: the states keep a chunk's factor for as long as
// they remember, so one float's error would add up over the chunks.  2^x = 2^n e^r, r = f ln 2, |f| <= 1/2; r in
// two parts, the Taylor series' terms from the square on in one float: off by about r^2 2^-23, 2^-25 at
// most, and by far less for the weak decays that are remembered long.
__device__ __forceinline__ float2 power2(long long x) {
  x = max(x, -(300ll << 32));
  const int n = (int)((x + (1ll << 31)) >> 32);
  const int d = (int)(x - ((long long)n << 32));            // f in the same units
  const float top = __int2float_rz(d), low = __int2float_rn(d - __float2int_rz(top));
  constexpr float kLn2 = 0.693147182f * 0x1p-32f, kLn2Lo = -1.90465421e-9f * 0x1p-32f;
  const float r = top * kLn2;
  const float r_lo = fmaf(top, kLn2, -r) + fmaf(top, kLn2Lo, low * kLn2);
  float e = 1.f / 40320.f;
  e = fmaf(e, r, 1.f / 5040.f);
  e = fmaf(e, r, 1.f / 720.f);
  e = fmaf(e, r, 1.f / 120.f);
  e = fmaf(e, r, 1.f / 24.f);
  e = fmaf(e, r, 1.f / 6.f);
  e = fmaf(e, r, 0.5f);
  const float rest = fmaf(e * r, r, r_lo);
  const float a = 1.f + r, b = r - (a - 1.f);               // 1 + r
  const float hi = a + (rest + b), lo = (rest + b) - (hi - a);
  return make_float2(ldexpf(hi, n), ldexpf(lo, n));
}
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

// WAY: 0 forward, 1 backward, 2 as the run says (97 KB of code for 78, and 3 to 9% more time a chunk:
// only the launch that needs both ways at once takes it).
template <int WAY, int NT>
__device__ __forceinline__ void run_block(const TcRun &P, int block) {
  constexpr int SLICE = 64 / NT;      // tokens of a slice of w o Y: NT terms in 32 columns, two slots
  constexpr int SLICES = C / SLICE;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Run &r = P.r;
  const bool BACK = WAY == 2 ? r.back != 0 : WAY == 1;
  const uint32_t sb = ptx::smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int H = r.cut.H;
  Piece pc;
  const bool only = r.state_only != 0;
  if (!find_unit(r.cut, block, only, &pc)) return;
  const int h = block % H;
  const size_t cut_unit = (size_t)pc.cut * H + h;
  // the runs with four terms that have a launch of their own (the forward's, dv's) have no dots, marks or fp32 rows
  constexpr bool PLAIN = WAY != 2 && NT == 4;
  const bool marks = !PLAIN && !only && r.marks, out_f32 = !PLAIN && r.out_f32;
  const __nv_bfloat16 *const m_all = PLAIN ? nullptr : static_cast<const __nv_bfloat16 *>(r.m);
  if (only && (pc.count < 2 || pc.s == (BACK ? 0 : pc.count - 1))) return;
  if (sb & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts on it
    if (tid == 0) atomicExch(P.status, kStatusTimeout);
    return;
  }
  const int nch = (pc.len + C - 1) / C;
  auto bar = [&](int b) { return sb + OFF_MISC + MISC_BAR + 8u * (uint32_t)b; };
  const uint32_t dec = sb + OFF_MISC;
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
      const bool group = b == BAR_OREAD || b == BAR_WFREE || b == BAR_WFREE + 1 || b == BAR_S || b == BAR_UREAD ||
                         b == BAR_UREAD + 1 || b == BAR_CLEAN || b == BAR_GREAD;
      const bool four = b == BAR_FULL || b == BAR_FULL + 1;                      // half a group
      const bool two = b == BAR_P || b == BAR_ROWFREE;                           // groups
      const bool both = (b == BAR_FREE || b == BAR_FREE + 1) && !only;           // issuers
      ptx::mbar_init(bar(b), group ? 8 : four ? 4 : two ? 16 : both ? 2 : 1);
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
      const bool skip = P.dbg_skip && block == 0;
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
        if (k >= 1 && !wait(BAR_XS, (uint32_t)k + 1u)) break;
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
    const bool lead = ptx::elect_one();
    constexpr uint32_t idKN = ptx::idesc_bf16(128, 128, false, true);
    bool ok = true;
    for (int k = 0; k < nch && ok; ++k) {
      const int s = k & 1;
      // where U goes is free: G has been read, which was formed after the last U had been read; without
      // rows, the last but one U has been read
      const uint32_t tu = tm + (only && s ? TM_OUT : TM_G);
      ok = wait_warp(BAR_Z + s, (uint32_t)(k >> 1));
      if (ok) ok = !only ? wait_warp(BAR_GREAD, (uint32_t)k) : k < 2 || wait_warp(BAR_UREAD + s, (uint32_t)(k >> 1) + 1u);
#pragma unroll 1
      for (int i = 0; i < SLICES && ok; ++i) {
        const int n = SLICES * k + i, slot = n & 1, t0 = (BACK ? SLICES - 1 - i : i) * SLICE;
        ok = wait_warp(BAR_FULL + slot, (uint32_t)(n >> 1));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t zd = mnmaj(sb + OFF_Z + (uint32_t)s * kTile + (uint32_t)t0 * 128u);
#pragma unroll
        for (int part = 0; part < NT; ++part)
#pragma unroll
          for (int kk = 0; kk < SLICE / 16; ++kk)
            ptx::umma_bf16_ts_if(lead, tu, tm + TM_W + (uint32_t)slot * kSlot + (uint32_t)(part * (SLICE / 2) + kk * 8),
                                 zd + kk * kMnStep, idKN, part > 0 || kk > 0 || i > 0);
        ptx::umma_commit_if(lead, bar(BAR_EMPTY + slot));
      }
      if (!ok) break;
      ptx::umma_commit_if(lead, bar(BAR_U + s));
      ptx::umma_commit_if(lead, bar(BAR_FREE + s));
    }
    ptx::umma_commit_if(lead, bar(BAR_DRAIN));  // all products, before the tensor memory is freed
    drain_bar(bar(BAR_DRAIN), 0u, P.wait_ns);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- the rows' products
    if (!only) {
      const bool lead = ptx::elect_one();
      constexpr uint32_t idKK = ptx::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idKN = ptx::idesc_bf16(128, 128, false, true);
      for (int k = 0; k < nch; ++k) {
        const int s = k & 1;
        const uint64_t x = kmaj(sb + OFF_X), y = kmaj(sb + OFF_Y + (uint32_t)s * kTile);
        const uint64_t z = mnmaj(sb + OFF_Z + (uint32_t)s * kTile), st = mnmaj(sb + OFF_S);
        if (!wait_warp(BAR_X, (uint32_t)k) || !wait_warp(BAR_Y + s, (uint32_t)(k >> 1))) break;
        if (rows_of(k) < C && !wait_warp(BAR_CLEAN, 0u)) break;
        if (k && !wait_warp(BAR_UREAD + (s ^ 1), (uint32_t)((k - 1) >> 1))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) ptx::umma_bf16_if(lead, tm + TM_G, x + k_step(kk), y + k_step(kk), idKK, kk > 0);
        ptx::umma_commit_if(lead, bar(BAR_G));
        if (!wait_warp(BAR_S, (uint32_t)k) || (k && !wait_warp(BAR_OREAD, (uint32_t)k + 1u))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::umma_bf16_if(lead, tm + TM_OUT, x + k_step(kk), st + kk * kMnStep, idKN, kk > 0);
        ptx::umma_commit_if(lead, bar(BAR_XS));
        if (!wait_warp(BAR_Z + s, (uint32_t)(k >> 1)) || !wait_warp(BAR_P, (uint32_t)k)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::umma_bf16_ts_if(lead, tm + TM_OUT, tm + TM_P + kk * 8, z + kk * kMnStep, idKN, 1u);
        ptx::umma_commit_if(lead, bar(BAR_PZ));
        ptx::umma_commit_if(lead, bar(BAR_FREE + s));
      }
      ptx::umma_commit_if(lead, bar(BAR_DRAIN + 1));
      drain_bar(bar(BAR_DRAIN + 1), 0u, P.wait_ns);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- decays
    // Lane l sums tokens 4 l .. 4 l + 3; 8 lanes are a block of 32 tokens.  The sums are whole numbers
    // of 2^-32 in log2 (a chunk may hold resets beside weak decays, which fp32 sums would blur; in
    // fp64 this warp took 5000 cycles a chunk, more than anything else).  Forward, `edge` of token i
    // is the decay from its block's start to it, itself included; backward, from it to the block's
    // end, itself not.
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
    using fix = long long;
    auto value = [](fix x) { return __ll2float_rn(x) * 0x1p-32f; };
    // 2^x: the whole part by the exponent, so that what is left keeps 24 bits
    auto power = [](fix x) {
      const int n = max((int)(x >> 32), -252), a = n >> 1;
      return ptx::ex2(__uint2float_rn((uint32_t)x) * 0x1p-32f) * __uint_as_float((uint32_t)(a + 127) << 23) *
             __uint_as_float((uint32_t)(n - a + 127) << 23);
    };
    fix logs = 0;
    bool lost = false;  // a NaN was among them: the state is NaN from there on
    float a[4];
    if (nch > 0) load(0, a);
    bool ok = true;
    for (int k = 0; k < nch && ok; ++k) {
      const uint32_t stage = dec + DEC_W + (uint32_t)(k & 1) * DEC_STAGE;
      fix own[4];  // inclusive sums inside the lane
      int nan = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        own[j] = __float2ll_rn(fmaxf(a[j], kMinLog) * kLog2 * 0x1p32f) + (j ? own[j - 1] : 0);
        nan |= (int)isnan(a[j]) << j;
      }
      const uint32_t nans = __ballot_sync(0xffffffffu, nan != 0);
      if (k + 1 < nch) load(k + 1, a);
      fix incl = own[3];
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const fix up = __shfl_up_sync(0xffffffffu, incl, d, 8);
        if ((lane & 7) >= d) incl += up;
      }
      const fix total = __shfl_sync(0xffffffffu, incl, 7, 8), before = incl - own[3];
      fix far = 0, all = 0;  // from the edge of the lane's block to the chunk's far end; the chunk's
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const fix t = __shfl_sync(0xffffffffu, total, 8 * b);
        all += t;
        if (BACK ? b < (lane >> 3) : b > (lane >> 3)) far += t;
      }
      logs = max(logs + all, kMinLogs);
      const bool mild = all >= -kMild;
      float2 g = power2(all);
      float one[4], two[4];
      uint32_t w[2][3];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const fix in = before + own[j], rest = BACK ? in : total - in;
        const float first = value(mild ? all - rest - far : BACK ? total - in : in);
        one[j] = mild ? ptx::ex2(first) : first;
        two[j] = ptx::ex2(mild ? -first : value(rest));
        float left = power(rest + far);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const uint32_t b = bf16_bits(left);
          left -= bf16_value((uint16_t)b);
          w[j >> 1][n] = j & 1 ? w[j >> 1][n] | b << 16 : b;
        }
      }
      if (nans) {  // the tokens that the state reaches through it, and the state
        lost = true;
        g.x = __int_as_float(0x7fc00000);
        bool hit = (BACK ? nans >> lane >> 1 : nans & ((1u << lane) - 1u)) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = BACK ? 3 - i : i;
          if (!BACK) hit |= (nan >> j & 1) != 0;
          if (hit) one[j] = g.x;
          if (BACK) hit |= (nan >> j & 1) != 0;
        }
      }
      if (k >= 2) ok = wait_warp(BAR_WFREE + (k & 1), (uint32_t)(k >> 1) + 1u);
      if (!ok) break;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int n = 0; n < 3; ++n) sts_u32(stage + 24 * lane + 12 * q + 4 * n, w[q][n]);
      if (lane == 0) sts_v2(stage + DEC_G, make_uint2(__float_as_uint(g.x), __float_as_uint(g.y)));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(BAR_DEC + (k & 1)));
      if (!only) {
        if (k) ok = wait_warp(BAR_ROWFREE, (uint32_t)k + 1u);
        if (!ok) break;
        sts_v4(dec + DEC_EDGE + 16 * lane, make_uint4(__float_as_uint(one[0]), __float_as_uint(one[1]),
                                                      __float_as_uint(one[2]), __float_as_uint(one[3])));
        sts_v4(dec + DEC_BETA + 16 * lane, make_uint4(__float_as_uint(two[0]), __float_as_uint(two[1]),
                                                      __float_as_uint(two[2]), __float_as_uint(two[3])));
        if ((lane & 7) == 0) sts_f32(dec + DEC_TOT + (lane >> 3) * 4, mild ? 1.f : value(total));
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_ROWDEC));
      }
    }
    if (only && lane == 0) r.piece_log[cut_unit] = lost ? (double)NAN : (double)logs * (0x1p-32 / (double)kLog2);
  } else if (warp < kOut0) {
    // ---------------------------------------------------------------- P: half a token row a thread
    const int wq = warp & 3, row = wq * 32 + lane, half = (warp - kRows0) >> 2;
    const uint32_t lanes = tm + ((uint32_t)(wq * 32) << 16);
    for (int k = 0; k < (only ? 0 : nch); ++k) {
      if (!wait_warp(BAR_ROWDEC, (uint32_t)k)) break;
      const float edge = lds_f32(dec + DEC_EDGE + row * 4);
      const bool mild = lds_f32(dec + DEC_TOT) > 0.f;
      if (!wait_warp(BAR_G, (uint32_t)k)) break;
      ptx::tc_fence_after();
      // two of the four blocks of 32 columns each
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int cb = 2 * half + i;
        const bool none = BACK ? cb < wq : cb > wq;
        uint32_t out[16], g[32];
        if (!none) {
          ptx::tmem_ld32(lanes + TM_G + cb * 32, g);
          ptx::tmem_wait_ld();
        }
        if (i) {  // U may take G's place
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(BAR_GREAD));
        }
        if (none) {
#pragma unroll
          for (int j = 0; j < 16; ++j) out[j] = 0u;
        } else {
          if (mild) {
            const float2 f2 = m_all ? make_float2(edge, edge) : make_float2(1.f, 1.f);
#pragma unroll
            for (int j4 = 0; j4 < 8; ++j4) {
              const float4 be = lds_f4(dec + DEC_BETA + cb * 128 + j4 * 16);
              const float2 v = mul2(mul2(f2, make_float2(be.x, be.y)), pair(g[4 * j4], g[4 * j4 + 1]));
              const float2 u = mul2(mul2(f2, make_float2(be.z, be.w)), pair(g[4 * j4 + 2], g[4 * j4 + 3]));
              out[2 * j4] = pack_bf16x2(v.x, v.y);
              out[2 * j4 + 1] = pack_bf16x2(u.x, u.y);
            }
            if (cb == wq)
#pragma unroll
              for (int j = 0; j < 16; ++j)
                out[j] &= ((BACK ? 2 * j >= lane : 2 * j <= lane) ? 0xffffu : 0u) |
                          ((BACK ? 2 * j + 1 >= lane : 2 * j + 1 <= lane) ? 0xffff0000u : 0u);
          } else if (cb == wq) {
            // both tokens in one block: the decay between them, pair by pair
            const float2 minus = make_float2(-1.f, -1.f), e2 = make_float2(edge, edge);
#pragma unroll
            for (int j4 = 0; j4 < 8; ++j4) {
              const float4 e = lds_f4(dec + DEC_EDGE + cb * 128 + j4 * 16);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int j = j4 * 4 + 2 * q;
                const float2 d = fma2(q ? make_float2(e.z, e.w) : make_float2(e.x, e.y), minus, e2);
                const float2 v = mul2(make_float2(ptx::ex2(d.x), ptx::ex2(d.y)), pair(g[j], g[j + 1]));
                out[2 * j4 + q] = pack_bf16x2((BACK ? j >= lane : j <= lane) ? v.x : 0.f,
                                              (BACK ? j + 1 >= lane : j + 1 <= lane) ? v.y : 0.f);
              }
            }
          } else {
            // through the edges of the two blocks: a row factor times a column factor, both <= 1
            float between = edge;
            for (int b = BACK ? wq + 1 : cb + 1; b < (BACK ? cb : wq); ++b) between += lds_f32(dec + DEC_TOT + b * 4);
            const float alpha = ptx::ex2(between);
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
            for (int j4 = 0; j4 < 8; ++j4) {
              const float4 be = lds_f4(dec + DEC_BETA + cb * 128 + j4 * 16);
              const float2 v = mul2(mul2(a2, make_float2(be.x, be.y)), pair(g[4 * j4], g[4 * j4 + 1]));
              const float2 u = mul2(mul2(a2, make_float2(be.z, be.w)), pair(g[4 * j4 + 2], g[4 * j4 + 3]));
              out[2 * j4] = pack_bf16x2(v.x, v.y);
              out[2 * j4 + 1] = pack_bf16x2(u.x, u.y);
            }
          }
        }
        ptx::tmem_st16(lanes + TM_P + cb * 16, out);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(bar(BAR_ROWFREE));
        ptx::mbar_arrive(bar(BAR_P));
      }
    }
  } else if (warp < kState0) {
    // ---------------------------------------------------------------- out: half a token row a thread
    const int wq = warp & 3, row = wq * 32 + lane, half = (warp - kOut0) >> 2;
    const uint32_t lanes = tm + ((uint32_t)(wq * 32) << 16) + TM_OUT + half * 64;
    const uint32_t tile = sb + OFF_O + (uint32_t)half * kBlock;
    for (int k = 0; k < (only ? 0 : nch); ++k) {
      const bool in = row < rows_of(k);
      const size_t tok = (size_t)pc.t0 + (size_t)chunk_no(k) * C + row;
      const __nv_bfloat16 *m = nullptr;
      if (m_all && in) {
        m = m_all + (tok * r.Hm + h / (H / r.Hm)) * D + half * 64;
        prefetch_l2(m);
      }
      if (!wait_warp(BAR_ROWDEC, (uint32_t)k)) break;
      float f = lds_f32(dec + DEC_EDGE + row * 4);
      const bool mild = lds_f32(dec + DEC_TOT) > 0.f;
      if (!mild) {
        for (int b = BACK ? wq + 1 : 0; b < (BACK ? 4 : wq); ++b) f += lds_f32(dec + DEC_TOT + b * 4);
        f = ptx::ex2(f);
      }
      float2 f2 = make_float2(f, f);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(BAR_ROWFREE));
      if (!mild || m_all) {
        if (!wait_warp(BAR_XS, (uint32_t)k)) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[16];
          ptx::tmem_ld16(lanes + c * 16, v);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(f * __uint_as_float(v[j]));
          ptx::tmem_st16(lanes + c * 16, v);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        f2 = make_float2(1.f, 1.f);
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(bar(BAR_P));
        ptx::bulk_wait_group_read0();  // this warp's rows of the tile
      }
      float2 dot = make_float2(0.f, 0.f);
      const bool whole = wq * 32 + 32 <= rows_of(k) && !out_f32;
      uint4 mw[2];  // 16 values of m's row, asked for one step ahead
      if (m)
#pragma unroll
        for (int j = 0; j < 2; ++j) mw[j] = *reinterpret_cast<const uint4 *>(m + 8 * j);
      if (!wait_warp(BAR_PZ, (uint32_t)k)) break;
      ptx::tc_fence_after();
      const size_t at_out = (tok * H + h) * D + half * 64;
#pragma unroll 1
      for (int cb = 0; cb < 4; ++cb) {
        __syncwarp();
        uint32_t u[16];
        ptx::tmem_ld16(lanes + cb * 16, u);
        ptx::tmem_wait_ld();
        float2 o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = mul2(f2, pair(u[2 * j], u[2 * j + 1]));
        if (m)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w[4] = {mw[j].x, mw[j].y, mw[j].z, mw[j].w};
            if (cb < 3) mw[j] = *reinterpret_cast<const uint4 *>(m + (cb + 1) * 16 + 8 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot = fma2(pair(w[i] << 16, w[i] & 0xffff0000u), o[4 * j + i], dot);
          }
        if (out_f32) {
          if (in) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(r.out) + at_out + cb * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = make_float4(o[2 * j].x, o[2 * j].y, o[2 * j + 1].x, o[2 * j + 1].y);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 w = make_uint4(pack_bf16x2(o[4 * j].x, o[4 * j].y), pack_bf16x2(o[4 * j + 1].x, o[4 * j + 1].y),
                                       pack_bf16x2(o[4 * j + 2].x, o[4 * j + 2].y), pack_bf16x2(o[4 * j + 3].x, o[4 * j + 3].y));
            if (whole) sts_v4(tile + swz(row, (uint32_t)(2 * cb + j)), w);
            else if (in) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(r.out) + at_out + cb * 16 + 8 * j) = w;
          }
        }
      }
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(bar(BAR_OREAD));
        if (whole) {
          ptx::tma_store_3d(&P.tm_o, tile + (uint32_t)wq * 4096u, half * 64, h, pc.t0 + chunk_no(k) * C + wq * 32);
          ptx::bulk_commit_group();
        }
      }
      if (m) r.dots[(size_t)(half * H + h) * r.cut.t_total + tok] = dot.x + dot.y;
    }
    if (lane == 0) ptx::bulk_wait_group0();
  } else {
    // ---------------------------------------------------------------- state (warp: 32 y rows x 64 z columns) and w o Y
    // (warp: 32 y columns, every other slice)
    const int wq = warp & 3, half = (warp - kState0) >> 2, yrow = wq * 32 + lane, stid = tid - 32 * kState0;
    const uint32_t quad = tm + ((uint32_t)(wq * 32) << 16);
    // 16 columns of a state in memory: [dy][dz], or [dz][dy] with `flip`
    auto load_state = [&](const float *p, bool flip, int z0, uint32_t (&v)[16]) {
      if (!flip) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = *reinterpret_cast<const uint4 *>(p + yrow * D + z0 + 4 * j);
          v[4 * j] = w.x; v[4 * j + 1] = w.y; v[4 * j + 2] = w.z; v[4 * j + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(p[(z0 + j) * D + yrow]);
      }
    };
    // this thread's 64 columns of the state in tensor memory: to memory, to a mark, and multiplied with one
    auto put_state = [&](float *p, bool flip) {
#pragma unroll 1
      for (int z0 = 64 * half; z0 < 64 * half + 64; z0 += 16) {
        uint32_t v[16];
        ptx::tmem_ld16(quad + TM_S + z0, v);
        ptx::tmem_wait_ld();
        if (!flip) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(p + yrow * D + z0 + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) p[(z0 + j) * D + yrow] = __uint_as_float(v[j]);
        }
      }
    };
    auto put_mark = [&](size_t mu) {
      float *p = r.marks + mu * (D * D) + 4 * yrow;
#pragma unroll 1
      for (int z0 = 64 * half; z0 < 64 * half + 64; z0 += 16) {
        uint32_t v[16];
        ptx::tmem_ld16(quad + TM_S + z0, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4 *>(p + (z0 / 4 + j) * 512) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    };
    auto dot_mark = [&](size_t mu) {
      const float *p = r.marks + mu * (D * D) + 4 * yrow;
      float dot = 0.f;
#pragma unroll 1
      for (int z0 = 64 * half; z0 < 64 * half + 64; z0 += 16) {
        uint32_t v[16];
        float4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const float4 *>(p + (z0 / 4 + j) * 512);
        ptx::tmem_ld16(quad + TM_S + z0, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dot = fmaf(w[j].x, __uint_as_float(v[4 * j]), fmaf(w[j].y, __uint_as_float(v[4 * j + 1]),
                fmaf(w[j].z, __uint_as_float(v[4 * j + 2]), fmaf(w[j].w, __uint_as_float(v[4 * j + 3]), dot))));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      if (lane == 0) r.mark_dots[mu * kMarkDots + (warp - kState0)] = dot;
    };
    // this lane's row of the four matrices (8 columns x 8 tokens) of 16 columns and 16 tokens
    const int row = ((lane >> 4) << 3) | (lane & 7);
    const uint32_t chunk = (uint32_t)(wq & 1) * 4u + (uint32_t)(lane >> 3 & 1);
    const uint32_t mine = (uint32_t)(wq >> 1) * kBlock;
    // this half's slices first .. last - 1 (in the order of the walk) of chunk k's w o Y, two tokens to a word,
    // transposed into the half's own slot of tensor memory
    auto weigh_slices = [&](int k, int first, int last) {
      const int s = k & 1;
      const uint32_t y = sb + OFF_Y + (uint32_t)s * kTile;
#pragma unroll 1
      for (int i = first; i < last; ++i) {
        const int n = SLICES / 2 * k + i, t0 = (BACK ? SLICES - 1 - (2 * i + half) : 2 * i + half) * SLICE;
        uint32_t terms[SLICE / 16][2][NT][4];
#pragma unroll
        for (int t = 0; t < SLICE / 16; ++t) {
          // weights of the pairs of tokens that this lane's columns of the matrices are
          const uint32_t ws = dec + DEC_W + (uint32_t)s * DEC_STAGE + (uint32_t)(t0 / 2 + 8 * t + (lane & 3)) * 12u;
          __nv_bfloat162 w[2][3];
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < (NT == 2 ? 2 : 3); ++j) w[q][j] = bf2(__float_as_uint(lds_f32(ws + 48 * q + 4 * j)));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t yw[4];
            ptx::ldmatrix4_trans(y + mine + (uint32_t)(t0 + 16 * t) * 128u + swz(row, chunk + 2u * c), yw);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              uint32_t got[NT];
              weigh<NT>(bf2(yw[p]), w[p >> 1][0], w[p >> 1][1], w[p >> 1][2], got);
#pragma unroll
              for (int m = 0; m < NT; ++m) terms[t][c][m][p] = got[m];
            }
          }
        }
        if (n && !wait_warp(BAR_EMPTY + half, (uint32_t)n + 1u)) return false;
        ptx::tc_fence_after();
#pragma unroll
        for (int t = 0; t < SLICE / 16; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < NT; ++m)
              ptx::tmem_st_16x8(quad + TM_W + ((uint32_t)(16 * c) << 16) + (uint32_t)half * kSlot +
                                    (uint32_t)(m * (SLICE / 2) + 8 * t),
                                terms[t][c][m]);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(BAR_FULL + half));
      }
      return true;
    };
    const float *start = nullptr;
    float *dst = nullptr;
    bool flip_start = false, flip_dst = false;
    if (only) {
      dst = r.piece_state + cut_unit * D * D;
    } else {
      if (r.piece_state && pc.count > 1) {
        start = r.piece_state + cut_unit * D * D;
      } else if (r.start) {
        start = r.start + ((size_t)pc.n * H + h) * D * D;
        flip_start = r.start_t;
      }
      if (r.fin && pc.s == (BACK ? 0 : pc.count - 1)) {
        dst = r.fin + ((size_t)pc.n * H + h) * D * D;
        flip_dst = r.fin_t;
      }
    }
#pragma unroll 1
    for (int c = 4 * half; c < 4 * half + 4; ++c) {
      uint32_t v[16], zero[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = zero[j] = 0u;
      if (start) load_state(start, flip_start, c * 16, v);
      __syncwarp();
      ptx::tmem_st16(quad + TM_S + c * 16, zero);
      ptx::tmem_st16(quad + TM_OUT + c * 16, v);  // as if it were the U of a chunk before the first
    }
    ptx::tmem_wait_st();
    // marks of this thread's part of the state behind group `g` of chunks
    auto mark_unit = [&](int g) { return (size_t)mark_slot(pc.unit / H, pc.t0 + g * kGroup * C) * H + h; };
    auto ends_group = [&](int no) { return (no + 1) % kGroup == 0 || no == nch - 1; };
    float2 g2 = make_float2(1.f, 0.f);  // the last chunk's decay
    for (int k = 0; k <= nch; ++k) {
      const int s = k & 1;
      const uint32_t par = (uint32_t)(k >> 1);
      const bool last = k == nch;
      if (!last) {
        const int rows = rows_of(k);
        const uint32_t y = sb + OFF_Y + (uint32_t)s * kTile;
        if (!wait_warp(BAR_DEC + s, par) || !wait_warp(BAR_Y + s, par)) break;
        if (rows < C) {
          // rows behind the sequence meet zero weights, which a NaN would outlive
          if (!wait_warp(BAR_Z + s, par)) break;
          for (int t = stid >> 4; t < C; t += 16)
            if (t >= rows) {
              const uint32_t to = y + (uint32_t)(stid >> 3 & 1) * kBlock + swz(t, (uint32_t)(stid & 7));
              sts_v4(to, make_uint4(0u, 0u, 0u, 0u));
              sts_v4(to + (OFF_Z - OFF_Y), make_uint4(0u, 0u, 0u, 0u));
            }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(BAR_CLEAN));
          if (!wait_warp(BAR_CLEAN, 0u)) break;  // other warps' rows are read too
        }
        // the first slice, while the last U is still summed
        if (!weigh_slices(k, 0, 1)) break;
      }
      // the state before the k-th chunk walked, and its copy for X S.  This loop is what a chunk waits for:
      // all that only some calls or chunks do stands behind it (jumped over in it, it cost half as much again).
      if (k && !wait_warp(BAR_U + (s ^ 1), (uint32_t)((k - 1) >> 1))) break;
      if (k && !only && !wait_warp(BAR_XS, (uint32_t)k + 1u)) break;  // the last copy has been read
      ptx::tc_fence_after();
      {
        const uint32_t tu = quad + (k == 0 || (only && !s) ? TM_OUT : TM_G);  // U of chunk k - 1
        const float2 hi2 = make_float2(g2.x, g2.x), lo2 = make_float2(g2.y, g2.y);
#pragma unroll 1
        for (int c = 4 * half; c < 4 * half + 4; ++c) {  // 16 columns each
          uint32_t v[16], u[16];
          ptx::tmem_ld16(quad + TM_S + c * 16, v);
          ptx::tmem_ld16(tu + c * 16, u);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 x = pair(v[2 * j], v[2 * j + 1]);
            const float2 w = fma2(hi2, x, fma2(lo2, x, pair(u[2 * j], u[2 * j + 1])));
            v[2 * j] = __float_as_uint(w.x);
            v[2 * j + 1] = __float_as_uint(w.y);
            u[j] = pack_bf16x2(w.x, w.y);
          }
          ptx::tmem_st16(quad + TM_S + c * 16, v);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            sts_v4(sb + OFF_S + half * kBlock + swz(yrow, (uint32_t)(2 * (c & 3) + j)),
                   make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]));
        }
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (k) ptx::mbar_arrive(bar(BAR_UREAD + (s ^ 1)));
        ptx::mbar_arrive(bar(BAR_S));
      }
      if (last) {
        if (dst) put_state(dst, flip_dst);
        if (!BACK && k && marks) put_mark(mark_unit((k - 1) / kGroup));
        break;
      }
      if (marks) {
        const int no = chunk_no(k);  // forward: the group in front of chunk k is done; backward: k's begins
        if (!BACK && k && ends_group(k - 1)) put_mark(mark_unit((k - 1) / kGroup));
        if (BACK && ends_group(no)) {
          const size_t mu = mark_unit(no / kGroup);
          if (WAY == 1 || r.mark_dots) dot_mark(mu);
          else put_mark(mu);
        }
        // the next group's mark, two chunks ahead
        if (BACK && (WAY == 1 || r.mark_dots) && no % kGroup == 1 && no > kGroup) {
          const char *next = reinterpret_cast<const char *>(r.marks + mark_unit(no / kGroup - 1) * (D * D)) + stid * 128;
          prefetch_l2(next);
          prefetch_l2(next + 32768);
        }
      }
      if (!weigh_slices(k, 1, SLICES / 2)) break;
      const uint32_t gs = dec + DEC_W + (uint32_t)s * DEC_STAGE + DEC_G;
      g2 = make_float2(lds_f32(gs), lds_f32(gs + 4));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(BAR_WFREE + s));
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

template <int WAY, int NT>
__global__ void __launch_bounds__(kThreads, 1) run_tc_kernel(const __grid_constant__ TcRun P) {
  run_block<WAY, NT>(P, blockIdx.x);
}
// The three runs of the gradients side by side (dq, dv, dk), where one alone leaves SMs idle or would
// need its sequences cut.  All with the terms that dv needs: a body for each number of terms made the
// kernel larger than the instruction caches hold, and every chunk slower.
struct TcGrads {
  TcRun run[3];
};
__global__ void __launch_bounds__(kThreads, 1) grads_tc_kernel(const __grid_constant__ TcGrads P) {
  run_block<2, 4>(P.run[blockIdx.x % 3], blockIdx.x / 3);
}

// mark_dots of two runs' marks.
__global__ void __launch_bounds__(256) marks_kernel(const float *a, const float *b, float *mark_dots, Cut c) {
  static_assert(kMarkDots == 8, "a partial sum a warp");
  const int H = c.H, unit = blockIdx.x, h = unit % H;
  Piece pc;
  if (!find_piece(c, unit / H, &pc)) return;
  for (int g = blockIdx.y; g * kGroup * C < pc.len; g += gridDim.y) {
    const size_t mu = (size_t)mark_slot(unit / H, pc.t0 + g * kGroup * C) * H + h;
    const float4 *x = reinterpret_cast<const float4 *>(a + mu * (D * D)) + threadIdx.x;
    const float4 *y = reinterpret_cast<const float4 *>(b + mu * (D * D)) + threadIdx.x;
    float dot = 0.f;
#pragma unroll 8
    for (int j = 0; j < D * D / 1024; ++j) {
      const float4 v = x[j * 256], w = y[j * 256];
      dot = fmaf(v.x, w.x, fmaf(v.y, w.y, fmaf(v.z, w.z, fmaf(v.w, w.w, dot))));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if ((threadIdx.x & 31) == 0) mark_dots[mu * kMarkDots + (threadIdx.x >> 5)] = dot;
  }
}

// dlog_a_t = sum_{t <= i in the group} (q_i . dq_i - k_i . dk_i) + <S, dLoss/dS> behind the group.  The dots carry
// bf16 products whose errors would add up along a sequence; the marks' product starts each group afresh.
// It is a_t <S_{t-1}, dLoss/dS_t>: exactly 0 at a reset, where the sums leave the roundings of what cancels.
// A warp per group of kGroup chunks.
constexpr int kDlogWarps = 4;
__global__ void __launch_bounds__(32 * kDlogWarps) dlog_tc_kernel(const float *dots_q, const float *dots_k,
                                                                  const float *mark_dots, const __nv_bfloat16 *log_a,
                                                                  Cut c, int no_start, __nv_bfloat16 *dlog) {
  constexpr int kTokens = kGroup * C;
  const int H = c.H, unit = blockIdx.x, h = unit % H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Piece pc;
  if (!find_piece(c, unit / H, &pc)) return;
  const size_t half = (size_t)H * c.t_total;  // the dots of the other half of the columns
  for (int g = blockIdx.y * kDlogWarps + warp; g * kTokens < pc.len; g += gridDim.y * kDlogWarps) {
    const size_t t0 = (size_t)pc.t0 + (size_t)g * kTokens, at = (size_t)h * c.t_total + t0;
    const int cnt = min(kTokens, pc.len - g * kTokens);
    float v[kTokens / 32];
    uint32_t resets = 0;
#pragma unroll
    for (int j = 0; j < kTokens / 32; ++j) {
      const size_t i = at + 32 * j + lane;
      if (32 * j + lane < cnt && __bfloat162float(log_a[(t0 + 32 * j + lane) * H + h]) <= kMinLog) resets |= 1u << j;
      v[j] = 32 * j + lane < cnt ? (dots_q[i] + dots_q[half + i]) - (dots_k[i] + dots_k[half + i]) : 0.f;
    }
    const float *end = mark_dots + ((size_t)mark_slot(unit / H, (int)t0) * H + h) * kMarkDots;
    float behind = 0.f;
#pragma unroll
    for (int w = 0; w < kMarkDots; ++w) behind += end[w];
#pragma unroll
    for (int j = kTokens / 32 - 1; j >= 0; --j) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float down = __shfl_down_sync(0xffffffffu, v[j], d);
        if (lane + d < 32) v[j] += down;
      }
      // the first token decays nothing where no state comes in
      const size_t out = (t0 + 32 * j + lane) * H + h;
      const bool first = no_start && pc.s == 0 && g == 0 && 32 * j + lane == 0;
      if (32 * j + lane < cnt)
        dlog[out] = __float2bfloat16_rn(first || (resets >> j & 1) ? 0.f : v[j] + behind);
      behind += __shfl_sync(0xffffffffu, v[j], 0);
    }
  }
}

template <int WAY, int NT>
cudaError_t launch_t(const TcRun &P, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = prepare_kernel(run_tc_kernel<WAY, NT>, (int)kSmemBytes, ready);
  if (e != cudaSuccess) return e;
  run_tc_kernel<WAY, NT><<<(unsigned)run_blocks(P.r.cut, P.r.state_only), kThreads, kSmemBytes, s>>>(P);
  return cudaGetLastError();
}

bool fill(TcRun *P, const Run &r, int32_t *status, uint64_t hook_ns) {
  memset(P, 0, sizeof(*P));
  P->r = r;
  P->status = status;
  P->wait_ns = hook_ns ? hook_ns : kWaitNs;
  P->dbg_skip = hook_ns != 0;
  const int64_t T = r.cut.t_total;
  if (T == 0) return true;
  bool ok = make_row_tile_map(&P->tm_y, r.y, T, r.Hy, C) && make_row_tile_map(&P->tm_z, r.z, T, r.Hz, C);
  if (ok && !r.state_only) ok = make_row_tile_map(&P->tm_x, r.x, T, r.Hx, C);
  if (ok && !r.state_only && !r.out_f32) ok = make_row_tile_map(&P->tm_o, r.out, T, r.cut.H, 32);
  return ok;
}

}  // namespace

cudaError_t launch_run_tc(const Run &r, int terms, int32_t *status, cudaStream_t s) {
  uint64_t hook_ns = 0;
  if (!take_debug_timeout(GDN2_DEBUG_LINATTN, &hook_ns)) hook_ns = 0;
  TcRun P;
  if (!fill(&P, r, status, hook_ns)) return cudaErrorInvalidValue;
  if (r.back) return terms == 4 ? launch_t<1, 4>(P, s) : launch_t<1, 2>(P, s);
  return terms == 4 ? launch_t<0, 4>(P, s) : launch_t<0, 2>(P, s);
}

cudaError_t launch_grads_tc(const Run *r, int32_t *status, cudaStream_t s) {
  uint64_t hook_ns = 0;
  if (!take_debug_timeout(GDN2_DEBUG_LINATTN, &hook_ns)) hook_ns = 0;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = prepare_kernel(grads_tc_kernel, (int)kSmemBytes, ready);
  if (e != cudaSuccess) return e;
  TcGrads P;
  for (int i = 0; i < 3; ++i)
    if (!fill(&P.run[i], r[i], status, hook_ns)) return cudaErrorInvalidValue;
  grads_tc_kernel<<<(unsigned)(3 * run_blocks(r[0].cut, r[0].state_only)), kThreads, kSmemBytes, s>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_marks(const float *a, const float *b, float *mark_dots, const Cut &c, cudaStream_t s) {
  const int64_t groups = (int64_t)c.t_total / (kGroup * C) + 1;  // of the longest piece, at most
  const dim3 grid((unsigned)((int64_t)c.n_pieces * c.H), (unsigned)(groups < 32 ? groups : 32));
  marks_kernel<<<grid, 256, 0, s>>>(a, b, mark_dots, c);
  return cudaGetLastError();
}

cudaError_t launch_dlog_tc(const float *dots_q, const float *dots_k, const float *mark_dots, const void *log_a, const Cut &c,
                           bool no_start, void *dlog, cudaStream_t s) {
  if (c.t_total == 0) return cudaSuccess;
  const int64_t groups = (int64_t)c.t_total / (kGroup * C * kDlogWarps) + 1;  // of the longest piece, at most
  const dim3 grid((unsigned)((int64_t)c.n_pieces * c.H), (unsigned)(groups < 16 ? groups : 16));
  dlog_tc_kernel<<<grid, 32 * kDlogWarps, 0, s>>>(dots_q, dots_k, mark_dots, static_cast<const __nv_bfloat16 *>(log_a), c,
                                                  no_start, static_cast<__nv_bfloat16 *>(dlog));
  return cudaGetLastError();
}

}  // namespace lin
}  // namespace gdn2
