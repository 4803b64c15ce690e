// ckpt8.cu -- activations kept in 8 bits between a forward and its backward pass.
//
// Every row is cut into blocks of 32 values that share a scale 2^e, e the smallest integer
// (>= -127) with max|x| <= 127 * 2^e; a value is kept as code = rint(x / 2^e), half to even, and
// the scale as the byte e + 127.  Dividing by a power of two is exact, so the only rounding is the
// rint: at most 2^(e-1), under max|x| / 127.  A code has 7 bits and a sign, so code * 2^e is a bf16
// value exactly and the tensor cores can take restored operands without a second rounding.
// A block that holds an infinity or a NaN gets the byte 255 and restores as NaN.
#include "linattn.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Scale byte of a block from the largest |x| as fp32 bits (they order like the values; NaN last).
// |x| = 1.m 2^(E-127) <= 127 * 2^e = 1.984375 * 2^(e+6): e = E - 133 where m <= 0x7e0000, else one more.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  const int b = (int)(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)max(b, 0);
}
// 2^-e; codes above `lim` are cut back: 64 * 2^122 would restore as infinity.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - min(byte, 254u)) << 23); }
__device__ __forceinline__ int code_of(float x, float inv, uint32_t byte) {
  if (byte == 255u) return 0;
  const int lim = byte >= 249u ? 63 : 127;
  return max(-lim, min(lim, __float2int_rn(x * inv)));
}
// Four codes.  x / 2^e is exact and at most 127, so adding 1.5 * 2^23 leaves it, rounded half to even,
// in the low bits: one operation where a conversion and two clamps took the save past its memory time.
__device__ __forceinline__ uint32_t codes4(const float *f, float inv) {
  constexpr float kShift = 12582912.f;
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = __float_as_uint(fmaf(f[i], inv, kShift));
  return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
}
// 2^e; 255 gives +inf, and 0 * inf = NaN is what such a block restores to.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&f)[8]) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack_bf16x2(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&f)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// cols % 8 == 0: a thread holds 8 values (one 16-byte load in bf16) and 4 lanes a block.  The unit
// of work is a (row, block) pair of 4 lanes, so a row's last block may have fewer than 4 live lanes.
// FLAT: cols % 32 == 0, so the rows need not be told apart and the 64-bit divisions, which took
// longer than the memory, fall away (32768 x 2048 bf16: 51 us).  Other multiples of 8 divide once a unit (2040
// columns: 64 us); what is no multiple of 8 goes one value a thread (2047 columns: 257 us).
// Streaming bounds it: a thread takes kUnits units a thread block's span apart and asks for all of
// them before it uses the first, 16 KB (bf16) a thread block in flight.
constexpr int kUnits = 4;
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads) save8_kernel(const T *__restrict__ x, int8_t *__restrict__ codes,
                                                         uint8_t *__restrict__ scales, int64_t rows, int cols,
                                                         int blocks) {
  const int64_t total = rows * blocks;
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 4 * kUnits) + (threadIdx.x >> 2);
  const int sub = threadIdx.x & 3;
  float f[kUnits][8];
  int64_t from[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t at = first + u * (kThreads / 4);
    if constexpr (FLAT) {
      from[u] = at < total ? at * 32 + sub * 8 : -1;
    } else {
      const int64_t row = at / blocks;
      const int col = (int)(at - row * blocks) * 32 + sub * 8;
      from[u] = at < total && col < cols ? row * cols + col : -1;
    }
    if (from[u] >= 0) load8<T>(x + from[u], f[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    uint32_t top = 0;
    if (from[u] >= 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, abs_bits(f[u][i]));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (from[u] < 0) continue;
    const uint32_t byte = scale_byte(top);
    const float inv = inverse_scale(byte);
    uint32_t w[2] = {codes4(f[u], inv), codes4(f[u] + 4, inv)};
    if (byte >= 249u) {  // near the end of fp32's range, or an infinity or a NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if ((i & 3) == 0) w[i >> 2] = 0;
        w[i >> 2] |= ((uint32_t)code_of(f[u][i], inv, byte) & 255u) << (8 * (i & 3));
      }
    }
    *reinterpret_cast<uint2 *>(codes + from[u]) = make_uint2(w[0], w[1]);
    if (sub == 0) scales[first + u * (kThreads / 4)] = (uint8_t)byte;
  }
}

// Any cols: a warp per block, a lane per value.
template <typename T>
__global__ void __launch_bounds__(kThreads) save1_kernel(const T *__restrict__ x, int8_t *__restrict__ codes,
                                                         uint8_t *__restrict__ scales, int64_t rows, int cols,
                                                         int blocks) {
  const int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (at >= rows * blocks) return;
  const int lane = threadIdx.x & 31;
  const int64_t row = at / blocks;
  const int col = (int)(at - row * blocks) * 32 + lane;
  const bool live = col < cols;
  const float f = live ? to_f32<T>(x[row * cols + col]) : 0.f;
  const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(f)));
  if (live) codes[row * cols + col] = (int8_t)code_of(f, inverse_scale(byte), byte);
  if (lane == 0) scales[at] = (uint8_t)byte;
}

// cols % 8 == 0: a thread restores kUnits times 8 values, all asked for before the first is used.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads) restore8_kernel(const int8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, T *__restrict__ x,
                                                            int64_t rows, int cols, int blocks) {
  const int per_row = cols >> 3;
  const int64_t total = rows * per_row, first = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  uint2 code[kUnits];
  uint32_t byte[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t at = first + u * kThreads;
    if (at >= total) break;
    code[u] = __ldcs(reinterpret_cast<const uint2 *>(codes + at * 8));
    if constexpr (FLAT) {
      byte[u] = scales[at >> 2];
    } else {
      const int64_t row = at / per_row;
      byte[u] = scales[row * blocks + ((int)(at - row * per_row) >> 2)];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t at = first + u * kThreads;
    if (at >= total) break;
    const float s = scale_value(byte[u]);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)(int8_t)((i < 4 ? code[u].x : code[u].y) >> (8 * (i & 3))) * s;
    if constexpr (sizeof(T) == 2) {
      const uint4 o = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                 pack_bf16x2(f[6], f[7]));
      *reinterpret_cast<uint4 *>(x + at * 8) = o;
    } else {
      float4 *o = reinterpret_cast<float4 *>(x + at * 8);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) restore1_kernel(const int8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, T *__restrict__ x,
                                                            int64_t rows, int cols, int blocks) {
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (at >= rows * cols) return;
  const int64_t row = at / cols;
  const int c = (int)(at - row * cols);
  x[at] = from_f32<T>((float)codes[at] * scale_value(scales[row * blocks + (c >> 5)]));
}

template <typename T>
cudaError_t save_t(const T *x, int8_t *codes, uint8_t *scales, int64_t rows, int cols, cudaStream_t s) {
  const int blocks = (cols + 31) / 32;
  const int64_t units = rows * blocks;
  const unsigned grid = (unsigned)((units * 4 + kThreads * kUnits - 1) / (kThreads * kUnits));
  if (cols % 32 == 0)
    save8_kernel<T, true><<<grid, kThreads, 0, s>>>(x, codes, scales, rows, cols, blocks);
  else if (cols % 8 == 0)
    save8_kernel<T, false><<<grid, kThreads, 0, s>>>(x, codes, scales, rows, cols, blocks);
  else
    save1_kernel<T><<<(unsigned)((units * 32 + kThreads - 1) / kThreads), kThreads, 0, s>>>(x, codes, scales, rows,
                                                                                             cols, blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t restore_t(const int8_t *codes, const uint8_t *scales, T *x, int64_t rows, int cols, cudaStream_t s) {
  const int blocks = (cols + 31) / 32;
  const int64_t n = cols % 8 == 0 ? rows * cols / 8 : rows * cols;
  const int64_t each = cols % 8 == 0 ? kThreads * kUnits : kThreads;
  const unsigned grid = (unsigned)((n + each - 1) / each);
  if (cols % 32 == 0)
    restore8_kernel<T, true><<<grid, kThreads, 0, s>>>(codes, scales, x, rows, cols, blocks);
  else if (cols % 8 == 0)
    restore8_kernel<T, false><<<grid, kThreads, 0, s>>>(codes, scales, x, rows, cols, blocks);
  else
    restore1_kernel<T><<<grid, kThreads, 0, s>>>(codes, scales, x, rows, cols, blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt8_save(const void *x, int8_t *codes, uint8_t *scales, int64_t rows, int cols, int dtype,
                              cudaStream_t s) {
  return dtype == GDN2_BF16 ? save_t(static_cast<const __nv_bfloat16 *>(x), codes, scales, rows, cols, s)
                            : save_t(static_cast<const float *>(x), codes, scales, rows, cols, s);
}

cudaError_t launch_ckpt8_restore(const int8_t *codes, const uint8_t *scales, void *x, int64_t rows, int cols, int dtype,
                                 cudaStream_t s) {
  return dtype == GDN2_BF16 ? restore_t(codes, scales, static_cast<__nv_bfloat16 *>(x), rows, cols, s)
                            : restore_t(codes, scales, static_cast<float *>(x), rows, cols, s);
}

}  // namespace gdn2
