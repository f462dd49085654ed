// Conversions to and from MXFP4 (OCP MX: blocks of 32 E2M1 values with one E8M0 scale).
//
// A block's scale is 2^(floor(log2 max) - 2): the exponent field of the largest magnitude,
// less 2, is the scale byte itself (subnormal maxima clamp to byte 0 = 2^-127), and the
// division is an exact multiplication by a power of two.  So the only rounding is the
// hardware's conversion to E2M1 (nearest even, saturating at 6).  Bound by memory: one read
// and one write of everything.  32768 x 2880 in bf16, both ways: 74 us = 6.4 TB/s (of a copy's
// 6.8; quantising alone, back to back, 34 us = 6.9 TB/s, from fp32 60 us = 7.1; with maxima taken
// one value at a time 42 in bf16).
#include <cstdint>

#include "experts_args.h"
#include "ptx.cuh"

namespace sa {
namespace {

// 8 floats -> 8 E2M1 codes, value i in bits [4 i, 4 i + 4).
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 8 E2M1 codes -> four pairs of f16 values.
__device__ __forceinline__ void unpack_e2m1x8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

__device__ __forceinline__ float half_bits_to_float(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.f32.f16 %0, t;\n\t}" : "=f"(f) : "r"(h & 0xFFFFu));
  return f;
}

constexpr int kThreads = 256;
// Pieces in flight per thread, and resident blocks per SM that the grids count on.  Two pieces of
// fp32 beside five blocks do not fit into the registers (spilled: 68 us for 32768 x 2880, one: 60).
template <bool kFp32>
constexpr int kQuantUnroll = kFp32 ? 1 : 2;
constexpr int kQuantBlocks = 5;
constexpr int kUnroll = 4;
constexpr int kDequantBlocks = 8;

// Two lanes share a block of 32 (16 values each: 32 bytes of bf16 in, 8 bytes of codes out).
// A row's pieces are even in number and so is the grid's step: blocks stay in their pairs.
template <bool kFp32>
__global__ void __launch_bounds__(kThreads, kQuantBlocks) mxfp4_quantize_kernel(const Mxfp4Args a) {
  constexpr int kUnroll = kQuantUnroll<kFp32>;
  constexpr int kLoads = kFp32 ? 4 : 2;  // of 16 bytes per piece
  const int pieces = a.k / 16;
  const long long total = a.rows * pieces;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  const long long step_row = step / pieces;
  const int step_col = static_cast<int>(step - step_row * pieces);
  long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  GridWalk at(i, pieces);
  // every lane of a warp makes the same number of rounds (the pairs exchange their maxima)
  for (long long base = i - threadIdx.x % 32; base < total; base += kUnroll * step) {
    uint4 p[kUnroll][kLoads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const long long j = i + u * step;
        p[u][l] = make_uint4(0, 0, 0, 0);
        if (j < total) p[u][l] = __ldcs(reinterpret_cast<const uint4*>(a.in) + kLoads * j + l);
      }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u, i += step, at.advance(step_row, step_col, pieces)) {
      float v[2][8];
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const uint32_t w[4] = {p[u][l].x, p[u][l].y, p[u][l].z, p[u][l].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (kFp32) {
            v[l >> 1][4 * (l & 1) + j] = __uint_as_float(w[j]);
          } else {
            v[l][2 * j] = __uint_as_float(w[j] << 16);
            v[l][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        }
      }
      uint32_t mx = 0;  // bits of the largest magnitude
      if constexpr (kFp32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) mx = max(mx, __float_as_uint(v[j >> 3][j & 7]) & 0x7FFFFFFFu);
      } else {  // two bf16 values at a time: their order is that of their bits
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          const uint32_t w[4] = {p[u][l].x, p[u][l].y, p[u][l].z, p[u][l].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = __vmaxu2(mx, w[j] & 0x7FFF7FFFu);
        }
        mx = max(mx << 16, mx & 0xFFFF0000u);
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      const uint32_t field = mx >> 23;
      const bool finite = field < 255u;
      const uint32_t byte = finite ? (field > 2u ? field - 2u : 0u) : 255u;
      const float inv = __uint_as_float((254u - (finite ? byte : 0u)) << 23);  // 2^(127 - byte)
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j >> 3][j & 7] *= inv;
      if (!finite) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j >> 3][j & 7] = 0.0f;
      }
      if (i < total) {
        reinterpret_cast<uint2*>(a.codes)[i] = make_uint2(pack_e2m1x8(v[0]), pack_e2m1x8(v[1]));
        if ((threadIdx.x & 1) == 0) {
          const int b = at.col / 2;
          uint8_t* s = a.scales + at.row * a.stride;
          s[b] = static_cast<uint8_t>(byte);
          if (b == a.k / 32 - 1)
            for (int c = b + 1; c < a.stride; ++c) s[c] = 0;  // padding
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, kDequantBlocks) mxfp4_dequantize_kernel(const Mxfp4Args a) {
  const int vecs = a.k / 8;
  const long long total = a.rows * vecs;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  const long long step_row = step / vecs;
  const int step_vec = static_cast<int>(step - step_row * vecs);
  long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  GridWalk at(i, vecs);
  while (i < total) {
    uint32_t codes[kUnroll], byte[kUnroll];
    GridWalk ahead = at;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u, ahead.advance(step_row, step_vec, vecs)) {
      codes[u] = byte[u] = 0;
      if (i + u * step < total) {
        codes[u] = __ldcs(reinterpret_cast<const uint32_t*>(a.in) + i + u * step);
        byte[u] = __ldg(a.scales + ahead.row * a.stride + ahead.col / 4);
      }
    }
    at = ahead;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u, i += step) {
      if (i >= total) break;
      // 2^(byte - 127): byte 0 is a subnormal fp32 number, byte 255 NaN
      const uint32_t bits = byte[u] == 255u ? 0x7FC00000u : byte[u] == 0u ? 0x00400000u : byte[u] << 23;
      const float scale = __uint_as_float(bits);
      uint32_t h[4], o[4];
      unpack_e2m1x8(codes[u], h);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(half_bits_to_float(h[j]) * scale, half_bits_to_float(h[j] >> 16) * scale);
      __stcs(reinterpret_cast<uint4*>(a.out) + i, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

// A grid that fills the device once, or less for small sizes; `values` per thread and step.
int blocks_for(const Mxfp4Args& a, int values, int per_sm, int sms) {
  const long long blocks = (a.rows * (a.k / values) + kThreads - 1) / kThreads, most = static_cast<long long>(per_sm) * sms;
  return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const Mxfp4Args& a, int sms, cudaStream_t stream) {
  const int grid = blocks_for(a, 16, kQuantBlocks, sms);
  if (a.is_fp32) mxfp4_quantize_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else mxfp4_quantize_kernel<false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const Mxfp4Args& a, int sms, cudaStream_t stream) {
  mxfp4_dequantize_kernel<<<blocks_for(a, 8, kDequantBlocks, sms), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
