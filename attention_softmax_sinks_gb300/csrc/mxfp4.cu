// Conversions to and from MXFP4 (OCP MX: blocks of 32 E2M1 values with one E8M0 scale).
//
// A block's scale is 2^(floor(log2 max) - 2): the exponent field of the largest magnitude,
// less 2, is the scale byte itself (subnormal maxima clamp to byte 0 = 2^-127), and the
// division is an exact multiplication by a power of two.  So the only rounding is the
// hardware's conversion to E2M1 (nearest even, saturating at 6).  Bound by memory: one read
// and one write of everything.
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

// Four lanes share a block of 32 (8 values each: 16 bytes of bf16 in, 4 bytes of codes out).
template <bool kFp32>
__global__ void __launch_bounds__(256) mxfp4_quantize_kernel(const Mxfp4Args a) {
  const int vecs = a.k / 8;  // a multiple of 4: a block's lanes are in one quad
  const long long total = a.rows * vecs;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i0 = static_cast<long long>(blockIdx.x) * blockDim.x; i0 < total; i0 += step) {
    const long long i = i0 + threadIdx.x;
    const bool in = i < total;
    float v[8];
    uint32_t mx = 0;
    if constexpr (kFp32) {
      float4 p = make_float4(0, 0, 0, 0), q = p;
      if (in) {
        p = __ldcs(reinterpret_cast<const float4*>(a.in) + 2 * i);
        q = __ldcs(reinterpret_cast<const float4*>(a.in) + 2 * i + 1);
      }
      v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
    } else {
      uint4 p = make_uint4(0, 0, 0, 0);
      if (in) p = __ldcs(reinterpret_cast<const uint4*>(a.in) + i);
      const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const uint32_t field = mx >> 23;
    const bool finite = field < 255u;
    const uint32_t byte = finite ? (field > 2u ? field - 2u : 0u) : 255u;
    const float inv = __uint_as_float((254u - (finite ? byte : 0u)) << 23);  // 2^(127 - byte)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = finite ? v[j] * inv : 0.0f;
    if (in) {
      reinterpret_cast<uint32_t*>(a.codes)[i] = pack_e2m1x8(v);
      if ((threadIdx.x & 3) == 0) {
        const long long row = i / vecs;
        const int b = static_cast<int>(i - row * vecs) / 4;
        uint8_t* s = a.scales + row * a.stride;
        s[b] = static_cast<uint8_t>(byte);
        if (b == a.k / 32 - 1)
          for (int p = b + 1; p < a.stride; ++p) s[p] = 0;  // padding
      }
    }
  }
}

__global__ void __launch_bounds__(256) mxfp4_dequantize_kernel(const Mxfp4Args a) {
  const int vecs = a.k / 8;
  const long long total = a.rows * vecs;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const long long row = i / vecs;
    const int b = static_cast<int>(i - row * vecs) / 4;
    const uint32_t codes = __ldcs(reinterpret_cast<const uint32_t*>(a.in) + i);
    const uint32_t byte = __ldg(a.scales + row * a.stride + b);
    // 2^(byte - 127): byte 0 is a subnormal fp32 number, byte 255 NaN
    const float scale = __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
    uint32_t h[4], o[4];
    unpack_e2m1x8(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack_bf16x2(half_bits_to_float(h[j]) * scale, half_bits_to_float(h[j] >> 16) * scale);
    reinterpret_cast<uint4*>(a.out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

int blocks_for(const Mxfp4Args& a, int sms) {
  const long long blocks = (a.rows * (a.k / 8) + 255) / 256, most = 32LL * sms;
  return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const Mxfp4Args& a, int sms, cudaStream_t stream) {
  const int grid = blocks_for(a, sms);
  if (a.is_fp32) mxfp4_quantize_kernel<true><<<grid, 256, 0, stream>>>(a);
  else mxfp4_quantize_kernel<false><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const Mxfp4Args& a, int sms, cudaStream_t stream) {
  mxfp4_dequantize_kernel<<<blocks_for(a, sms), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
