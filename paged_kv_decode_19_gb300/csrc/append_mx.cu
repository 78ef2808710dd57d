// append_paged_kv_mx: new tokens' K/V into a 4-bit cache: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a
// sign), two dims a byte, with a scale per row and block of 16 dims (e4m3) or 32 (a power of two).
//
// A row's value x stands as  code * s * g  (g = k_scale or v_scale of the call); with y = x / g and a =
// max |y| over the block:
//   e4m3: s = min(max(RN_e4m3(a / 6), 2^-9), 448)
//   e8m0: s = the smallest power of two 2^k with a <= 6 2^k, k in [-14, 13]
//   code = RN_e2m1(y / s), ties to even, saturating at 6
// A block that holds a non-finite value gets the scale NaN and codes 0.
// The quotients' roundings never move a value onto a border between codes: y and the borders times s
// have at most 24 and 7 significant bits, so a y that is off a border is off it by more than half a
// step of the quotient (and a / 6 likewise of e4m3's borders).
//
// Bound by the bytes (2 D elements in, D (1 + 2 / block) bytes out per token and head): rows need
// nothing but their own values, so a thread takes 16 dims, which share a scale (two threads of 32),
// and the stores alone wait for the token's slot.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace pd {

namespace {
constexpr int kThreads = 256;

// 16 consecutive elements as fp32
template <typename IT, bool VEC>
__device__ __forceinline__ void load16(const IT* src, float (&x)[16]) {
  if constexpr (VEC && sizeof(IT) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src) + i);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<IT>(w[k]);
        x[8 * i + 2 * k] = f.x;
        x[8 * i + 2 * k + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = to_f32(src[i]);
  }
}

// Eight values already divided by their scale -> eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t encode8(const float* q) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}
}  // namespace

template <typename IT, int SB, bool VEC>
__global__ void __launch_bounds__(kThreads) append_mx_kernel(const __grid_constant__ AppendMxParams a, int D) {
  const int per_row = a.H_kv * (D / 16);  // threads of a token's K (or V)
  const long long items = 2ll * a.T * per_row;
  pdl_wait();  // inputs and pages are the previous kernel's to write until it completes
  pdl_release();
  // a warp's 32 items (SB 32: a block's two are side by side, as per_row is even) in step
  for (long long i0 = (long long)blockIdx.x * kThreads + (threadIdx.x & ~31u); i0 < items;
       i0 += (long long)gridDim.x * kThreads) {
    const long long i = min(i0 + (threadIdx.x & 31), items - 1);
    const int row = (int)(i / per_row), j = (int)(i - (long long)row * per_row);
    const int t = row >> 1, kv = row & 1;
    long long slot = __ldg(a.slots + t);
    float y[16];
    load16<IT, VEC>(reinterpret_cast<const IT*>(kv ? a.v_new : a.k_new) + t * (kv ? a.v_stride : a.k_stride) + 16 * j, y);
    const float g = kv ? a.v_scale : a.k_scale;
    if (g != 1.f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __fdiv_rn(y[e], g);
    }
    unsigned m = 0;  // magnitude patterns order like the values, and a non-finite one shows as the largest
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(y[e]) & 0x7fffffffu);
    if constexpr (SB == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const bool finite = m < 0x7f800000u;
    float s;
    uint8_t sb;
    if constexpr (SB == 16) {
      const uint8_t c = f32_to_e4m3(__fdiv_rn(__uint_as_float(m), 6.f));
      sb = finite ? max(c, (uint8_t)1) : (uint8_t)0x7f;  // (code 1: 2^-9)
      F8 f;
      f.v = sb;
      s = to_f32(f);
    } else {
      // 6 = 1.5 * 2^2: two below the exponent, one more where the significand is above 1.5
      const int k = (int)(m >> 23) - 2 + ((m & 0x7fffffu) > 0x400000u ? 1 : 0);
      sb = finite ? (uint8_t)min(max(k, 127 - 14), 127 + 13) : (uint8_t)0xff;
      s = __uint_as_float((254u - sb) << 23);  // the inverse 2^-k, exact
    }
    uint2 codes = make_uint2(0u, 0u);
    if (finite) {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = SB == 16 ? __fdiv_rn(y[e], s) : y[e] * s;
      codes = make_uint2(encode8(y), encode8(y + 8));
    }
    if (slot >= a.n_slots) {
      set_error(a.err, kErrBadSlot);
      slot = -1;
    }
    if (slot >= 0 && i == i0 + (threadIdx.x & 31)) {
      const long long page = slot / a.P;
      const int h = 16 * j / D, d = 16 * j - h * D;
      const long long at = ((page * 2 + kv) * a.H_kv + h) * a.P + (slot - page * a.P);  // the row in the cache
      *reinterpret_cast<uint2*>(a.pages + at * (D / 2) + d / 2) = codes;
      if (SB == 16 || (d & 16) == 0) a.scales[at * (D / SB) + d / SB] = sb;
    }
  }
}

template <typename IT, int SB>
static cudaError_t launch_t(const AppendMxParams& a, int D, bool vec, int num_sms, cudaStream_t st) {
  const long long items = 2ll * a.T * a.H_kv * (D / 16);
  const dim3 grid((unsigned)std::min<long long>((items + kThreads - 1) / kThreads, (long long)num_sms * 32));
  return vec ? launch_pdl(append_mx_kernel<IT, SB, true>, grid, dim3(kThreads), 0, st, a, D)
             : launch_pdl(append_mx_kernel<IT, SB, false>, grid, dim3(kThreads), 0, st, a, D);
}

template <typename IT>
static cudaError_t launch_i(const AppendMxParams& a, int D, int sb, bool vec, int num_sms, cudaStream_t st) {
  return sb == 16 ? launch_t<IT, 16>(a, D, vec, num_sms, st) : launch_t<IT, 32>(a, D, vec, num_sms, st);
}

cudaError_t launch_append_mx(const AppendMxParams& a, int D, int sb, int in_dtype, int num_sms, cudaStream_t st) {
  const int eb = in_dtype == kF32 ? 4 : 2;
  // 16-byte loads where the tensors allow them, element loads else
  const bool vec = ((reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new)) & 15) == 0 &&
                   a.k_stride * eb % 16 == 0 && a.v_stride * eb % 16 == 0;
  if (in_dtype == kF32) return launch_i<float>(a, D, sb, vec, num_sms, st);
  if (in_dtype == kF16) return launch_i<__half>(a, D, sb, vec, num_sms, st);
  if (in_dtype == kBF16) return launch_i<__nv_bfloat16>(a, D, sb, vec, num_sms, st);
  return cudaErrorInvalidValue;
}

}  // namespace pd
