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
// Bound by the bytes (2 D elements in, D (1 + 2 / block) bytes out per token and head) and by the 200
// instructions of a warp's 32 items: rows need nothing but their own values, so a thread takes 16 dims,
// which share a scale (two threads of 32), and the stores alone wait for the token's slot.  Measured on
// one GB300: 8192 tokens of 8 heads of 128 from bf16 9.9 us (64 % of the copy rate on 43 MB; with IEEE
// divisions 16.7, with one item a thread instead of a grid-sized loop and one correction of a product
// 11.4, with shorter addresses 10.0), 256 tokens 1.43 us, 1777 of 4 heads of 64, a third of them skipped,
// 2.0 us (launches).
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace pd {

namespace {
constexpr int kThreads = 128;  // (256 threads: 1.56 and 10.1 us where 128 take 1.43 and 9.9)

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

// y / s, correctly rounded, for an s of at most four significant bits and r = 1 / s rounded: Markstein's
// correction of a product by the remainder, which the fma gives exactly.  (The remainder is taken
// negative, so that a zero keeps its sign.)
__device__ __forceinline__ float quotient(float y, float s, float r) {
  const float q = y * r;
  return fmaf(fmaf(q, s, -y), -r, q);
}
// The larger of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_abs(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
  return r;
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

// n / d for n < 2^31 by a multiplication.
struct Divisor {
  unsigned mul, shift, d;
  explicit Divisor(unsigned by) : d(by) {
    for (shift = 0; shift < 32 && (1ull << shift) < by; ++shift) {}
    mul = (unsigned)(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
  }
  __device__ __forceinline__ unsigned quot(unsigned n) const { return (__umulhi(n, mul) + n) >> shift; }
};

template <typename IT, int SB, bool VEC>
__global__ void __launch_bounds__(kThreads)
    append_mx_kernel(const __grid_constant__ AppendMxParams a, const __grid_constant__ Divisor per_row,
                     const __grid_constant__ Divisor per_page, int log_d) {
  pdl_wait();  // inputs and pages are the previous kernel's to write until it completes
  pdl_release();
  // an item is 16 dims of a token's K or V: item = (token, K | V, head, 16 dims); SB 32: a block's two
  // are side by side, in one warp
  const unsigned items = 2u * a.T * per_row.d, i0 = blockIdx.x * kThreads + threadIdx.x;
  const unsigned i = min(i0, items - 1);
  const unsigned row = per_row.quot(i), j = i - row * per_row.d;
  const int t = row >> 1, kv = row & 1;
  long long slot = __ldg(a.slots + t);
  float y[16];
  load16<IT, VEC>(reinterpret_cast<const IT*>(kv ? a.v_new : a.k_new) + t * (kv ? a.v_stride : a.k_stride) + 16 * j, y);
  const float g = kv ? a.v_scale : a.k_scale;
  if (g != 1.f) {
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = __fdiv_rn(y[e], g);
  }
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = max_abs(m, y[e]);
  if constexpr (SB == 32) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const bool finite = m <= FLT_MAX;
  float s, r;
  uint8_t sb;
  if constexpr (SB == 16) {
    const uint8_t c = f32_to_e4m3(quotient(m, 6.f, 1.f / 6.f));
    sb = finite ? max(c, (uint8_t)1) : (uint8_t)0x7f;  // (code 1: 2^-9)
    F8 f;
    f.v = sb;
    s = to_f32(f);
    r = __frcp_rn(s);
  } else {
    // 6 = 1.5 * 2^2: two below the exponent, one more where the significand is above 1.5
    const unsigned b = __float_as_uint(m);
    const int k = (int)(b >> 23) - 2 + ((b & 0x7fffffu) > 0x400000u ? 1 : 0);
    sb = finite ? (uint8_t)min(max(k, 127 - 14), 127 + 13) : (uint8_t)0xff;
    s = 0.f;
    r = __uint_as_float((254u - sb) << 23);  // 2^-k: the product is the quotient
  }
  uint2 codes = make_uint2(0u, 0u);
  if (finite) {
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = SB == 16 ? quotient(y[e], s, r) : y[e] * r;
    codes = make_uint2(encode8(y), encode8(y + 8));
  }
  if (i != i0 || slot < 0) return;
  if (slot >= a.n_slots) {
    set_error(a.err, kErrBadSlot);
    return;
  }
  const unsigned h = 16 * j >> log_d, d = 16 * j - (h << log_d);
  const unsigned page = slot >> 31 ? (unsigned)(slot / a.P) : per_page.quot((unsigned)slot);
  // the row in the cache (2 max_pages H_kv is below 2^31)
  const long long at = (long long)((page * 2 + kv) * a.H_kv + h) * a.P + (int)(slot - (long long)page * a.P);
  *reinterpret_cast<uint2*>(a.pages + (at << (log_d - 1)) + d / 2) = codes;
  if (SB == 16 || (d & 16) == 0) a.scales[((at << log_d) + d) / SB] = sb;
}

template <typename IT, int SB>
static cudaError_t launch_t(const AppendMxParams& all, int D, bool vec, cudaStream_t st) {
  const Divisor per_row((unsigned)(all.H_kv * (D / 16))), per_page((unsigned)all.P);
  const int log_d = D == 64 ? 6 : D == 128 ? 7 : 8;
  // as many tokens a launch as keep the items below 2^31
  const int most = (int)std::max(1ll, (1ll << 30) / (2ll * per_row.d));
  for (int t0 = 0; t0 < all.T; t0 += most) {
    AppendMxParams a = all;
    a.T = std::min(most, all.T - t0);
    a.slots += t0;
    a.k_new = reinterpret_cast<const IT*>(a.k_new) + t0 * a.k_stride;
    a.v_new = reinterpret_cast<const IT*>(a.v_new) + t0 * a.v_stride;
    const dim3 grid((unsigned)((2ll * a.T * per_row.d + kThreads - 1) / kThreads));
    const cudaError_t e = vec ? launch_pdl(append_mx_kernel<IT, SB, true>, grid, dim3(kThreads), 0, st, a, per_row, per_page, log_d)
                              : launch_pdl(append_mx_kernel<IT, SB, false>, grid, dim3(kThreads), 0, st, a, per_row, per_page, log_d);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename IT>
static cudaError_t launch_i(const AppendMxParams& a, int D, int sb, bool vec, cudaStream_t st) {
  return sb == 16 ? launch_t<IT, 16>(a, D, vec, st) : launch_t<IT, 32>(a, D, vec, st);
}

cudaError_t launch_append_mx(const AppendMxParams& a, int D, int sb, int in_dtype, cudaStream_t st) {
  const int eb = in_dtype == kF32 ? 4 : 2;
  // 16-byte loads where the tensors allow them, element loads else
  const bool vec = ((reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new)) & 15) == 0 &&
                   a.k_stride * eb % 16 == 0 && a.v_stride * eb % 16 == 0;
  if (in_dtype == kF32) return launch_i<float>(a, D, sb, vec, st);
  if (in_dtype == kF16) return launch_i<__half>(a, D, sb, vec, st);
  if (in_dtype == kBF16) return launch_i<__nv_bfloat16>(a, D, sb, vec, st);
  return cudaErrorInvalidValue;
}

}  // namespace pd
