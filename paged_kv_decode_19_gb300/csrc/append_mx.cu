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
// Bound by the bytes (2 D elements in, D (1 + 2 / block) bytes out per token and head), by the loads
// under way and by the instructions: rows need nothing but their own values, so a thread takes 16 dims, which share
// a scale (two threads of 32), of a token's K and of its V, with one slot and one address for both, and the
// stores alone wait for the slot.  Quotients are corrected products: without a cache scale there is no division;
// with one a thread divides its largest magnitude, of K and of V, and every value only if the scale is outside
// 2^-60 .. 2^60 or that quotient is 2^120 or more, or NaN.  Measured on one GB300: 8192 tokens of 8 heads of 128 from bf16 8.4 us (75 % of the copy rate
// on 43 MB; with IEEE divisions 16.7, with K and V on threads of their own 9.8), with power-of-two scales
// 7.9, from fp32 13.0 (87 %; K and V apart 12.4), under a cache scale of 0.37 10.4 (with divisions by it
// 13.8); 256 tokens 1.5 us, 1777 of 4 heads of 64, a third of them skipped, 1.8 us (launches).
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace pd {

namespace {
constexpr int kThreads = 128;  // (64 threads: 8.8 us where 128 take 8.4, with power-of-two scales 8.8 and 7.9; 256: 8.5 and 7.9)

// The larger of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_abs(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
  return r;
}
// The same of two pairs; the signs of the result mean nothing.
template <typename IT>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same_v<IT, __half>) asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 consecutive elements as they are
template <typename IT>
struct Raw {
  uint32_t w[16 * sizeof(IT) / 4];
};
template <typename IT, bool VEC>
__device__ __forceinline__ Raw<IT> load16(const IT* src) {
  constexpr int N = 16 * sizeof(IT) / 4;
  Raw<IT> x;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
      x.w[4 * i] = v.x;
      x.w[4 * i + 1] = v.y;
      x.w[4 * i + 2] = v.z;
      x.w[4 * i + 3] = v.w;
    }
  } else if constexpr (sizeof(IT) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) x.w[i] = __float_as_uint(__ldg(src + i));
  } else {
    const uint16_t* at = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
    for (int i = 0; i < N; ++i) x.w[i] = __ldg(at + 2 * i) | (uint32_t)__ldg(at + 2 * i + 1) << 16;
  }
  return x;
}
// ... as fp32; returns their largest magnitude, NaN if one is.
template <typename IT>
__device__ __forceinline__ float unpack16(Raw<IT> r, float (&x)[16]) {
  if constexpr (sizeof(IT) == 4) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = __uint_as_float(r.w[i]);
      m = max_abs(m, x[i]);
    }
    return m;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<IT>(r.w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
#pragma unroll
    for (int n = 4; n > 0; n >>= 1) {
#pragma unroll
      for (int i = 0; i < n; ++i) r.w[i] = max_abs2<IT>(r.w[i], r.w[i + n]);
    }
    const float2 f = unpack2<IT>(r.w[0]);
    return max_abs(max_abs(0.f, f.x), f.y);
  }
}

// y / s, correctly rounded, for r = 1 / s rounded: Markstein's correction of a product by its remainder,
// which the fma gives exactly.  One correction is enough for an s of at most four significant bits; for
// any s the first may start 1.5 steps off, and the second makes it exact.  (The remainder is taken
// negative, so that a zero keeps its sign.)  No product may overflow.
__device__ __forceinline__ float corrected(float q, float y, float s, float r) {
  return fmaf(fmaf(q, s, -y), -r, q);
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

// 16 dims of a row with the cache's scale g (recip: 1 / g, or 0) -> their codes, and the block's scale.
template <typename IT, int SB>
__device__ __forceinline__ uint2 quantise16(const Raw<IT>& raw, float g, float recip, uint8_t& sb) {
  float y[16];
  float m = unpack16<IT>(raw, y);
  if (g != 1.f) {
    m = __fdiv_rn(m, g);  // (the largest quotient is the largest value's)
    if (recip != 0.f && m < 0x1p120f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = corrected(corrected(y[e] * recip, y[e], g, recip), y[e], g, recip);
    } else {  // products that could overflow
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __fdiv_rn(y[e], g);
    }
  }
  if constexpr (SB == 32) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const bool finite = m <= FLT_MAX;
  float r, rest = 0.f;
  if constexpr (SB == 16) {
    const uint8_t c = f32_to_e4m3(corrected(m * (1.f / 6.f), m, 6.f, 1.f / 6.f));
    sb = finite ? max(c, (uint8_t)1) : (uint8_t)0x7f;  // (code 1: 2^-9)
    F8 f;
    f.v = sb;
    const float s = to_f32(f);
    r = __frcp_rn(s);
    // 1 / s in two parts, the first short of it (12 bits: no s that is not a power of two has a
    // reciprocal that ends there) and the second 24 bits of the rest.  y r + y r_rest, off by 2^-36 of
    // the quotient before it is rounded, rounds as the quotient wherever a code's border is in question
    // (y and a border times s have at most 24 and 7 bits, so the quotient is that border, or off it by
    // 2^-28 more than half a step); both parts are positive, so that a zero keeps its sign.
    const float all = r;
    r = __uint_as_float(__float_as_uint(r) & ~0xfffu);
    rest = fmaf(-s, r, 1.f) * all;
  } else {
    // 6 = 1.5 * 2^2: two below the exponent, one more where the significand is above 1.5
    const unsigned b = __float_as_uint(m);
    const int k = (int)(b >> 23) - 2 + ((b & 0x7fffffu) > 0x400000u ? 1 : 0);
    sb = finite ? (uint8_t)min(max(k, 127 - 14), 127 + 13) : (uint8_t)0xff;
    r = __uint_as_float((254u - sb) << 23);  // 2^-k: the product is the quotient
  }
  uint2 codes = make_uint2(0u, 0u);
  if (finite) {
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = SB == 16 ? fmaf(y[e], r, y[e] * rest) : y[e] * r;
    codes = make_uint2(encode8(y), encode8(y + 8));
  }
  return codes;
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
  // an item is 16 dims of a token's K and V: item = (token, head, 16 dims); SB 32: a block's two are
  // side by side, in one warp
  const unsigned items = (unsigned)a.T * per_row.d, i0 = blockIdx.x * kThreads + threadIdx.x;
  const unsigned i = min(i0, items - 1);
  const unsigned t = per_row.quot(i), j = i - t * per_row.d;
  const long long slot = __ldg(a.slots + t);
  const Raw<IT> k = load16<IT, VEC>(reinterpret_cast<const IT*>(a.k_new) + t * a.k_stride + 16 * j);
  const Raw<IT> v = load16<IT, VEC>(reinterpret_cast<const IT*>(a.v_new) + t * a.v_stride + 16 * j);
  uint8_t ks, vs;
  const uint2 kc = quantise16<IT, SB>(k, a.k_scale, a.k_recip, ks);
  const uint2 vc = quantise16<IT, SB>(v, a.v_scale, a.v_recip, vs);
  if (i != i0 || slot < 0) return;
  if (slot >= a.n_slots) {
    set_error(a.err, kErrBadSlot);
    return;
  }
  const unsigned h = 16 * j >> log_d, d = 16 * j - (h << log_d);
  const unsigned page = slot >> 31 ? (unsigned)(slot / a.P) : per_page.quot((unsigned)slot);
  // the row in the cache (2 max_pages H_kv is below 2^31)
  const long long at = (long long)(page * 2 * a.H_kv + h) * a.P + (int)(slot - (long long)page * a.P);
  const long long of_v = (long long)a.H_kv * a.P;  // rows from K's to V's
  uint8_t* const codes = a.pages + (at << (log_d - 1)) + d / 2;
  *reinterpret_cast<uint2*>(codes) = kc;
  *reinterpret_cast<uint2*>(codes + (of_v << (log_d - 1))) = vc;
  if (SB == 16 || (d & 16) == 0) {
    uint8_t* const scales = a.scales + ((at << log_d) + d) / SB;
    scales[0] = ks;
    scales[(of_v << log_d) / SB] = vs;
  }
}

template <typename IT, int SB>
static cudaError_t launch_t(const AppendMxParams& all, int D, bool vec, cudaStream_t st) {
  const Divisor per_row((unsigned)(all.H_kv * (D / 16))), per_page((unsigned)all.P);
  const int log_d = D == 64 ? 6 : D == 128 ? 7 : 8;
  // as many tokens a launch as keep the items below 2^31
  const int most = (int)std::max(1ll, (1ll << 30) / per_row.d);
  for (int t0 = 0; t0 < all.T; t0 += most) {
    AppendMxParams a = all;
    a.T = std::min(most, all.T - t0);
    a.slots += t0;
    a.k_new = reinterpret_cast<const IT*>(a.k_new) + t0 * a.k_stride;
    a.v_new = reinterpret_cast<const IT*>(a.v_new) + t0 * a.v_stride;
    const dim3 grid((unsigned)(((long long)a.T * per_row.d + kThreads - 1) / kThreads));
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
