// append_paged_kv_bs: new tokens' K/V into an 8-bit cache with one fp32 scale per (page,
// K | V, KV head, block of S rows).
//
// For a block that receives new rows x, with amax = max |x| over the block's new rows and
// all D dims of the head:
//   need = the smallest power of two 2^k, k >= -126, with amax <= M 2^k  (M = 448 e4m3, 127 int8)
//   scale' = need                     if the block holds no row of the sequence yet
//          = max(scale, need)         otherwise; its old codes c become RN(c scale / scale')
//   code = RN(x / scale')
// A power of two makes x / scale' and the ratio of two such scales exact: an e4m3 code that
// is recoded loses nothing until it is subnormal, an int8 code only the bits shifted out, and
// the result does not depend on how a sequence was cut into appends for e4m3 normals.  A
// caller's own scale (any finite positive fp32) is kept until it has to grow; x is then divided.
// A non-finite new value makes the block's scale NaN and its new codes 0: every output that
// attends the block is then NaN, until the block is refilled from its first row.
//
// Bound by the bytes (2 x row in, D bytes out) for prefill chunks and by the chain of dependent
// loads (sequence search, table, rows) for one token per sequence.  One warp per (touched block,
// K | V, head): the rows of a block are in registers when they fit (kKeep steps of 32 / (D / 8)
// rows), so each is read once; the maximum is taken on the integer patterns (magnitude bits order
// like the values, and a non-finite one shows as the largest).  Measured on one GB300: 9713 tokens
// of 8 heads of 128 in five sequences 13.1 us (67 % of the copy rate on 60 MB, inputs from HBM;
// 14.4 with three blocks of eight warps an SM instead of eight of four; the 64 registers that eight
// blocks leave spill 8 to 24 bytes a thread with vector loads, up to 68 with element loads), 256
// sequences of one token 6.4 us, of which the loads one after the other are most; from fp32 22.2 and
// 6.0 us, heads of 256 24.4.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace pd {

template <typename T> struct Bits16;  // pattern of +inf of a 16-bit type
template <> struct Bits16<__nv_bfloat16> { static constexpr unsigned inf = 0x7f80u; };
template <> struct Bits16<__half> { static constexpr unsigned inf = 0x7c00u; };

// 8 consecutive elements of a row, as loaded
template <typename IT>
struct Row8 {
  static constexpr int NW = (int)sizeof(IT) * 2;  // 32-bit words
  uint32_t w[NW];
};

template <typename IT, bool VEC>
__device__ __forceinline__ Row8<IT> load_row8(const IT* src) {
  Row8<IT> r;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < Row8<IT>::NW / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (sizeof(IT) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(__ldg(reinterpret_cast<const float*>(src) + i));
  } else {
    const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = (uint32_t)__ldg(s + 2 * i) | ((uint32_t)__ldg(s + 2 * i + 1) << 16);
  }
  return r;
}

template <typename IT>
__device__ __forceinline__ void row8_f32(const Row8<IT>& r, float (&x)[8]) {
  if constexpr (sizeof(IT) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<IT>(r.w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Running maximum of the magnitude patterns (two 16-bit lanes, or one 32-bit).
template <typename IT>
__device__ __forceinline__ unsigned max_bits(const Row8<IT>& r, unsigned m) {
#pragma unroll
  for (int i = 0; i < Row8<IT>::NW; ++i)
    m = sizeof(IT) == 4 ? max(m, r.w[i] & 0x7fffffffu) : __vmaxu2(m, r.w[i] & 0x7fff7fffu);
  return m;
}

// The smallest power of two 2^k, k >= -126, with amax <= M 2^k, M = 1.75 * 2^8 (e4m3) or
// 1.984375 * 2^6 (int8): from amax's exponent, and one more where its mantissa is above M's.
template <typename CT>
__device__ __forceinline__ float pow2_scale(float amax) {
  constexpr bool kE4 = std::is_same<CT, F8>::value;
  const unsigned b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - (kE4 ? 8 : 6) + ((b & 0x7fffffu) > (kE4 ? 0x600000u : 0x7e0000u) ? 1 : 0);
  return __uint_as_float((unsigned)max(e, 1) << 23);
}

// 8 values already divided by the scale -> 8 codes.  int8: adding 1.5 * 2^23 rounds to
// nearest even and leaves the integer in the low byte (|x| <= 127 by the choice of scale).
template <typename CT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8]) {
  uint2 r;
  if constexpr (std::is_same<CT, F8>::value) {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    r.x = (uint32_t)h[0] | ((uint32_t)h[1] << 16);
    r.y = (uint32_t)h[2] | ((uint32_t)h[3] << 16);
  } else {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(x[i] + 12582912.f);
    r.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    r.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  }
  return r;
}

template <typename CT>
__device__ __forceinline__ void decode8(uint2 c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? c.x : c.y;
    const uint8_t b = (uint8_t)(w >> (8 * (i & 3)));
    if constexpr (std::is_same<CT, F8>::value) {
      F8 f;
      f.v = b;
      x[i] = to_f32(f);
    } else {
      x[i] = (float)(int8_t)b;
    }
  }
}

// Slots: sequence b owns slots [append_indptr[b] / S + 2 b, append_indptr[b+1] / S + 2 b + 2),
// at least as many as the blocks its new rows touch (n rows touch at most (n - 2) / S + 2);
// blockIdx.x is the slot, a warp takes one (head, K | V) of its block.
template <typename IT, typename CT, int D, bool VEC>
__global__ void __launch_bounds__(kAppendWarps * 32, 8)
    append_bs_kernel(const __grid_constant__ AppendBsParams a) {
  constexpr int LPR = D / 8;                  // lanes per row
  constexpr int RPS = 32 / LPR;               // rows per step of the warp
  constexpr int kKeep = sizeof(IT) == 4 ? 4 : 8;  // steps of rows kept in registers
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
  pdl_wait();  // inputs, pages and scales are the previous kernel's to write until it completes
  pdl_release();
  if (item >= 2 * a.H_kv) return;
  const int kv = item / a.H_kv, h = item - kv * a.H_kv;
  const int S = a.S, P = a.P;

  // The last sequence b with append_indptr[b] / S + 2 b <= slot.  A lane takes one candidate and
  // loads all of its sequence's numbers at once, so that the search costs one round trip when b
  // is among the 32 around the place that even sequences give (always, up to 32 sequences);
  // else 32 candidates a round narrow the range first.
  const int slot = blockIdx.x;
  int c_a0 = 0, c_a1 = 0, c_i0 = 0, c_i1 = 0, c_last = 0;
  auto among = [&](int base) -> int {  // how many of candidates base .. base + 31 start at or before slot
    const int c = base + lane;
    bool le = false;
    if (c < a.B) {
      c_a0 = a.append_indptr[c];
      c_a1 = a.append_indptr[c + 1];
      c_i0 = a.indptr[c];
      c_i1 = a.indptr[c + 1];
      c_last = a.length_info[c];
      le = c_a0 / S + 2 * c <= slot;
    }
    return __popc(__ballot_sync(0xffffffffu, le));
  };
  int base = max(0, min((int)((long long)slot * a.B / gridDim.x) - 16, a.B - 32));
  int cnt = among(base);
  if ((cnt == 0 && base > 0) || (cnt == 32 && base + 32 < a.B)) {
    base = 0;
    for (int n = a.B; n > 32;) {
      const int step = (n + 31) / 32;
      const int c = base + lane * step;
      const bool le = lane * step < n && a.append_indptr[c] / S + 2 * c <= slot;
      const int k = max(__popc(__ballot_sync(0xffffffffu, le)), 1) - 1;
      base += k * step;
      n = min(step, n - k * step);
    }
    cnt = among(base);
  }
  const int win = min(max(cnt, 1) - 1, a.B - 1 - base), b = base + win;
  const int a0 = __shfl_sync(0xffffffffu, c_a0, win), a1 = __shfl_sync(0xffffffffu, c_a1, win);
  const int i0 = __shfl_sync(0xffffffffu, c_i0, win), i1 = __shfl_sync(0xffffffffu, c_i1, win);
  const int last = __shfl_sync(0xffffffffu, c_last, win);
  const int n_new = a1 - a0;
  const long long L = i1 > i0 ? (long long)(i1 - i0 - 1) * P + last : 0;
  if (a0 < 0 || n_new < 0 || a1 > a.T || i0 < 0 || i1 < i0 || i1 > a.nnz || n_new > L || last > P || last < 0 ||
      L > INT_MAX - 256) {
    if (lane == 0) set_error(a.err, kErrBadLength);
    return;
  }
  if (n_new == 0) return;
  const int first = (int)L - n_new;  // offset of the sequence's first new row
  const int blk = first / S + (slot - (a0 / S + 2 * b));
  if (blk < first / S || blk > ((int)L - 1) / S) return;
  const int o0 = max(blk * S, first), o1 = min(blk * S + S, (int)L);
  const int pidx = blk * S / P;
  const int page = a.values[i0 + pidx];
  if (page < 0 || page >= a.max_pages) {
    if (lane == 0) set_error(a.err, kErrBadPage);
    return;
  }
  const size_t kvblk = ((size_t)page * 2 + kv) * a.H_kv + h;
  const int in_page = blk * S - pidx * P;  // the block's first row in its page
  float* const scale_at = a.scales + kvblk * (P / S) + in_page / S;
  uint8_t* const rows = a.pages + (kvblk * P + in_page) * D;
  const IT* const src = reinterpret_cast<const IT*>(kv ? a.v_new : a.k_new) +
                        (long long)(a0 + o0 - first) * (kv ? a.v_stride : a.k_stride) + h * D;
  const long long stride = kv ? a.v_stride : a.k_stride;
  const int n_old = o0 - blk * S, n = o1 - o0;
  const float old_scale = n_old ? *scale_at : 0.f;
  const int sub = lane / LPR, c8 = (lane % LPR) * 8;

  Row8<IT> keep[kKeep];
  unsigned m = 0;
  for (int r0 = 0; r0 < n; r0 += kKeep * RPS) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int r = r0 + i * RPS + sub;
      if (r < n) {
        keep[i] = load_row8<IT, VEC>(src + r * stride + c8);
      } else {
#pragma unroll
        for (int k = 0; k < Row8<IT>::NW; ++k) keep[i].w[k] = 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) m = max_bits<IT>(keep[i], m);
  }
  float amax;
  bool finite;
  if constexpr (sizeof(IT) == 4) {
    m = __reduce_max_sync(0xffffffffu, m);
    amax = __uint_as_float(m);
    finite = m < 0x7f800000u;
  } else {
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    amax = unpack2<IT>(m).x;
    finite = m < Bits16<IT>::inf;
  }
  float scale = finite ? pow2_scale<CT>(amax) : __uint_as_float(0x7fc00000u);
  if (n_old) {
    if (!(old_scale == old_scale)) scale = old_scale;  // stays NaN
    else if (finite) scale = fmaxf(old_scale, scale);
    if (scale != old_scale && scale == scale) {  // grown: the block's old codes change units
      const float ratio = old_scale / scale;
      for (int r = sub; r < n_old; r += RPS) {
        uint2* at = reinterpret_cast<uint2*>(rows + (size_t)r * D + c8);
        float x[8];
        decode8<CT>(*at, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], ratio);  // (not fused into the encoding)
        *at = encode8<CT>(x);
      }
    }
  }
  const bool ok = scale == scale;
  const unsigned sb = __float_as_uint(scale);
  const bool pow2 = (sb & 0x807fffffu) == 0u && sb != 0u && sb < 0x7f000000u;  // (warp-uniform)
  const float inv = pow2 ? __uint_as_float(0x7f000000u - sb) : 0.f;           // 2^-k, exact
  uint8_t* const to = rows + (size_t)n_old * D + c8;
  for (int r0 = 0; r0 < n; r0 += kKeep * RPS) {
    if (n > kKeep * RPS) {  // the rows did not all stay in registers
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int r = r0 + i * RPS + sub;
        if (r < n) keep[i] = load_row8<IT, VEC>(src + r * stride + c8);
      }
    }
    if (pow2) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int r = r0 + i * RPS + sub;
        float x[8];
        row8_f32<IT>(keep[i], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= inv;
        if (r < n) *reinterpret_cast<uint2*>(to + (size_t)r * D) = encode8<CT>(x);
      }
    } else {  // a caller's scale that is no power of two, or NaN (codes 0)
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int r = r0 + i * RPS + sub;
        float x[8];
        row8_f32<IT>(keep[i], x);
        if (r < n) {
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            uint32_t one = 0;
            if (ok) {
              const float q[8] = {__fdiv_rn(x[0], scale), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              one = encode8<CT>(q).x;
            }
            to[(size_t)r * D + k] = (uint8_t)one;
#pragma unroll
            for (int e = 0; e < 7; ++e) x[e] = x[e + 1];
          }
        }
      }
    }
  }
  if (lane == 0) *scale_at = scale;
}

template <typename IT, typename CT, int D>
static cudaError_t launch_d(const AppendBsParams& a, bool vec, cudaStream_t st) {
  const dim3 grid((unsigned)(a.T / a.S + 2 * a.B), (unsigned)append_bs_grid_y(a.H_kv));
  const dim3 block(kAppendWarps * 32);
  return vec ? launch_pdl(append_bs_kernel<IT, CT, D, true>, grid, block, 0, st, a)
             : launch_pdl(append_bs_kernel<IT, CT, D, false>, grid, block, 0, st, a);
}

template <typename IT, typename CT>
static cudaError_t launch_c(const AppendBsParams& a, int D, bool vec, cudaStream_t st) {
  switch (D) {
    case 64: return launch_d<IT, CT, 64>(a, vec, st);
    case 128: return launch_d<IT, CT, 128>(a, vec, st);
    case 256: return launch_d<IT, CT, 256>(a, vec, st);
  }
  return cudaErrorInvalidValue;
}

template <typename IT>
static cudaError_t launch_i(const AppendBsParams& a, int D, int kv_dtype, bool vec, cudaStream_t st) {
  return kv_dtype == kE4M3 ? launch_c<IT, F8>(a, D, vec, st) : launch_c<IT, I8>(a, D, vec, st);
}

cudaError_t launch_append_bs(const AppendBsParams& a, int D, int in_dtype, int kv_dtype, cudaStream_t st) {
  const int eb = in_dtype == kF32 ? 4 : 2;
  // 16-byte row loads where the tensors allow them, element loads else (eight times the requests)
  const bool vec = ((reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new)) & 15) == 0 &&
                   a.k_stride * eb % 16 == 0 && a.v_stride * eb % 16 == 0;
  if (in_dtype == kF32) return launch_i<float>(a, D, kv_dtype, vec, st);
  if (in_dtype == kF16) return launch_i<__half>(a, D, kv_dtype, vec, st);
  if (in_dtype == kBF16) return launch_i<__nv_bfloat16>(a, D, kv_dtype, vec, st);
  return cudaErrorInvalidValue;
}

}  // namespace pd
