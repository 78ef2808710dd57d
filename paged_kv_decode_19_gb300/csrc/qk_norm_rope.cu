// qk_norm_rope: per-head RMS norm of the query and key heads and the position rotation, in
// one pass over the rows of a projection's output.
//
// For token t and head h, x = the head's D values:
//   y_d = x_d / sqrt(mean(x^2) + eps) * (w_d + w_offset)      (no weights: y = x)
//   for i < rd / 2, (a, b) = (y_i, y_{i + rd/2}) or (y_{2i}, y_{2i+1}):
//     (a, b) <- (a cos - b sin, b cos + a sin) * attention_factor,  angle = position[t] f_i
//   dims rd .. D - 1 pass through; one rounding at the end.
// The frequencies are fp64 radians per position.  A block turns each into a 64-bit fraction
// of a revolution once, F = 2^64 frac(f / 2 pi); position * F mod 2^64 is then the angle
// reduced exactly, so a far position loses nothing (rope_cos_sin_accurate).
//
// Bound by the bytes, 2 x row, for many tokens and by launch and load latency for few.  A
// row is read by D / 8 lanes in 16-byte chunks (one for 16-bit types) and stays in
// registers: the mean needs log2(D / 8) shuffles and the rotate-half partner is a shuffle of
// the normalised values.  The angles depend on the token alone, so a block computes a token's
// rd / 2 cosines and sines once, in shared memory, for all its heads; they cost about 40
// instructions each, which one row a lane would otherwise pay eight times over.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace pd {

constexpr int kQkThreads = 256;
constexpr int kQkMaxD = 512;  // head dim of the general kernel

__device__ __forceinline__ float weight_at(const void* w, int dtype, int d) {
  if (dtype == kF32) return __ldg(reinterpret_cast<const float*>(w) + d);
  const unsigned short b = __ldg(reinterpret_cast<const unsigned short*>(w) + d);
  return dtype == kBF16 ? __uint_as_float((unsigned)b << 16) : __half2float(__ushort_as_half(b));
}

// 2^64 frac(f / 2 pi), with 1 / 2 pi in two fp64 parts: the rounding of one alone, 2^-53 of the
// turns, would reach the angle of a high frequency at a far position.
__device__ __forceinline__ unsigned long long freq_turns(double f) {
  const double c1 = 0.15915494309189535, c2 = -9.839338337591243e-18;
  const double hi = f * c1, lo = fma(f, c1, -hi) + f * c2;
  return (unsigned long long)((hi - floor(hi)) * 18446744073709551616.0) +
         (unsigned long long)(long long)(lo * 18446744073709551616.0);
}

// 8 consecutive elements of a row (16-byte aligned) as floats, and back.
template <typename XT>
struct Vec8 {
  uint4 v[sizeof(XT) * 8 / 16];
};
template <typename XT>
__device__ __forceinline__ void unpack8(const Vec8<XT>& r, float (&x)[8]) {
  if constexpr (sizeof(XT) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((&r.v[i >> 2].x)[i & 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<XT>((&r.v[0].x)[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename XT>
__device__ __forceinline__ Vec8<XT> pack8(const float (&x)[8]) {
  Vec8<XT> r;
  if constexpr (sizeof(XT) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) (&r.v[i >> 2].x)[i & 3] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) (&r.v[0].x)[i] = pack2<XT>(x[2 * i], x[2 * i + 1]);
  }
  return r;
}

// Rows in 16-byte chunks: D a multiple of 8 (at most 8 LPR), 16-byte aligned rows, a rotated
// part that ends on a chunk (rotate-half: each half does).  MODE 0 no rotation, 1 rotate-half,
// 2 interleaved.  blockIdx.y: which RU * 256 / LPR heads of the token; tokens by grid stride.
template <typename XT, int MODE, int LPR, int RU>
__global__ void __launch_bounds__(kQkThreads)
    qk_norm_rope_kernel(const __grid_constant__ QkParams a) {
  constexpr int RG = kQkThreads / LPR;  // rows per pass of the block
  __shared__ __align__(16) float s_w[2][8 * LPR];
  __shared__ __align__(16) float s_cos[2][MODE ? 4 * LPR : 4], s_sin[2][MODE ? 4 * LPR : 4];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, sub = tid % LPR, row0 = blockIdx.y * (RG * RU) + tid / LPR;
  const int H = a.Hq + a.Hk, nf = a.rd / 2;
  for (int i = tid; i < 2 * a.D; i += kQkThreads) {
    const int k = i >= a.D, d = i - k * a.D;
    const void* w = k ? a.k_weight : a.q_weight;
    if (w) s_w[k][d] = weight_at(w, a.w_dtype, d) + a.w_offset;
  }
  unsigned long long F = 0;
  if (MODE && tid < nf) F = freq_turns(__ldg(a.freq + tid));
  const int c = sub * 8;             // this lane's dims
  const bool live = c < a.D, turns = MODE && c < a.rd;
  // rotate-half: this lane's chunk and its partner's, half a rotated part away
  const bool first_half = c < nf;
  const int partner = (tid & 31) + (first_half ? nf / 8 : -(nf / 8));
  const int f0 = MODE == 1 ? (first_half ? c : c - nf) : c / 2;
  for (int t = blockIdx.x, buf = 0; t < a.T; t += gridDim.x, buf ^= 1) {
    Vec8<XT> raw[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int r = row0 + u * RG;
#pragma unroll
      for (int i = 0; i < (int)(sizeof(XT) * 8 / 16); ++i) raw[u].v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < H && live) {
        const bool k = r >= a.Hq;
        const XT* src = reinterpret_cast<const XT*>(k ? a.k : a.q) +
                        (k ? t * a.k_stride + (r - a.Hq) * a.k_head : t * a.q_stride + r * a.q_head) + c;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(XT) * 8 / 16); ++i)
          raw[u].v[i] = *(reinterpret_cast<const uint4*>(src) + i);
      }
    }
    if (MODE && tid < nf) {
      float co, si;
      rope_cos_sin_accurate(__ldg(a.positions + t), F, co, si);
      s_cos[buf][tid] = co * a.attention_factor;
      s_sin[buf][tid] = si * a.attention_factor;
    }
    __syncthreads();  // (two buffers: one barrier per token)
    float co[8], si[8];  // MODE 2 uses the first four
#pragma unroll
    for (int i = 0; i < 8; ++i) co[i] = si[i] = 0.f;
    if (turns) {
#pragma unroll
      for (int i = 0; i < (MODE == 1 ? 8 : 4); i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&s_cos[buf][f0 + i]);
        const float4 y = *reinterpret_cast<const float4*>(&s_sin[buf][f0 + i]);
        co[i] = x.x; co[i + 1] = x.y; co[i + 2] = x.z; co[i + 3] = x.w;
        si[i] = y.x; si[i + 1] = y.y; si[i + 2] = y.z; si[i + 3] = y.w;
      }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int r = row0 + u * RG;
      const bool k = r >= a.Hq;
      float x[8];
      unpack8<XT>(raw[u], x);
      if (a.q_weight || a.k_weight) {  // (the shuffles take the whole warp)
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (k ? a.k_weight != nullptr : a.q_weight != nullptr) {
          const float rs = rsqrtf(ss * a.inv_D + a.eps);
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 w = *reinterpret_cast<const float4*>(&s_w[k][c + i]);
            x[i] *= rs * w.x;
            x[i + 1] *= rs * w.y;
            x[i + 2] *= rs * w.z;
            x[i + 3] *= rs * w.w;
          }
        }
      }
      if constexpr (MODE == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_sync(0xffffffffu, x[i], partner & 31);
          if (turns) x[i] = x[i] * co[i] + (first_half ? -other : other) * si[i];
        }
      } else if constexpr (MODE == 2) {
        if (turns) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = p * co[i] - q * si[i];
            x[2 * i + 1] = q * co[i] + p * si[i];
          }
        }
      }
      if (r < H && live) {
        XT* dst = reinterpret_cast<XT*>(k ? a.k_out : a.q_out) +
                  (k ? t * a.k_out_stride + (r - a.Hq) * a.k_out_head : t * a.q_out_stride + r * a.q_out_head) + c;
        const Vec8<XT> o = pack8<XT>(x);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(XT) * 8 / 16); ++i) *(reinterpret_cast<uint4*>(dst) + i) = o.v[i];
      }
    }
  }
}

// Any head dim up to kQkMaxD, any alignment and strides: a warp per row, the normalised row
// in shared memory between the norm and the rotation.
template <typename XT>
__global__ void __launch_bounds__(kQkThreads)
    qk_norm_rope_any_kernel(const __grid_constant__ QkParams a) {
  constexpr int NW = kQkThreads / 32, kPer = kQkMaxD / 32;
  __shared__ float s_row[NW][kQkMaxD];
  __shared__ float s_cos[kQkMaxD / 2], s_sin[kQkMaxD / 2];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.Hq + a.Hk, nf = a.rd / 2, D = a.D;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int i = tid; i < nf; i += kQkThreads) {
      float co, si;
      rope_cos_sin_accurate(__ldg(a.positions + t), freq_turns(__ldg(a.freq + i)), co, si);
      s_cos[i] = co * a.attention_factor;
      s_sin[i] = si * a.attention_factor;
    }
    __syncthreads();
    for (int r = blockIdx.y * NW + warp; r < H; r += gridDim.y * NW) {
      const bool k = r >= a.Hq;
      const int h = k ? r - a.Hq : r;
      const XT* src = reinterpret_cast<const XT*>(k ? a.k : a.q) +
                      (k ? t * a.k_stride + h * a.k_head : t * a.q_stride + h * a.q_head);
      XT* dst = reinterpret_cast<XT*>(k ? a.k_out : a.q_out) +
                (k ? t * a.k_out_stride + h * a.k_out_head : t * a.q_out_stride + h * a.q_out_head);
      const void* w = k ? a.k_weight : a.q_weight;
      float x[kPer], ss = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int d = lane + 32 * i;
        x[i] = d < D ? to_f32(src[d]) : 0.f;
        ss = fmaf(x[i], x[i], ss);
      }
      const float rs = w ? rsqrtf(warp_sum(ss) * a.inv_D + a.eps) : 1.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int d = lane + 32 * i;
        if (d < D) s_row[warp][d] = w ? x[i] * (rs * (weight_at(w, a.w_dtype, d) + a.w_offset)) : x[i];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int d = lane + 32 * i;
        if (d >= D) continue;
        float y = s_row[warp][d];
        if (d < a.rd) {
          const bool half = a.mode == 1;
          const int f = half ? (d < nf ? d : d - nf) : d >> 1;
          const bool lead = half ? d < nf : (d & 1) == 0;
          const float o = s_row[warp][half ? (d < nf ? d + nf : d - nf) : d ^ 1];
          y = y * s_cos[f] + (lead ? -o : o) * s_sin[f];
        }
        dst[d] = from_f32<XT>(y);
      }
      __syncwarp();  // the row is rewritten by the next
    }
    __syncthreads();  // the angles are rewritten by the next token
  }
}

// ------------------------------------------------------------------------- dispatch
template <typename XT, int MODE, int LPR>
static cudaError_t launch_vec(const QkParams& a, int num_sms, cudaStream_t st) {
  constexpr int RG = kQkThreads / LPR;
  const int H = a.Hq + a.Hk;
  // Few tokens: one pass of rows per block, so that every row is in flight at once.  Many:
  // up to four passes per block share a token's angles and barrier.
  const int passes = (H + RG - 1) / RG;
  if ((long long)a.T * passes <= 8ll * num_sms || passes == 1) {
    const dim3 grid((unsigned)min((long long)a.T, 8ll * num_sms), (unsigned)passes);
    return launch_pdl(qk_norm_rope_kernel<XT, MODE, LPR, 1>, grid, dim3(kQkThreads), 0, st, a);
  }
  const int per = passes <= 2 ? 2 : passes == 3 ? 3 : 4;
  const dim3 grid((unsigned)min((long long)a.T, 8ll * num_sms), (unsigned)((passes + per - 1) / per));
  if (per == 2) return launch_pdl(qk_norm_rope_kernel<XT, MODE, LPR, 2>, grid, dim3(kQkThreads), 0, st, a);
  if (per == 3) return launch_pdl(qk_norm_rope_kernel<XT, MODE, LPR, 3>, grid, dim3(kQkThreads), 0, st, a);
  return launch_pdl(qk_norm_rope_kernel<XT, MODE, LPR, 4>, grid, dim3(kQkThreads), 0, st, a);
}

template <typename XT, int MODE>
static cudaError_t launch_mode(const QkParams& a, int num_sms, cudaStream_t st) {
  if (a.D <= 64) return launch_vec<XT, MODE, 8>(a, num_sms, st);
  if (a.D <= 128) return launch_vec<XT, MODE, 16>(a, num_sms, st);
  return launch_vec<XT, MODE, 32>(a, num_sms, st);
}

template <typename XT>
static cudaError_t launch_x(const QkParams& a, int num_sms, cudaStream_t st) {
  const int mode = a.rd ? a.mode : 0;
  constexpr int eb = (int)sizeof(XT);
  uintptr_t any = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                  reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out);
  const long long strides[8] = {a.q_stride, a.k_stride, a.q_out_stride, a.k_out_stride,
                                a.q_head, a.k_head, a.q_out_head, a.k_out_head};
  for (long long s : strides) any |= (uintptr_t)(s * eb);
  const bool vec = any % 16 == 0 && a.D % 8 == 0 && a.D <= 256 && a.rd % (mode == 1 ? 16 : 8) == 0;
  if (vec) {
    if (mode == 1) return launch_mode<XT, 1>(a, num_sms, st);
    if (mode == 2) return launch_mode<XT, 2>(a, num_sms, st);
    return launch_mode<XT, 0>(a, num_sms, st);
  }
  const int H = a.Hq + a.Hk, passes = (H + kQkThreads / 32 - 1) / (kQkThreads / 32);
  const int gx = (int)min((long long)a.T, 8ll * num_sms);
  const int gy = max(1, min(passes, 8 * num_sms / gx));
  return launch_pdl(qk_norm_rope_any_kernel<XT>, dim3((unsigned)gx, (unsigned)gy), dim3(kQkThreads), 0, st, a);
}

cudaError_t launch_qk_norm_rope(const QkParams& a, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == kBF16) return launch_x<__nv_bfloat16>(a, num_sms, st);
  if (dtype == kF16) return launch_x<__half>(a, num_sms, st);
  if (dtype == kF32) return launch_x<float>(a, num_sms, st);
  return cudaErrorInvalidValue;
}

}  // namespace pd
