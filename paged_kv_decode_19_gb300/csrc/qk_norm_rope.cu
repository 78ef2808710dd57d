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
// row is read by D / 8 lanes and stays in registers; the mean needs log2(D / 8) shuffles.  The angles depend on the token alone, so a
// warp computes a token's rd / 2 cosines and sines once, in shared memory, for all the heads it
// takes; they cost about 40 instructions each, which a row's lanes would otherwise pay per value.
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
__device__ __forceinline__ void unpack8(const Vec8<XT>& r, float2 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(XT) == 4)
      x[i] = make_float2(__uint_as_float((&r.v[i >> 1].x)[2 * (i & 1)]), __uint_as_float((&r.v[i >> 1].x)[2 * (i & 1) + 1]));
    else
      x[i] = unpack2<XT>((&r.v[0].x)[i]);
  }
}
template <typename XT>
__device__ __forceinline__ Vec8<XT> pack8(const float2 (&x)[4]) {
  Vec8<XT> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(XT) == 4) {
      (&r.v[i >> 1].x)[2 * (i & 1)] = __float_as_uint(x[i].x);
      (&r.v[i >> 1].x)[2 * (i & 1) + 1] = __float_as_uint(x[i].y);
    } else {
      (&r.v[0].x)[i] = pack2<XT>(x[i].x, x[i].y);
    }
  }
  return r;
}

// Four floats of shared memory at `a` and four at `b` (16-byte aligned) as pairs.
__device__ __forceinline__ void load_pairs(const float* a, const float* b, float2 (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(a), y = *reinterpret_cast<const float4*>(b);
  v[0] = make_float2(x.x, x.y);
  v[1] = make_float2(x.z, x.w);
  v[2] = make_float2(y.x, y.y);
  v[3] = make_float2(y.z, y.w);
}

// Rows in vectors: D a multiple of 8 (at most 8 LPR), 16-byte aligned rows, a rotated part that
// is a multiple of 8.  MODE 0 no rotation, 1 rotate-half, 2 interleaved; a lane holds eight dims,
// both of every rotated pair (rotate-half: four of each half, as two 8-byte accesses of a 16-bit
// row; a 16-byte chunk and shuffles for the partner cost 1.5 us more for 8192 tokens of 40 heads of
// 128, bf16).  A pass is 32 / LPR heads of one token, all queries or all keys; a warp takes
// part `p` of the `parts` of a token's passes (grid stride over the T * parts tasks), GP passes
// at a time, the next GP loaded while these are computed.  No block barrier after the start:
// the warps drift apart, so that loads, products and stores of different tokens overlap (a block
// per token with a barrier for its angles took 48 us).  80 registers (three blocks an SM; rotate-half
// below D 256 spills 8 bytes).  33.2 us are 75 % of the copy rate; the same
// kernel takes 28.3 us without norm and rotation, 30.1 with the norm alone, 31.0 with the rotation.
//
// With x' the rotation partner of x, an output is rs (x A + x' B), A = w cos and B = -+ w' sin:
// A and B are the same for every query (key) head of a token, so a row costs two products per
// value, packed in pairs.
template <typename XT, int MODE, int LPR>
__global__ void __launch_bounds__(kQkThreads, 3)
    qk_norm_rope_kernel(const __grid_constant__ QkParams a) {
  constexpr int NW = kQkThreads / 32, RW = 32 / LPR;  // rows per pass
  constexpr int NV = (int)sizeof(XT) * 8 / 16, GP = sizeof(XT) == 4 ? 2 : 4;
  constexpr int NF = MODE ? 4 * LPR : 4;              // frequencies, at most
  __shared__ __align__(16) float s_w[2][8 * LPR];
  __shared__ unsigned long long s_F[NF];
  __shared__ __align__(16) float s_ang[NW][2][NF];    // a warp's token: cosines, sines
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % LPR, row = lane / LPR;
  const int nf = a.rd / 2, q_passes = (a.Hq + RW - 1) / RW, passes = q_passes + (a.Hk + RW - 1) / RW;
  for (int i = tid; i < 16 * LPR; i += kQkThreads) {
    const int k = i / (8 * LPR), d = i % (8 * LPR);
    const void* w = k ? a.k_weight : a.q_weight;
    s_w[k][d] = w && d < a.D ? weight_at(w, a.w_dtype, d) + a.w_offset : 1.f;
  }
  if (MODE && tid < nf) s_F[tid] = freq_turns(__ldg(a.freq + tid));
  __syncthreads();
  // This lane's dims: d .. d + 3 and d + apart .. + 3.  Rotate-half: pairs of the rotated part,
  // then of what passes; else eight in a row.
  int d = sub * 8, apart = 4;
  if (MODE == 1) {
    const int i = sub * 4;
    d = i < nf ? i : a.rd + i - nf;
    apart = i < nf ? nf : (a.D - a.rd) / 2;
  }
  const bool live = sub * 8 < a.D, turns = MODE && d < a.rd;
  const int f0 = MODE == 1 ? d : d / 2;  // this lane's first frequency
  const long long tasks = (long long)a.T * a.parts;
  for (long long task = (long long)blockIdx.x * NW + warp; task < tasks; task += (long long)gridDim.x * NW) {
    const int t = (int)(task / a.parts), part = (int)(task - (long long)t * a.parts);
    const int p0 = part * passes / a.parts, p1 = (part + 1) * passes / a.parts;
    bool have_angles = MODE == 0;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {  // the queries' passes of the part, then the keys'
      const int s0 = k ? max(p0 - q_passes, 0) : min(p0, q_passes);
      int n = (k ? max(p1 - q_passes, 0) : min(p1, q_passes)) - s0;
      if (n <= 0) continue;
      // (a pass's step fits 32 bits with room for GP of them: checked by the launch)
      const int head = (int)(k ? a.k_head : a.q_head), head_to = (int)(k ? a.k_out_head : a.q_out_head);
      const int step = RW * head, step_to = RW * head_to;
      const XT* src = reinterpret_cast<const XT*>(k ? a.k : a.q) + (k ? t * a.k_stride : t * a.q_stride) +
                      (long long)(row + s0 * RW) * head + d;
      XT* dst = reinterpret_cast<XT*>(k ? a.k_out : a.q_out) + (k ? t * a.k_out_stride : t * a.q_out_stride) +
                (long long)(row + s0 * RW) * head_to + d;
      // passes with a head for this lane: all but perhaps the side's last
      int mine = live ? min(n, ((k ? a.Hk : a.Hq) - row + RW - 1) / RW - s0) : 0;
      const bool normed = k ? a.k_weight != nullptr : a.q_weight != nullptr;
      auto load = [&](Vec8<XT> (&raw)[GP]) {  // the next GP passes
#pragma unroll
        for (int u = 0; u < GP; ++u)
          if (u < mine) {
            if constexpr (MODE == 1 && NV == 1) {
              const uint2 x = *reinterpret_cast<const uint2*>(src + u * step);
              const uint2 y = *reinterpret_cast<const uint2*>(src + u * step + apart);
              raw[u].v[0] = make_uint4(x.x, x.y, y.x, y.y);
            } else {
#pragma unroll
              for (int i = 0; i < NV; ++i) raw[u].v[i] = *reinterpret_cast<const uint4*>(src + u * step + i * apart);
            }
          }
        src += GP * step;
      };
      Vec8<XT> cur[GP], nxt[GP];
#pragma unroll
      for (int u = 0; u < GP; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i) cur[u].v[i] = nxt[u].v[i] = make_uint4(0u, 0u, 0u, 0u);
      load(cur);
      if constexpr (MODE != 0) {
        if (!have_angles) {
          have_angles = true;
          const int pos = __ldg(a.positions + t);
          __syncwarp();  // the last token's angles have been read
#pragma unroll
          for (int i = 0; i < NF; i += 32) {
            if (i + lane < nf) {
              float co, si;
              rope_cos_sin_accurate(pos, s_F[i + lane], co, si);
              s_ang[warp][0][i + lane] = co * a.attention_factor;
              s_ang[warp][1][i + lane] = si * a.attention_factor;
            }
          }
          __syncwarp();
        }
      }
      float2 A[4], B[4];
      load_pairs(&s_w[k][d], &s_w[k][live ? d + apart : d], A);
      if constexpr (MODE != 0) {
        float2 co[4], si[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) co[i] = make_float2(1.f, 1.f), si[i] = make_float2(0.f, 0.f);
        if (turns) {
          const float4 x = *reinterpret_cast<const float4*>(&s_ang[warp][0][f0]);
          const float4 y = *reinterpret_cast<const float4*>(&s_ang[warp][1][f0]);
          if constexpr (MODE == 1) {
            co[0] = co[2] = make_float2(x.x, x.y), co[1] = co[3] = make_float2(x.z, x.w);
            si[2] = make_float2(y.x, y.y), si[3] = make_float2(y.z, y.w);
            si[0] = make_float2(-y.x, -y.y), si[1] = make_float2(-y.z, -y.w);
          } else {
            co[0] = make_float2(x.x, x.x), co[1] = make_float2(x.y, x.y);
            co[2] = make_float2(x.z, x.z), co[3] = make_float2(x.w, x.w);
            si[0] = make_float2(-y.x, y.x), si[1] = make_float2(-y.y, y.y);
            si[2] = make_float2(-y.z, y.z), si[3] = make_float2(-y.w, y.w);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          B[i] = mul_f2(MODE == 1 ? A[i ^ 2] : make_float2(A[i].y, A[i].x), si[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] = mul_f2(A[i], co[i]);
      }
      // the passes of `cur`, of which the lane stores the first `now`; the full group has no branch, so
      // that its passes' shuffles and products interleave (36.7 -> 33.2 us)
      auto group = [&](int now, auto full) {
#pragma unroll
        for (int u = 0; u < GP; ++u) {
          if (!decltype(full)::value && u >= n) break;  // (warp-uniform)
          float2 x[4], y[4];
          unpack8<XT>(cur[u], x);
          float rs = 1.f;
          if (normed) {
            float2 ss = mul_f2(x[0], x[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) ss = fma_f2(x[i], x[i], ss);
            float sum = ss.x + ss.y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            rs = rsqrtf(sum * a.inv_D + a.eps);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 z = mul_f2(x[i], A[i]);
            if (MODE && turns) z = fma_f2(MODE == 1 ? x[i ^ 2] : make_float2(x[i].y, x[i].x), B[i], z);
            y[i] = mul_f2(z, make_float2(rs, rs));
          }
          if (u < now) {
            const Vec8<XT> o = pack8<XT>(y);
            if constexpr (MODE == 1 && NV == 1) {
              *reinterpret_cast<uint2*>(dst + u * step_to) = make_uint2(o.v[0].x, o.v[0].y);
              *reinterpret_cast<uint2*>(dst + u * step_to + apart) = make_uint2(o.v[0].z, o.v[0].w);
            } else {
#pragma unroll
              for (int i = 0; i < NV; ++i) *reinterpret_cast<uint4*>(dst + u * step_to + i * apart) = o.v[i];
            }
          }
        }
      };
#pragma unroll 1
      for (; n >= GP; n -= GP) {
        const int now = mine;
        mine -= GP;
        load(nxt);  // (none left: nothing)
        group(now, std::true_type{});
        dst += GP * step_to;
#pragma unroll
        for (int u = 0; u < GP; ++u) cur[u] = nxt[u];
      }
      if (n > 0) group(mine, std::false_type{});
    }
  }
}

// Any head dim up to kQkMaxD, any alignment and strides: a warp per row, the normalised row
// in shared memory between the norm and the rotation.  Element by element, so bound by its requests:
// 8192 tokens of 40 heads of 100, bf16, 283 us (7 % of the copy rate), one token 4.2 us.
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
static cudaError_t launch_vec(QkParams a, int num_sms, cudaStream_t st) {
  constexpr int NW = kQkThreads / 32, RW = 32 / LPR;
  const int passes = (a.Hq + RW - 1) / RW + (a.Hk + RW - 1) / RW;
  // A token's angles and coefficients are worth sharing among its heads while there are warps
  // enough (about 16 a multiprocessor); with fewer tokens the heads are spread over more warps.
  const long long want = 16ll * num_sms;
  a.parts = (int)min((long long)passes, max(1ll, (want + a.T - 1) / a.T));
  const long long tasks = (long long)a.T * a.parts;
  const dim3 grid((unsigned)min((tasks + NW - 1) / NW, 4ll * num_sms));
  return launch_pdl(qk_norm_rope_kernel<XT, MODE, LPR>, grid, dim3(kQkThreads), 0, st, a);
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
  bool near = true;  // heads near enough for 32-bit steps
  for (int i = 4; i < 8; ++i) near = near && strides[i] < (1ll << 26) && strides[i] > -(1ll << 26);
  const bool vec = near && any % 16 == 0 && a.D % 8 == 0 && a.D <= 256 && a.rd % 8 == 0;
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
