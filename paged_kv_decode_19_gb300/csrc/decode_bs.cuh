// Tensor-core decode of an 8-bit KV cache with one fp32 scale per (page, K | V, KV head,
// block of S rows), S a multiple of 16 (sm_103a).
//
//   s_r = sm_scale log2(e) ks[block(r)] q.c_r,   out = sum_r 2^(s_r) vs[block(r)] e_r / sum_r 2^(s_r)
//
// with c_r, e_r the codes (e4m3 or int8) of K and V row r.  The work split, the schedule
// and the merge of partial states are those of the 16-bit kernel (decode_mma.cuh,
// decode_common.cuh): every warp is an independent worker on its share of the pages.
//
// What bounds it: the codes, 2 D bytes per row and KV head, read once from HBM.  Each warp
// keeps a ring of NST 16-row tiles (K and V codes) in shared memory, filled by TMA boxes of
// 16 rows that one lane issues NST tiles ahead; a tile's two scales arrive beside it by
// 4-byte cp.async on the same mbarrier.  The ring holds the bytes in flight (an SM needs
// about 45 KB of them at the HBM rate and a 1 us latency), so the registers hold only the
// tile at hand.  The boxes are swizzled (128- or 64-byte rows) and the fragment rows
// permuted (tile_row) so that the 16-byte fragment reads of K and of V are free of bank
// conflicts.
//
// Arithmetic (mma.sync m16n8k16, fp32 accumulation: at most 8 query columns share a KV
// head's tile, an eighth of the rows a tcgen05 tile would need, and the loads bound it):
//   - codes become f16 exactly.  Q is scaled per column by a power of two into the upper
//     f16 range [2^14, 2^15): a bf16 or f16 value then keeps all its bits unless it is below
//     2^-28 of the column's largest, so one product per k-tile is exact to fp32 accumulation.
//   - the softmax denominator d = sum 2^(s - m) is held in fp32 against the running maximum
//     m of s; the weights of P.V, w = 2^(s - n) vs, go to f16 (11 significant bits) against
//     their own running maximum n of s + log2 vs, so blocks whose scales differ by any
//     factor keep the same relative precision.  out = O 2^(n - m) / d.
//   - both maxima are lazy: they move only when exceeded by more than 2^kLazyMaxBs.
// A non-finite scale makes the outputs that attend the block non-finite, as a non-finite
// row of an unquantised cache does; rows outside the attended ranges never count.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_mma.cuh"

namespace pd {

#ifndef PD_BS_STAGES
#define PD_BS_STAGES 6
#endif
#ifndef PD_BS_BLOCKS
#define PD_BS_BLOCKS 2
#endif
constexpr float kLazyMaxBs = 8.f;
// Polls of a wait for the warp's own copies before it gives up (kErrTimeout): each poll
// suspends for at most kPollNs, about a second in all, far above any memory latency.
constexpr unsigned kPollNs = 2000, kWaitPolls = 1u << 19;

// ----------------------------------------------------------------------------- mbarrier, TMA
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One arrival once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void mbar_arrive_cp_async(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok) : "r"(bar), "r"(parity), "r"(kPollNs) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned polls) {
  for (unsigned i = 0; i < polls; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
// Box of the tensor map at (x bytes, row y, block z) -> shared memory, counted on `bar`.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* tm, int x, int y, int z,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_scale(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// ----------------------------------------------------------------------------- geometry
template <int D>
struct BsTile {
  static constexpr int RB = D;           // bytes per row
  static constexpr int KT = D / 16;      // k-tiles of QK, m-tiles of PV
  static constexpr int KCH = D / 64;     // 16-byte K chunks per row and thread
  static constexpr int RL = D / 8;       // V bytes (output dims) per row and thread
  static constexpr int kBytes = 16 * RB; // one tile of K (or V) codes
  static constexpr int kStage = 2 * kBytes;
  static_assert(D == 64 || D == 128, "head dim");
};
template <int D, int NW, int NST>
constexpr int bs_smem_bytes() { return NW * NST * BsTile<D>::kStage + 1024; }

// Row of the tile that fragment row g (0..7; g + 8: the row + 8) holds.  Even g keep their
// row, odd g take (g - 1) ^ 5: rows 2i and 2i + 1 of K, read by one phase of 8 lanes, then
// differ in bit 2 (other half of the swizzled 128-byte line), and rows 0, 2, 4, 6 (or 1, 3,
// 5, 7) of V, read by the four quad lanes, in bits 1-2 (other 32-byte quarters).
__device__ __forceinline__ int tile_row(int g) { return (g & 6) ^ ((g & 1) * 5); }
// Byte offset of byte `x` of row `r` of a tile, in the TMA's swizzle (16-byte chunk index
// xor row mod 8 for 128-byte rows, xor (row / 2) mod 4 for 64-byte rows).
template <int D>
__device__ __forceinline__ int tile_off(int r, int x) {
  return r * D + (x ^ (D == 128 ? (r & 7) << 4 : ((r >> 1) & 3) << 4));
}

// four codes -> two f16x2 (codes 0, 1 and 2, 3), exact
template <typename CT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (std::is_same<CT, F8>::value) {
    lo = e4m3x2_to_f16x2((uint16_t)(w & 0xffff));
    hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  } else {
    // code + 128 below the f16 exponent of 1024: the pattern is 1024 + 128 + code
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x5140), b = __byte_perm(u, 0x64646464u, 0x5342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// ----------------------------------------------------------------------------- kernel
template <typename CT, typename QT, int D, bool MQ, int NW, int NST>
__global__ void __launch_bounds__(NW * 32, PD_BS_BLOCKS)
    decode_bs_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tm) {
  using T = BsTile<D>;
  constexpr int NT = NW * 32;
  constexpr int KT = T::KT, KCH = T::KCH, RL = T::RL;
  extern __shared__ uint8_t s_raw[];
  __shared__ int s_units[kStartCacheB];            // start-up scan scratch
  __shared__ float s_mw[NW][34][kMaxGroupPerCta];  // per-warp merge scratch
  __shared__ int s_msl[NW][32];
  __shared__ long long s_pend[NW][2][4];           // per-warp deferred merges
  __shared__ WorkerStart s_start[NW];
  __shared__ __align__(8) uint64_t s_bar[NW][NST];
  __shared__ __align__(8) float2 s_sc[NW][NST];    // scales (K, V) of the stage's tile
  __shared__ int4 s_info[NW][NST];                 // its attended rows [x, y), first row's index z

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring = ((smem_u32(s_raw) + 1023u) & ~1023u) + (uint32_t)(warp * NST * T::kStage);
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm) : "memory");
    prefetch_l2_share(p.Q, (size_t)p.B * p.q_len * p.H_qo * D * sizeof(QT), blockIdx.x, gridDim.x);
    if (p.values) prefetch_l2_share(p.values, (size_t)p.nnz_pages * sizeof(int32_t), blockIdx.x, gridDim.x);
  }
  if (lane == 0) {
    // two arrivals per fill: the issuing lane's (with the boxes' bytes) and its cp.async copies'
    for (int i = 0; i < NST; ++i) mbar_init(smem_u32(&s_bar[warp][i]), 2);
    mbar_init_fence();
  }
  if (!p.early_inputs) {
    pdl_wait();
    pdl_release();
  }
  worker_starts<NT, NW>(p, s_start, s_units);  // the last block-wide barrier of the kernel

  const int g_id = lane >> 2, q4 = lane & 3;
  const WorkerStart ws = s_start[warp];
  if (ws.b < 0) return;  // no units for this worker

  const int P = p.P;
  const int zg = p.mode == kSchedBalanced ? p.zg : 1;
  const long long Wn = (long long)gridDim.x * NW / zg;
  const long long wid = (long long)blockIdx.x * NW + warp;

  Segment sg;
  sg.b = ws.b;
  sg.hz = ws.hz;
  sg.off = ws.off;
  sg.seq = load_seq(p, sg.b);
  sg.n = units_of(sg.seq, P);
  const int C = p.mode == kSchedBalanced ? p.seg_cost : 0;
  const long long cx1 = p.mode == kSchedBalanced ? ws.x1 : sg.off + sg.n;

  int npend = 0;
  if (lane < 2) s_pend[warp][lane][0] = -1;
  __syncwarp();

  // this thread's fragment rows (+ 8: the second half) and their byte offsets in a tile
  const int kr = tile_row(g_id);
  int koff[KCH], voff[2];
#pragma unroll
  for (int c = 0; c < KCH; ++c) koff[c] = tile_off<D>(kr, 16 * (4 * c + q4));
  const int vr[2] = {tile_row(2 * q4), tile_row(2 * q4 + 1)};
#pragma unroll
  for (int i = 0; i < 2; ++i) voff[i] = tile_off<D>(vr[i], RL * g_id);

  // The ring: tiles are filled into stage `ist` and read from stage `cst`, in order.
  int ist = 0, cst = 0, in_flight = 0;
  uint32_t cph = 0;      // parity of the fill that stage cst waits for
  bool waited = !p.early_inputs;
  bool dead = false;     // a wait ran out: no further fills

  for (;;) {
  const int ua = (int)min(max(ws.x0 - sg.off - C, 0ll), (long long)sg.n);
  const int ub = (int)min(max(cx1 - sg.off - C, 0ll), (long long)sg.n);
  if (ua < ub) {
  const int hk = sg.hz / p.n_z, z = sg.hz - (sg.hz / p.n_z) * p.n_z;
  const Pieces pcs = make_pieces(0, sg.seq.L, sg.seq, P);
  const int pend = min(ub, sg.seq.L > 0 ? pcs.count() : 0);
  const int c0 = z * kMaxGroupPerCta;
  const int hcount = min(kMaxGroupPerCta, p.ncol - c0);

  // Raw Q of column g_id at this lane's B-fragment dims (16 (4c + q4) .. + 15), loaded first
  const bool have_q = g_id < hcount;
  uint4 qraw[2 * KCH];
  {
    const QT* qrow = reinterpret_cast<const QT*>(p.Q) + col_row<MQ>(p, sg.b, hk, c0 + (have_q ? g_id : 0)) * D;
#pragma unroll
    for (int c = 0; c < 2 * KCH; ++c)
      qraw[c] = have_q ? __ldg(reinterpret_cast<const uint4*>(qrow + 16 * (4 * (c >> 1) + q4) + 8 * (c & 1)))
                       : make_uint4(0u, 0u, 0u, 0u);
  }
  int lim0 = 0, lim1 = 0;  // attended-row limits of this lane's two score columns
  if constexpr (MQ) {
    const int cc = c0 + 2 * q4;
    lim0 = sg.seq.L - p.q_len + 1 + cc / p.group;
    lim1 = sg.seq.L - p.q_len + 1 + (cc + 1) / p.group;
  }

  // ---------------------------------------------------------------- tile stream
  // Pieces (page, slot range) [ua, pend) in order, 32 at a time: lane i holds piece
  // pb_base + i, handed out with shuffles.
  struct Tile {
    int blk;                      // K block (page, hk) of the cache; -1: no more tiles
    int piece, t, s_lo, s_hi, r_lo;
  };
  int pb_base = -64, pb_page = -1, pb_slots = 0, pb_row = 0;
  auto first_tile_from = [&](int j) -> Tile {
    Tile tl;
    tl.blk = -1;
    tl.piece = pend;
    tl.t = tl.s_lo = tl.s_hi = tl.r_lo = 0;
    for (; j < pend; ++j) {
      if (j >= pb_base + 32) {
        pb_base = j;
        pb_page = -1;
        if (j + lane < pend) {
          const Piece pc = get_piece(pcs, j + lane, P);
          pb_page = lookup_page(p, sg.seq, pc.page_idx);  // -1 (error recorded) if out of range
          pb_slots = pc.s_lo | (pc.s_hi << 16);
          pb_row = pc.r_lo;
        }
      }
      const int src = j - pb_base;
      const int pg = __shfl_sync(0xffffffffu, pb_page, src);
      if (pg < 0) continue;  // bad page id: its rows are skipped
      const int sl = __shfl_sync(0xffffffffu, pb_slots, src);
      tl.piece = j;
      tl.s_lo = sl & 0xffff;
      tl.s_hi = sl >> 16;
      tl.t = tl.s_lo >> 4;
      tl.r_lo = __shfl_sync(0xffffffffu, pb_row, src);
      tl.blk = pg * 2 * p.H_kv + hk;
      break;
    }
    return tl;
  };
  auto next_tile = [&](const Tile& c) -> Tile {
    if ((c.t + 1) * 16 < c.s_hi) {  // (warp-uniform)
      Tile n = c;
      n.t = c.t + 1;
      return n;
    }
    return first_tile_from(c.piece + 1);
  };
  // the tile's boxes and scales -> stage ist
  auto issue = [&](const Tile& c) {
    if (lane == 0) {
      const uint32_t bar = smem_u32(&s_bar[warp][ist]);
      const uint32_t dst = ring + ist * T::kStage;
      s_info[warp][ist] = make_int4(c.s_lo - c.t * 16, c.s_hi - c.t * 16, c.r_lo + c.t * 16 - c.s_lo, 0);
      const float* ks = p.scales + (size_t)c.blk * p.n_sb + (c.t * 16) / p.scale_rows;
      cp_async_scale(smem_u32(&s_sc[warp][ist].x), ks);
      cp_async_scale(smem_u32(&s_sc[warp][ist].y), ks + (size_t)p.H_kv * p.n_sb);
      mbar_arrive_cp_async(bar);
      mbar_arrive_expect_tx(bar, T::kStage);
      tma_load_box(dst, &tm, 0, c.t * 16, c.blk, bar);
      tma_load_box(dst + T::kBytes, &tm, 0, c.t * 16, c.blk + p.H_kv, bar);
    }
    ist = ist + 1 == NST ? 0 : ist + 1;
    ++in_flight;
  };

  Tile nxt = first_tile_from(ua);
  if (!waited) {  // pages and scales may still be written by the previous kernel until here
    pdl_wait();
    pdl_release();
    waited = true;
  }
#pragma unroll 1
  for (int i = 0; i < NST && nxt.blk >= 0 && !dead; ++i) {
    issue(nxt);
    nxt = next_tile(nxt);
  }

  // ---------------------------------------------------------------- Q^T B fragments
  // k-tile kt: dims 16 (4 (kt >> 2) + q4) + 4 (kt & 3) + {0, 1} and + {2, 3} of column g_id,
  // times 2^(14 - e), e the exponent of the column's largest magnitude
  uint32_t qf[KT][2];
  float cs0, cs1;  // column factors of this lane's score columns: 2^(e - 14) sm_scale log2(e)
  {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < 2 * KCH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<QT>(comp(qraw[c], i));
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^(14 - e) and its inverse, both normal: e is kept in [-100, 126]
    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255) - 127, -100), 126);
    const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
    const float cs = __uint_as_float((unsigned)(127 - 14 + e) << 23) * p.score_scale;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 f = unpack2<QT>(comp(qraw[2 * (kt >> 2) + ((kt & 3) >> 1)], 2 * (kt & 1) + h));
        qf[kt][h] = pack2<__half>(f.x * up, f.y * up);
      }
    cs0 = __shfl_sync(0xffffffffu, cs, 8 * q4);      // column 2 q4
    cs1 = __shfl_sync(0xffffffffu, cs, 8 * q4 + 4);  // column 2 q4 + 1
  }

  float st_m[2] = {kEmptyM, kEmptyM}, st_d[2] = {0.f, 0.f}, st_n[2] = {kEmptyM, kEmptyM};
  float oacc[KT][4];
#pragma unroll
  for (int i = 0; i < KT; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;

  __syncwarp();  // lane 0's s_info is read by the warp
#pragma unroll 1
  while (in_flight > 0) {
    const bool ok = mbar_wait(smem_u32(&s_bar[warp][cst]), cph, dead ? 1024u : kWaitPolls);
    if (__any_sync(0xffffffffu, !ok)) {
      dead = true;  // what follows is not used: the error word says so
      if (lane == 0) set_error(p.err, kErrTimeout);
    }
    const uint8_t* kt_base = s_raw + (ring - smem_u32(s_raw)) + cst * T::kStage;
    const uint8_t* vt_base = kt_base + T::kBytes;
    const int4 info = s_info[warp][cst];
    const float2 sc2 = s_sc[warp][cst];
    // ---------------------------------------------------------------- S^T = C Q^T
    uint4 ka[2][KCH];
#pragma unroll
    for (int c = 0; c < KCH; ++c) {
      ka[0][c] = *reinterpret_cast<const uint4*>(kt_base + koff[c]);
      ka[1][c] = *reinterpret_cast<const uint4*>(kt_base + 8 * D + koff[c]);
    }
    float qacc[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) qacc[c][0] = qacc[c][1] = qacc[c][2] = qacc[c][3] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      uint32_t a[4];
      codes_to_f16<CT>(comp(ka[0][kt >> 2], kt & 3), a[0], a[2]);
      codes_to_f16<CT>(comp(ka[1][kt >> 2], kt & 3), a[1], a[3]);
      Mma<__half>::run(qacc[kt & 1], a, qf[kt][0], qf[kt][1]);
    }
    // V rows vr[0], vr[1], vr[0] + 8, vr[1] + 8: bytes RL g_id .. + RL - 1
    uint32_t va[4][RL / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* src = vt_base + (i >> 1) * 8 * D + voff[i & 1];
      if constexpr (RL == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        va[i][0] = v.x;
        va[i][1] = v.y;
        va[i][2] = v.z;
        va[i][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        va[i][0] = v.x;
        va[i][1] = v.y;
      }
    }
    // ---------------------------------------------------------------- online softmax (log2)
    const bool full = info.x <= 0 && info.y >= 16;
    const float f0 = cs0 * sc2.x, f1 = cs1 * sc2.x;
    float sc[4];
    sc[0] = (qacc[0][0] + qacc[1][0]) * f0;  // row kr, columns 2 q4, 2 q4 + 1
    sc[1] = (qacc[0][1] + qacc[1][1]) * f1;
    sc[2] = (qacc[0][2] + qacc[1][2]) * f0;  // row kr + 8
    sc[3] = (qacc[0][3] + qacc[1][3]) * f1;
    if (!full) {
      if (kr < info.x || kr >= info.y) sc[0] = sc[1] = -INFINITY;
      if (kr + 8 < info.x || kr + 8 >= info.y) sc[2] = sc[3] = -INFINITY;
      // rows outside may hold any code (e4m3 NaN): their V bytes are zeroed
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = vr[i & 1] + 8 * (i >> 1);
        if (r < info.x || r >= info.y) {
#pragma unroll
          for (int k = 0; k < RL / 4; ++k) va[i][k] = 0u;
        }
      }
    }
    if constexpr (MQ) {  // causal among the new tokens
      const int r0 = info.z + kr;
      if (r0 >= lim0) sc[0] = -INFINITY;
      if (r0 >= lim1) sc[1] = -INFINITY;
      if (r0 + 8 >= lim0) sc[2] = -INFINITY;
      if (r0 + 8 >= lim1) sc[3] = -INFINITY;
    }
    const float lv = __log2f(sc2.y);
    {
      const float t0 = fmaxf(sc[0], sc[2]), t1 = fmaxf(sc[1], sc[3]);
      const float over = fmaxf(fmaxf(t0 - st_m[0], t1 - st_m[1]),
                               fmaxf(t0 + lv - st_n[0], t1 + lv - st_n[1]));
      if (__any_sync(0xffffffffu, over > kLazyMaxBs)) {
        const float tm0 = max_over_groups(t0), tm1 = max_over_groups(t1);
        const float mn0 = fmaxf(st_m[0], tm0), mn1 = fmaxf(st_m[1], tm1);
        st_d[0] *= fast_exp2(st_m[0] - mn0);
        st_d[1] *= fast_exp2(st_m[1] - mn1);
        st_m[0] = mn0;
        st_m[1] = mn1;
        const float nn0 = fmaxf(st_n[0], tm0 + lv), nn1 = fmaxf(st_n[1], tm1 + lv);
        const float a0 = fast_exp2(st_n[0] - nn0), a1 = fast_exp2(st_n[1] - nn1);
        st_n[0] = nn0;
        st_n[1] = nn1;
#pragma unroll
        for (int mt = 0; mt < KT; ++mt) {
          oacc[mt][0] *= a0;
          oacc[mt][1] *= a1;
          oacc[mt][2] *= a0;
          oacc[mt][3] *= a1;
        }
      }
    }
    float pr[4];
    pr[0] = fast_exp2(sc[0] - st_m[0]);
    pr[1] = fast_exp2(sc[1] - st_m[1]);
    pr[2] = fast_exp2(sc[2] - st_m[0]);
    pr[3] = fast_exp2(sc[3] - st_m[1]);
    st_d[0] += pr[0] + pr[2];
    st_d[1] += pr[1] + pr[3];
    // weights of P.V: 2^(s - n) vs = p 2^(m - n) vs; a row that does not count weighs 0
    // whatever the scale (the exponent is capped so that a zero scale stays zero)
    const float w0 = sc2.y * fast_exp2(fminf(st_m[0] - st_n[0], 126.f));
    const float w1 = sc2.y * fast_exp2(fminf(st_m[1] - st_n[1], 126.f));
    pr[0] = pr[0] == 0.f ? 0.f : pr[0] * w0;
    pr[1] = pr[1] == 0.f ? 0.f : pr[1] * w1;
    pr[2] = pr[2] == 0.f ? 0.f : pr[2] * w0;
    pr[3] = pr[3] == 0.f ? 0.f : pr[3] * w1;
    // P^T as a B fragment: fragment rows 2q, 2q + 1 | 2q + 8, 2q + 9 of column g_id
    uint32_t pb0, pb1;
    {
      const uint32_t x0 = pack2<__half>(pr[0], pr[2]);  // column 2q: rows of g_id, g_id + 8
      const uint32_t x1 = pack2<__half>(pr[1], pr[3]);  // column 2q + 1
      const int srcA = 8 * q4 + (g_id >> 1), srcB = srcA + 4;
      const uint32_t a0 = __shfl_sync(0xffffffffu, x0, srcA);
      const uint32_t a1 = __shfl_sync(0xffffffffu, x1, srcA);
      const uint32_t b0 = __shfl_sync(0xffffffffu, x0, srcB);
      const uint32_t b1 = __shfl_sync(0xffffffffu, x1, srcB);
      const uint32_t wa = (g_id & 1) ? a1 : a0, wb = (g_id & 1) ? b1 : b0;
      pb0 = __byte_perm(wa, wb, 0x5410);
      pb1 = __byte_perm(wa, wb, 0x7632);
    }
    // ---------------------------------------------------------------- O^T += V^T P^T
    // m-tile mt: rows g_id / g_id + 8 are dims RL g_id + 2 mt / + 1
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) {
      const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
      uint32_t a[4];
      codes_to_f16<CT>(__byte_perm(va[0][mt >> 1], va[1][mt >> 1], sel), a[0], a[1]);
      codes_to_f16<CT>(__byte_perm(va[2][mt >> 1], va[3][mt >> 1], sel), a[2], a[3]);
      Mma<__half>::run(oacc[mt], a, pb0, pb1);
    }
    // every lane has its codes in registers: the stage takes the next tile
    cst = cst + 1 == NST ? 0 : cst + 1;
    if (cst == 0) cph ^= 1;
    --in_flight;
    __syncwarp();
    if (nxt.blk >= 0 && !dead) {
      issue(nxt);
      nxt = next_tile(nxt);
      __syncwarp();
    }
  }
  st_d[0] = sum_over_groups(st_d[0]);
  st_d[1] = sum_over_groups(st_d[1]);

  // ---------------------------------------------------------------- finish the segment
  // This thread holds columns 2 q4 (o0, o2) and 2 q4 + 1 (o1, o3), dims RL g_id .. + RL - 1
  const bool whole = (ua == 0 && ub == sg.n);
  const size_t slot = (size_t)(2 * wid + (sg.off <= ws.x0 ? 0 : 1)) * kMaxGroupPerCta;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int j = 2 * q4 + hh;
    if (j < hcount) {
      const bool empty = st_d[hh] == 0.f;
      float inv = empty ? 0.f : exp2f(st_n[hh] - st_m[hh]) / st_d[hh];
      float l = empty ? kEmptyM : st_m[hh] + log2f(st_d[hh]);
      const size_t row = col_row<MQ>(p, sg.b, hk, c0 + j);
      if (whole && p.sink) {
        const SinkAdj sa = apply_sink(p, col_head<MQ>(p, hk, c0 + j), l);
        inv *= sa.scale;
        l = sa.lse;
      }
      float v[RL];
#pragma unroll
      for (int o = 0; o < RL; ++o) v[o] = oacc[o >> 1][hh + 2 * (o & 1)] * inv;
      if (whole) {
        store_run<RL>(p, row * D + RL * g_id, v);
      } else {
        float4* po = reinterpret_cast<float4*>(p.part_o + (slot + j) * D + RL * g_id);
#pragma unroll
        for (int i = 0; i < RL / 4; ++i) po[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      if (g_id == 0) {
        if (whole) p.lse[row] = l;
        else p.part_lse[slot + j] = l;
      }
    }
  }
  if (!whole) {
    // publish the partial; the worker completing the segment's count merges later
    fence_acq_rel_gpu();
    __syncwarp();
    int last = 0;
    if (lane == 0) {
      int* cnt = p.counters + (size_t)sg.b * p.H_kv * p.n_z + sg.hz;
      const int mine = ub - ua;
      const int prev = atomicAdd(cnt, mine);
      last = (prev + mine == sg.n);
      if (last) *cnt = 0;
    }
    last = __shfl_sync(0xffffffffu, last, 0);
    if (last) {
      fence_acq_rel_gpu();
      if (lane == 0) {
        s_pend[warp][npend][0] = sg.b;
        s_pend[warp][npend][1] = sg.hz;
        s_pend[warp][npend][2] = sg.off;
        s_pend[warp][npend][3] = sg.n;
      }
      npend = 1;  // at most two entries
    }
  }
  }  // ua < ub
  if (sg.off + C + sg.n >= cx1 || !next_segment(p, sg, C)) break;
  }  // segments

  // ---------------------------------------------------------------- deferred merges
  __syncwarp();
  for (int i = 0; i < 2; ++i) {
    const long long b = s_pend[warp][i][0];
    if (b < 0) continue;
    const int hz = (int)s_pend[warp][i][1];
    const long long off = s_pend[warp][i][2];
    const int n = (int)s_pend[warp][i][3];
    const int hk = hz / p.n_z, z = hz - hk * p.n_z;
    const int c0 = z * kMaxGroupPerCta;
    const int hcount = min(kMaxGroupPerCta, p.ncol - c0);
    constexpr int kBudget = 8;  // float4 partial rows per lane in flight
    constexpr int kV4 = (4 * (D / 4) + 31) / 32, kV8 = (8 * (D / 4) + 31) / 32;
    if (hcount <= 4)
      warp_merge<D, 4, (kBudget / kV4 > 1 ? kBudget / kV4 : 1), MQ>(p, (int)b, off, C, n, ws.U, Wn, hk, c0, hcount, s_mw[warp], s_msl[warp], zg, (int)(wid % zg));
    else
      warp_merge<D, 8, (kBudget / kV8 > 1 ? kBudget / kV8 : 1), MQ>(p, (int)b, off, C, n, ws.U, Wn, hk, c0, hcount, s_mw[warp], s_msl[warp], zg, (int)(wid % zg));
  }
}

// ----------------------------------------------------------------------------- launch
template <typename CT, typename QT, int D, bool MQ>
static cudaError_t launch_bs_t(const DecodeParams& p, const CUtensorMap& tm, dim3 grid,
                               cudaStream_t st, MmaConfig* cfg) {
  constexpr int NW = kMmaWarps, NST = PD_BS_STAGES;
  constexpr int dyn = bs_smem_bytes<D, NW, NST>();
  auto kern = decode_bs_kernel<CT, QT, D, MQ, NW, NST>;
  // the dynamic shared memory above 48 KB is opted into on every query of the launch
  // configuration, which the host makes once per device and variant before the first launch
  if (cfg) {
    cfg->threads = NW * 32;
    cfg->smem_bytes = dyn;
    int n = 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, NW * 32, dyn);
    if (e != cudaSuccess) return e;
    cfg->ctas_per_sm = n;
    return cudaSuccess;
  }
  return launch_pdl(kern, grid, dim3(NW * 32), dyn, st, p, tm);
}

template <typename CT>
static cudaError_t launch_bs_any(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                                 cudaStream_t st, MmaConfig* cfg) {
  const bool mq = p.q_len > 1;
  auto with_q = [&](auto q_tag) -> cudaError_t {
    using QT = decltype(q_tag);
    if (p.D == 128)
      return mq ? launch_bs_t<CT, QT, 128, true>(p, tm, grid, st, cfg)
                : launch_bs_t<CT, QT, 128, false>(p, tm, grid, st, cfg);
    if (p.D == 64)
      return mq ? launch_bs_t<CT, QT, 64, true>(p, tm, grid, st, cfg)
                : launch_bs_t<CT, QT, 64, false>(p, tm, grid, st, cfg);
    return cudaErrorInvalidValue;
  };
  if (q_dtype == kBF16) return with_q(__nv_bfloat16{});
  if (q_dtype == kF16) return with_q(__half{});
  return cudaErrorInvalidValue;
}

}  // namespace pd
