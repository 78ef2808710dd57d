// Tensor-core decode of an 8-bit KV cache with one fp32 scale per (page, K | V, KV head,
// block of S rows), S a multiple of 16 (sm_103a).
//
//   s_r = sm_scale log2(e) ks[block(r)] q.c_r,   out = sum_r 2^(s_r) vs[block(r)] e_r / sum_r 2^(s_r)
//
// with c_r, e_r the codes (e4m3 or int8) of K and V row r.  The work split and the schedule are
// those of the 16-bit kernel (decode_mma.cuh, decode_common.cuh): every warp is an independent
// worker on its share of the pages.
//
// What bounds it: the codes, 2 D bytes per row and KV head, read once from HBM (DRAM traffic
// 1.001 to 1.005 of them).  Each warp keeps a ring of two stages in shared memory, NQ 16-row
// tiles each (8 KB); a tile's K and V rows come by one 5-D TMA box and its two scales by 4-byte cp.async on the
// stage's mbarrier, issued by NQ lanes at once while the other stage is computed.  Eight warps an
// SM then hold up to 128 KB in flight (the HBM rate times a 1 us latency needs about 45 KB of an
// SM); more and smaller blocks, or deeper rings in fewer blocks, were slower (256 sequences: 197
// us with 12 warps of one tile at a time, 185 us now).  The boxes are swizzled (128- or 64-byte
// rows) and the fragment rows permuted (tile_row) so that the fragment reads of K and V are free
// of bank conflicts (D 64: two-way on V).
//   A warp's time per tile is a chain of dependent steps, so a stage's NQ tiles are computed
// together: their chains overlap and share the vote, the rescale and the wait (a tile alone in a
// warp: 0.83 us one by one, 0.42 us now).  Short lists are padded with empty tiles; one copy of the
// code for full stages only keeps the loop in reach of the instruction cache, whose misses are the
// largest stall left (int8: 1.0 of 5.1 cycles an instruction; e4m3: 1.5 of 6.7, level with the
// fixed waits between dependent instructions).
//   Measured on one GB300 (of the 6779 GB/s copy rate): eight contexts of 32K to 128K rows 194 us
// (96 %; e4m3 in blocks of 64 rows 191 us, 98 %), 256 sequences of 300 to 4200 rows 185 us (91 %),
// 32 of 512 to 4096 rows 34 us (55 %: about 3 us until the first tile, 3 us of uneven ends and 7 us
// of merging stand beside 18.5 us of bytes), 300 rows alone 7.0 us.
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
// A NaN or infinite scale makes the outputs that attend the block NaN, whatever the weights;
// rows outside the attended ranges never count.
#pragma once

#include <cuda.h>

#include <cfloat>
#include <type_traits>

#include "decode_mma.cuh"

namespace pd {

constexpr int kBsStages = 2;  // ring stages per warp
constexpr int kBsBlocks = 2;  // resident blocks per SM: shared memory (84 KB at D 128) and 256 registers
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
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(bar) : "memory");
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
// Rows y .. y + 15 of a page's head, K then V (one box of the tensor map) -> shared memory,
// counted on `bar`.
__device__ __forceinline__ void tma_load_tile(uint32_t dst, const CUtensorMap* tm, int y, int head, int page,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %2, %5}], [%6];"
      ::"r"(dst), "l"(tm), "r"(0), "r"(y), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_chunk(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
  static constexpr int kPair = 2 * kBytes;  // K and V
  static constexpr int NQ = D == 64 ? 4 : 2;      // tiles computed together
  static constexpr int NST = kBsStages;        // ring stages per warp, of NQ tiles each
  static constexpr int kStage = NQ * kPair;
  static constexpr int kState = kMaxGroupPerCta * D * 4;  // a partial state's outputs, fp32
  static_assert(D == 64 || D == 128, "head dim");
};
// the warps' rings, then the state each may hold from its first segment
template <int D, int NW>
constexpr int bs_smem_bytes() { return NW * (BsTile<D>::NST * BsTile<D>::kStage + BsTile<D>::kState) + 1024; }

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

// The smaller of two, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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

// Four consecutive output dims at element idx (a multiple of 4).
__device__ __forceinline__ void store_four(const DecodeParams& p, size_t idx, float4 v) {
  if (p.out_dtype == kF32) {
    float* o = reinterpret_cast<float*>(p.out) + idx;
    if (p.out_vec16) *reinterpret_cast<float4*>(o) = v;
    else o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
  } else {
    const bool bf = p.out_dtype == kBF16;
    const uint32_t a = bf ? pack2<__nv_bfloat16>(v.x, v.y) : pack2<__half>(v.x, v.y);
    const uint32_t b = bf ? pack2<__nv_bfloat16>(v.z, v.w) : pack2<__half>(v.z, v.w);
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + idx;
    if (p.out_vec16) *reinterpret_cast<uint2*>(o) = make_uint2(a, b);
    else o[0] = (uint16_t)a, o[1] = (uint16_t)(a >> 16), o[2] = (uint16_t)b, o[3] = (uint16_t)(b >> 16);
  }
}

// A warp's partial state of a segment: the segment (its place on the cost line, sequence, head
// slice, units; the slice's KV head, first column and columns) and how many of its units the
// state holds; b < 0: none.
struct PartEntry {
  long long off;
  int b, hz, mine, n, hk, c0, hcount;
};
// ----------------------------------------------------------------------------- kernel
// ROWS: tiles of 16 consecutive attended rows of any pages, gathered row by row, each row with its
// own scales; else tiles are 16 rows of one page that share a scale (page size and rows per scale
// multiples of 16).
template <typename CT, typename QT, int D, bool MQ, bool ROWS, int NW>
__global__ void __launch_bounds__(NW * 32, kBsBlocks)
    decode_bs_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tm) {
  using T = BsTile<D>;
  constexpr int NT = NW * 32;
  constexpr int KT = T::KT, KCH = T::KCH, RL = T::RL, NQ = T::NQ, NST = T::NST;
  extern __shared__ uint8_t s_raw[];
  __shared__ PartEntry s_part[NW][2];              // each warp's partial states: first, last segment
  __shared__ float s_plse[NW][2][kMaxGroupPerCta]; // their lse
  __shared__ int s_last[2 * NW];
  __shared__ WorkerStart s_start[NW];
  __shared__ __align__(8) uint64_t s_bar[NW][NST];
  __shared__ float4 s_meta[NW][NST][NQ];  // of a tile: K and V scale, attended rows, first row's index
  __shared__ float2 s_rowsc[ROWS ? NW : 1][ROWS ? NST : 1][ROWS ? NQ * 16 : 1];  // ROWS: each row's scales,
  __shared__ unsigned s_rowok[ROWS ? NW : 1][ROWS ? NST : 1][ROWS ? NQ / 2 : 1];  // and which rows count

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* const rings = s_raw + (((smem_u32(s_raw) + 1023u) & ~1023u) - smem_u32(s_raw));
  const uint32_t bar0 = smem_u32(&s_bar[warp][0]), meta0 = smem_u32(&s_meta[warp][0][0]);
  uint8_t* const my_ring = rings + warp * NST * T::kStage;
  const uint32_t ring = smem_u32(my_ring);
  // the rings' space before the first fill: scratch of the start-up scan; after a warp's last
  // tile, its part: the state of its last segment
  static_assert(NW * NST * T::kStage >= kStartCacheB * 4 && NST * T::kStage >= T::kState, "scratch");
  int* const s_units = reinterpret_cast<int*>(rings);
  auto state_of = [&](int w, int side) -> float* {
    return reinterpret_cast<float*>(side ? rings + w * NST * T::kStage : rings + NW * NST * T::kStage + w * T::kState);
  };
  if (threadIdx.x == 0) {
    if constexpr (!ROWS) asm volatile("prefetch.tensormap [%0];" ::"l"(&tm) : "memory");  // (ROWS: none)
    prefetch_l2_share(p.Q, (size_t)p.B * p.q_len * p.H_qo * D * sizeof(QT), blockIdx.x, gridDim.x);
    if (p.values) prefetch_l2_share(p.values, (size_t)p.nnz_pages * sizeof(int32_t), blockIdx.x, gridDim.x);
  }
  if (lane == 0) {
    // per tile two arrivals: the issuing lane's (with the box's bytes) and its cp.async copies'; ROWS:
    // per stage one of every lane's copies
    for (int i = 0; i < NST; ++i) mbar_init(bar0 + i * 8, ROWS ? 32 : 2 * NQ);
    mbar_init_fence();
  }
  // With a host plan the start-up reads launch parameters alone and runs under the tail of the
  // kernel before; otherwise, as everywhere, nothing of the caller's is read before it completes.
  bool waited = false;
  if (!p.early_inputs && !p.hp_B) {
    pdl_wait();
    pdl_release();
    waited = true;
  }
  worker_starts<NT, NW>(p, s_start, s_units);
  // the scan's shared memory accesses before the fills that overwrite its scratch
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (lane < 2) s_part[warp][lane].b = -1;
  __syncthreads();  // no block-wide barrier until every warp has finished its range

  const int g_id = lane >> 2, q4 = lane & 3;
  const WorkerStart ws = s_start[warp];
  const int P = p.P;
  const int zg = p.mode == kSchedBalanced ? p.zg : 1;

  Segment sg;
  sg.b = max(ws.b, 0);  // (ws.b < 0: no units for this worker)
  sg.hz = ws.hz;
  sg.off = ws.off;
  sg.seq = load_seq(p, sg.b);
  sg.n = units_of(sg.seq, P);
  const int C = p.mode == kSchedBalanced ? p.seg_cost : 0;
  const long long cx1 = p.mode != kSchedPerSegment ? ws.x1 : sg.off + sg.n;

  // this thread's fragment rows (+ 8: the second half) and their byte offsets in a tile
  const int kr = tile_row(g_id);
  int koff[KCH], voff[2];
#pragma unroll
  for (int c = 0; c < KCH; ++c) koff[c] = tile_off<D>(kr, 16 * (4 * c + q4));
  const int vr[2] = {tile_row(2 * q4), tile_row(2 * q4 + 1)};
#pragma unroll
  for (int i = 0; i < 2; ++i) voff[i] = tile_off<D>(vr[i], RL * g_id);

  // The ring: NQ tiles at a time are filled into stage `ist` and read from stage `cst`, in order.
  int ist = 0, cst = 0;
  uint32_t cph = 0;   // parity of the fill that stage cst waits for
  bool dead = false;  // a wait ran out: no further fills
  if (!p.early_inputs && !waited) {
    pdl_wait();
    pdl_release();
    waited = true;
  }

  while (ws.b >= 0) {
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
  // The share's pieces are whole pages of at most two runs of attended offsets (A: the sinks,
  // or every row; B: the window), so its tiles are the multiples of 16 of each run in order.
  // Tiles come 32 at a time: lane i holds tile 32 m + i and issues it; the page ids of the
  // next 32 are loaded meanwhile.
  const int a_lo = max(pcs.ra0, (pcs.pa + min(ua, pcs.na)) * P), a_hi = min(pcs.ra1, (pcs.pa + min(pend, pcs.na)) * P);
  const int b_lo = max(pcs.ob0, (pcs.pb + max(ua - pcs.na, 0)) * P), b_hi = min(pcs.ob1, (pcs.pb + max(pend - pcs.na, 0)) * P);
  const int n_a = a_hi <= a_lo ? 0 : ROWS ? a_hi - a_lo : ((a_hi + 15) >> 4) - (a_lo >> 4);
  const int n_b = b_hi <= b_lo ? 0 : ROWS ? b_hi - b_lo : ((b_hi + 15) >> 4) - (b_lo >> 4);
  const int n_tiles = ROWS ? (n_a + n_b + 15) >> 4 : n_a + n_b;  // (ROWS: n_a, n_b count rows)
  auto tile_at = [&](int k) { return k < n_a ? ((a_lo >> 4) + k) << 4 : ((b_lo >> 4) + k - n_a) << 4; };  // offset
  auto load_page = [&](int k) -> int {  // page id of tile k, unchecked; -1 out of the table
    if (k >= n_tiles) return -1;
    const int pidx = tile_at(k) / P;
    return pidx < sg.seq.npages && (long long)sg.seq.page_begin + pidx < p.nnz_pages
               ? __ldg(p.values + sg.seq.page_begin + pidx) : -1;
  };
  int t_page = -1, t_row = 0, t_span = 0, t_r0 = 0, page_next = ROWS ? -1 : load_page(lane);
  auto load_batch = [&](int k0) {  // tiles k0 .. k0 + 31
    const int k = k0 + lane, page = page_next;
    page_next = load_page(k + 32);
    const int o = tile_at(k);
    const bool in_a = k < n_a;
    t_row = o % P;
    t_span = max((in_a ? a_lo : b_lo) - o, 0) | (min((in_a ? a_hi : b_hi) - o, 16) << 8);
    t_r0 = in_a ? o : o - pcs.shift;
    t_page = page;
    if (page < 0 || page >= p.max_pages) {
      if (k < n_tiles) set_error(p.err, kErrBadPage);
      t_page = -1;  // no such tile, or its rows do not count
    }
  };
  // ROWS: the page (unchecked; -1 out of the table) and slot of a lane's rows 32 h + lane of the
  // stage that starts with tile k, loaded one stage ahead
  int rw_page[NQ / 2], rw_slot[NQ / 2];
  auto load_rows = [&](int k) {
#pragma unroll
    for (int h = 0; h < NQ / 2; ++h) {
      const int i = k * 16 + 32 * h + lane;
      rw_page[h] = rw_slot[h] = -1;
      if (i < n_a + n_b) {
        const int o = i < n_a ? a_lo + i : b_lo + i - n_a, pidx = o / P;
        rw_slot[h] = o - pidx * P;
        if (pidx < sg.seq.npages && (long long)sg.seq.page_begin + pidx < p.nnz_pages)
          rw_page[h] = __ldg(p.values + sg.seq.page_begin + pidx);
      }
    }
  };
  if constexpr (ROWS) load_rows(0);
  // its rows -> stage ist: D / 16 lanes copy a row's 16-byte chunks, the row's own lane its scales
  auto issue_rows = [&](int k) {
    constexpr int CPR = D / 16, RPI = 32 / CPR;  // chunks per row, rows per instruction
    const size_t to_v = (size_t)p.H_kv * P * D;
#pragma unroll
    for (int h = 0; h < NQ / 2; ++h) {
      const int page = rw_page[h], slot = rw_slot[h];
      const bool ok = page >= 0 && page < p.max_pages;
      if (slot >= 0 && !ok) set_error(p.err, kErrBadPage);  // its row does not count
      const unsigned rows = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) s_rowok[warp][ist][h] = rows;
      float2* const sc = &s_rowsc[warp][ist][32 * h + lane];
      if (ok) {
        const float* ks = p.scales + ((size_t)page * 2 * p.H_kv + hk) * p.n_sb + ((slot * p.sb_mul) >> 20);
        cp_async_scale(smem_u32(&sc->x), ks);
        cp_async_scale(smem_u32(&sc->y), ks + (size_t)p.H_kv * p.n_sb);
      } else {
        *sc = make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int it = 0; it < CPR; ++it) {
        const int r = it * RPI + lane / CPR, x = lane % CPR * 16;  // row of the 32, byte of it
        const int pg = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, slot, r);
        if ((rows >> r) & 1) {
          const uint8_t* src = reinterpret_cast<const uint8_t*>(p.pages) +
                               (((size_t)pg * 2 * p.H_kv + hk) * P + sl) * D + x;
          const uint32_t dst = ring + ist * T::kStage + (2 * h + (r >> 4)) * T::kPair + tile_off<D>(r & 15, x);
          cp_async_chunk(dst, src);
          cp_async_chunk(dst + T::kBytes, src + to_v);
        }
      }
    }
    mbar_arrive_cp_async(bar0 + ist * 8);
    ist = ist + 1 == NST ? 0 : ist + 1;
    load_rows(k + NQ);
  };
  // tiles k .. k + NQ - 1 (the next in order; their lanes side by side) -> stage ist
  auto issue = [&](int k) {
    if constexpr (ROWS) return issue_rows(k);
    if ((k & 31) == 0) load_batch(k);
    const int i = lane - (k & 31);
    if ((unsigned)i < (unsigned)NQ) {
      const uint32_t bar = bar0 + ist * 8, dst = ring + ist * T::kStage + i * T::kPair;
      const uint32_t meta = meta0 + (ist * NQ + i) * 16;
      if (t_page >= 0) {
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(meta + 8), "r"(t_span), "r"(t_r0) : "memory");
        const float* ks = p.scales + (size_t)(t_page * 2 * p.H_kv + hk) * p.n_sb + ((t_row * p.sb_mul) >> 20);
        cp_async_scale(meta, ks);
        cp_async_scale(meta + 4, ks + (size_t)p.H_kv * p.n_sb);
        mbar_arrive_cp_async(bar);
        mbar_arrive_expect_tx(bar, T::kPair);
        tma_load_tile(dst, &tm, t_row, hk, t_page, bar);
      } else {  // no attended row, zero scales
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(meta), "r"(0) : "memory");
        mbar_arrive(bar);
        mbar_arrive(bar);
      }
    }
    ist = ist + 1 == NST ? 0 : ist + 1;
  };

  if (!waited) {  // pages and scales may still be written by the previous kernel until here
    pdl_wait();
    pdl_release();
    waited = true;
  }
  [[maybe_unused]] const int r_first = n_a ? a_lo : b_lo - pcs.shift;  // attended index of the share's first row
  // tiles are computed NQ at a time: the last few may be empty ones
  int k_issued = 0, k_end = dead ? 0 : (n_tiles + NQ - 1) / NQ * NQ;
#pragma unroll 1
  for (; k_issued < min(NST * NQ, k_end); k_issued += NQ) issue(k_issued);

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

  // NQ tiles from the ring: their chains of loads, products and exponentials are independent and
  // overlap in the warp, and share the vote and the rescale
  __syncwarp();  // (what the issuing lanes wrote beside their copies)
#pragma unroll 1
  for (int k = 0; k < k_end; k += NQ) {
    const bool ok = mbar_wait(bar0 + cst * 8, cph, dead ? 1024u : kWaitPolls);
    const uint8_t* const stage = my_ring + cst * T::kStage;
    float4 meta[NQ];  // K scale, V scale, attended rows [lo, hi) (bits 0-7, 8-15), first row's index
    float qacc[NQ][2][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if constexpr (!ROWS) meta[i] = s_meta[warp][cst][i];
      const uint8_t* kt_base = stage + i * T::kPair;
      // -------------------------------------------------------------- S^T = C Q^T
      uint4 ka[2][KCH];
#pragma unroll
      for (int c = 0; c < KCH; ++c) {
        ka[0][c] = *reinterpret_cast<const uint4*>(kt_base + koff[c]);
        ka[1][c] = *reinterpret_cast<const uint4*>(kt_base + 8 * D + koff[c]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) qacc[i][c][0] = qacc[i][c][1] = qacc[i][c][2] = qacc[i][c][3] = 0.f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        uint32_t a[4];
        codes_to_f16<CT>(comp(ka[0][kt >> 2], kt & 3), a[0], a[2]);
        codes_to_f16<CT>(comp(ka[1][kt >> 2], kt & 3), a[1], a[3]);
        Mma<__half>::run(qacc[i][kt & 1], a, qf[kt][0], qf[kt][1]);
      }
    }
    // V rows vr[0], vr[1], vr[0] + 8, vr[1] + 8: bytes RL g_id .. + RL - 1
    uint32_t va[NQ][4][RL / 4];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* src = stage + i * T::kPair + T::kBytes + (j >> 1) * 8 * D + voff[j & 1];
        if constexpr (RL == 16) {
          const uint4 v = *reinterpret_cast<const uint4*>(src);
          va[i][j][0] = v.x;
          va[i][j][1] = v.y;
          va[i][j][2] = v.z;
          va[i][j][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(src);
          va[i][j][0] = v.x;
          va[i][j][1] = v.y;
        }
      }
    // ---------------------------------------------------------------- online softmax (log2)
    float sc[NQ][4];
    float2 vsc[NQ];  // V scales of rows kr and kr + 8
    float t0 = -INFINITY, t1 = -INFINITY, u0 = -INFINITY, u1 = -INFINITY;  // maxima of s, s + log2 vs
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float ka, kb;
      bool full;
      unsigned rows;  // bit r: row r counts
      if constexpr (ROWS) {
        const float2 sa = s_rowsc[warp][cst][16 * i + kr], sb = s_rowsc[warp][cst][16 * i + kr + 8];
        ka = nan_if_inf(sa.x);
        kb = nan_if_inf(sb.x);
        vsc[i] = make_float2(nan_if_inf(sa.y), nan_if_inf(sb.y));
        rows = (s_rowok[warp][cst][i >> 1] >> (16 * (i & 1))) & 0xffffu;
        full = rows == 0xffffu;
      } else {
        ka = kb = nan_if_inf(meta[i].x);
        const float vs = nan_if_inf(meta[i].y);
        vsc[i] = make_float2(vs, vs);
        const int span = __float_as_int(meta[i].z);
        full = span == (16 << 8);
        rows = ((1u << (span >> 8)) - 1) & ~((1u << (span & 0xff)) - 1);
      }
      sc[i][0] = (qacc[i][0][0] + qacc[i][1][0]) * (cs0 * ka);  // row kr, columns 2 q4, 2 q4 + 1
      sc[i][1] = (qacc[i][0][1] + qacc[i][1][1]) * (cs1 * ka);
      sc[i][2] = (qacc[i][0][2] + qacc[i][1][2]) * (cs0 * kb);  // row kr + 8
      sc[i][3] = (qacc[i][0][3] + qacc[i][1][3]) * (cs1 * kb);
      if (!full) {  // (warp-uniform)
        if (!((rows >> kr) & 1)) sc[i][0] = sc[i][1] = -INFINITY;
        if (!((rows >> (kr + 8)) & 1)) sc[i][2] = sc[i][3] = -INFINITY;
        // rows outside may hold any code (e4m3 NaN): their V bytes are zeroed
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!((rows >> (vr[j & 1] + 8 * (j >> 1))) & 1)) {
#pragma unroll
            for (int k = 0; k < RL / 4; ++k) va[i][j][k] = 0u;
          }
        }
      }
      if constexpr (MQ) {  // causal among the new tokens
        const int r0 = (ROWS ? r_first + (k + i) * 16 : __float_as_int(meta[i].w)) + kr;
        if (r0 >= lim0) sc[i][0] = -INFINITY;
        if (r0 >= lim1) sc[i][1] = -INFINITY;
        if (r0 + 8 >= lim0) sc[i][2] = -INFINITY;
        if (r0 + 8 >= lim1) sc[i][3] = -INFINITY;
      }
      const float la = __log2f(vsc[i].x), lb = ROWS ? __log2f(vsc[i].y) : la;
      t0 = fmaxf(t0, fmaxf(sc[i][0], sc[i][2]));
      t1 = fmaxf(t1, fmaxf(sc[i][1], sc[i][3]));
      u0 = fmaxf(u0, fmaxf(sc[i][0] + la, sc[i][2] + lb));
      u1 = fmaxf(u1, fmaxf(sc[i][1] + la, sc[i][3] + lb));
    }
    const float over = fmaxf(fmaxf(t0 - st_m[0], t1 - st_m[1]), fmaxf(u0 - st_n[0], u1 - st_n[1]));
    if (__any_sync(0xffffffffu, over > kLazyMaxBs || !ok)) {
      if (__any_sync(0xffffffffu, !ok)) {
        dead = true;  // the tiles in flight are still waited for; the error word says the rest
        k_end = k_issued;
        if (lane == 0) set_error(p.err, kErrTimeout);
      }
      const float mn0 = fmaxf(st_m[0], max_over_groups(t0)), mn1 = fmaxf(st_m[1], max_over_groups(t1));
      st_d[0] *= fast_exp2(st_m[0] - mn0);
      st_d[1] *= fast_exp2(st_m[1] - mn1);
      st_m[0] = mn0;
      st_m[1] = mn1;
      const float nn0 = fmaxf(st_n[0], max_over_groups(u0)), nn1 = fmaxf(st_n[1], max_over_groups(u1));
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
    // weights of P.V: 2^(s - n) vs = p 2^(m - n) vs (the exponent is capped so that a zero scale
    // stays zero, and 2^(m - n) vs at the largest float so that a p of zero gives zero: it is above
    // that only where p is under 2^-119).  Of several queries one that does not attend a row weighs
    // it 0 whatever the scale; a weight of an attended row that underflowed still takes a NaN scale.
    // (ROWS: a row that does not count has scales of 0.)
    const float g0 = fast_exp2(fminf(st_m[0] - st_n[0], 126.f)), g1 = fast_exp2(fminf(st_m[1] - st_n[1], 126.f));
    uint32_t pb[NQ][2];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float pr[4];
      pr[0] = fast_exp2(sc[i][0] - st_m[0]);
      pr[1] = fast_exp2(sc[i][1] - st_m[1]);
      pr[2] = fast_exp2(sc[i][2] - st_m[0]);
      pr[3] = fast_exp2(sc[i][3] - st_m[1]);
      st_d[0] += pr[0] + pr[2];
      st_d[1] += pr[1] + pr[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = pr[e] * min_nan((e & 1 ? g1 : g0) * (e < 2 ? vsc[i].x : vsc[i].y), FLT_MAX);
        pr[e] = MQ && sc[i][e] == -INFINITY ? 0.f : w;
      }
      // P^T as a B fragment: fragment rows 2q, 2q + 1 | 2q + 8, 2q + 9 of column g_id
      const uint32_t x0 = pack2<__half>(pr[0], pr[2]);  // column 2q: rows of g_id, g_id + 8
      const uint32_t x1 = pack2<__half>(pr[1], pr[3]);  // column 2q + 1
      const int srcA = 8 * q4 + (g_id >> 1), srcB = srcA + 4;
      const uint32_t a0 = __shfl_sync(0xffffffffu, x0, srcA);
      const uint32_t a1 = __shfl_sync(0xffffffffu, x1, srcA);
      const uint32_t b0 = __shfl_sync(0xffffffffu, x0, srcB);
      const uint32_t b1 = __shfl_sync(0xffffffffu, x1, srcB);
      const uint32_t wa = (g_id & 1) ? a1 : a0, wb = (g_id & 1) ? b1 : b0;
      pb[i][0] = __byte_perm(wa, wb, 0x5410);
      pb[i][1] = __byte_perm(wa, wb, 0x7632);
    }
    // ---------------------------------------------------------------- O^T += V^T P^T
    // m-tile mt: rows g_id / g_id + 8 are dims RL g_id + 2 mt / + 1
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) {
      const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        uint32_t a[4];
        codes_to_f16<CT>(__byte_perm(va[i][0][mt >> 1], va[i][1][mt >> 1], sel), a[0], a[1]);
        codes_to_f16<CT>(__byte_perm(va[i][2][mt >> 1], va[i][3][mt >> 1], sel), a[2], a[3]);
        Mma<__half>::run(oacc[mt], a, pb[i][0], pb[i][1]);
      }
    }
    // every lane has its codes in registers: the stage takes the next tiles
    cst = cst + 1 == NST ? 0 : cst + 1;
    if (cst == 0) cph ^= 1;
    __syncwarp();
    if (k_issued < k_end) {
      issue(k_issued);
      k_issued += NQ;
    }
  }
  st_d[0] = sum_over_groups(st_d[0]);
  st_d[1] = sum_over_groups(st_d[1]);

  // ---------------------------------------------------------------- finish the segment
  // This thread holds columns 2 q4 (o0, o2) and 2 q4 + 1 (o1, o3), dims RL g_id .. + RL - 1.
  // A segment within the range goes to out/lse; else its state (O / d, lse) waits in shared
  // memory for the block's other warps.
  const bool whole = (ua == 0 && ub == sg.n);
  const int side = sg.off <= ws.x0 ? 0 : 1;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int j = 2 * q4 + hh;
    if (j < hcount) {
      const bool empty = st_d[hh] == 0.f;
      float inv = empty ? 0.f : fast_exp2(st_n[hh] - st_m[hh]) / st_d[hh];
      float l = empty ? kEmptyM : st_m[hh] + log2f(st_d[hh]);
      const size_t row = col_row<MQ>(p, sg.b, hk, c0 + j);
      if (whole && p.sink) {
        const SinkAdj sa = apply_sink(p, col_head<MQ>(p, hk, c0 + j), l);
        inv *= sa.scale;
        l = sa.lse;
      }
#pragma unroll
      for (int o = 0; o < RL / 4; ++o) {
        const float4 v = make_float4(oacc[2 * o][hh] * inv, oacc[2 * o][hh + 2] * inv,
                                     oacc[2 * o + 1][hh] * inv, oacc[2 * o + 1][hh + 2] * inv);
        if (whole) store_four(p, row * D + RL * g_id + 4 * o, v);
        else reinterpret_cast<float4*>(state_of(warp, side) + j * D + RL * g_id)[o] = v;
      }
      if (g_id == 0) {
        if (whole) p.lse[row] = l;
        else s_plse[warp][side][j] = l;
      }
    }
  }
  if (!whole && lane == 0) s_part[warp][side] = PartEntry{sg.off, sg.b, sg.hz, ub - ua, sg.n, hk, c0, hcount};
  }  // ua < ub
  if (sg.off + C + sg.n >= cx1 || !next_segment(p, sg, C)) break;
  }  // segments
  if (!waited) pdl_wait();  // (a worker without units: the block's partials still follow it)

  // ---------------------------------------------------------------- partial states
  // A segment's states within the block are merged first (lse = M + log2 sum 2^(lse_s - M), out =
  // sum 2^(lse_s - M) o_s / sum 2^(lse_s - M)).  If the block holds all of its units that is the
  // result; else the block publishes one state and adds its units to the segment's counter, and
  // the block that completes the count merges the blocks' states.  So a segment split over the
  // four warps of a block never leaves it, and one over several blocks costs a state per block.
  if (!__syncthreads_or(lane < 2 && s_part[warp][lane].b >= 0)) return;
  // lane k < 2 NW of every warp holds entry k; `same`: the entries of its segment
  const PartEntry mine_e = s_part[(lane >> 1) % NW][lane & 1];
  const bool held = lane < 2 * NW && mine_e.b >= 0;
  unsigned same_l = 0;
  int units = 0;  // of its segment in the block
  const int key_b = held ? mine_e.b : -1;  // (a match instruction takes a turn per distinct value)
#pragma unroll
  for (int k = 0; k < 2 * NW; ++k) {
    const int b = __shfl_sync(0xffffffffu, key_b, k), hz = __shfl_sync(0xffffffffu, mine_e.hz, k);
    const int x = __shfl_sync(0xffffffffu, mine_e.mine, k);
    if (b >= 0 && b == key_b && hz == mine_e.hz) {
      same_l |= 1u << k;
      units += x;
    }
  }
  const unsigned leaders = __ballot_sync(0xffffffffu, held && (same_l & ((1u << lane) - 1)) == 0);
  const unsigned whole_l = __ballot_sync(0xffffffffu, held && units == mine_e.n);
  const long long U = s_start[0].U, G = gridDim.x;
  // one output (final) or one state in slot `to`: four dims from `acc`, unnormalised, of a column
  auto put = [&](const PartEntry& e, int j, int d, float M, float den, float4 acc, bool final, long long to) {
    const bool empty = den == 0.f;
    float inv = empty ? 0.f : 1.f / den;
    float l = empty ? kEmptyM : M + log2f(den);
    if (final && p.sink) {
      const SinkAdj sa = apply_sink(p, col_head<MQ>(p, e.hk, e.c0 + j), l);
      inv *= sa.scale;
      l = sa.lse;
    }
    const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (final) {
      const size_t row = col_row<MQ>(p, e.b, e.hk, e.c0 + j);
      store_four(p, row * D + d, v);
      if (d == 0) p.lse[row] = l;
    } else {
      *reinterpret_cast<float4*>(p.part_o + (to * kMaxGroupPerCta + j) * D + d) = v;
      if (d == 0) p.part_lse[to * kMaxGroupPerCta + j] = l;
    }
  };
  auto weighted = [](float4& acc, float w, float4 o) {
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
  };
  // Slots of block c, for slice z of a segment: two per block and slice, for the segment that the
  // block's range starts in (or at) and the one that it ends in.
  auto slot_of = [&](long long c, bool ends_in, int hz) {
    return (2 * c + ends_in) * zg + (zg > 1 ? hz % zg : 0);
  };
#pragma unroll 1
  for (unsigned m = leaders; m; m &= m - 1) {
    const int L = __ffs(m) - 1;
    const PartEntry e = s_part[L >> 1][L & 1];
    unsigned rest = __shfl_sync(0xffffffffu, same_l, L);
    int id[NW];  // the segment's states: at most one per warp
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      id[i] = rest ? __ffs(rest) - 1 : -1;
      rest &= rest - 1;
    }
    const bool all = (whole_l >> L) & 1;
    const long long to = all ? 0 : slot_of(blockIdx.x, e.off > s_start[0].x0, e.hz);  // (x0: the block's)
#pragma unroll 1
    for (int it = threadIdx.x; it < e.hcount * (D / 4); it += NT) {
      const int j = it / (D / 4), d = it % (D / 4) * 4;
      float l[NW], M = kEmptyM, den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        l[i] = id[i] >= 0 ? s_plse[id[i] >> 1][id[i] & 1][j] : kEmptyM;
        M = fmaxf(M, l[i]);
      }
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        if (l[i] <= kEmptyM) continue;  // (NaN counts)
        const float w = fast_exp2(l[i] - M);
        den += w;
        weighted(acc, w, *reinterpret_cast<const float4*>(state_of(id[i] >> 1, id[i] & 1) + j * D + d));
      }
      put(e, j, d, M, den, acc, all, to);
    }
  }
  const unsigned open = leaders & ~whole_l;
  if (!open) return;
  fence_acq_rel_gpu();
  __syncthreads();
  if (warp == 0 && (open >> lane) & 1) {
    int* cnt = p.counters + (size_t)mine_e.b * p.H_kv * p.n_z + mine_e.hz;
    const int prev = atomicAdd(cnt, units);
    s_last[lane] = prev + units == mine_e.n;
    if (s_last[lane]) *cnt = 0;  // every other block's units have arrived: reset for reuse
  }
  __syncthreads();
#pragma unroll 1
  for (unsigned m = open; m; m &= m - 1) {
    const int L = __ffs(m) - 1;
    if (!s_last[L]) continue;
    fence_acq_rel_gpu();
    const PartEntry e = s_part[L >> 1][L & 1];
    const long long first = share_of(e.off + C, U, G);
    const int ns = (int)(share_of(e.off + C + e.n - 1, U, G) - first + 1);
    // state i: block first + i's; only the first can hold the segment as the one it ends in.  With
    // fewer positions than blocks some blocks between have no units and wrote nothing.
    const bool ends_in = e.off > div_floor(first * U, G);
    auto slot_at = [&](int i) { return slot_of(first + i, i == 0 && ends_in, e.hz); };
    auto holds = [&](int i) {
      return U >= G || div_floor((first + i) * U, G) < div_floor((first + i + 1) * U, G);
    };
#pragma unroll 1
    for (int it = threadIdx.x; it < e.hcount * (D / 4); it += NT) {
      const int j = it / (D / 4), d = it % (D / 4) * 4;
      float M = kEmptyM, den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int i0 = 0; i0 < ns; i0 += 8) {  // eight states' lse and rows in flight together
        float l[8], m8 = M;
        float4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const long long sl = slot_at(min(i0 + i, ns - 1)) * kMaxGroupPerCta + j;
          l[i] = __ldcg(p.part_lse + sl);
          o[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + sl * D + d));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i0 + i >= ns || !holds(i0 + i)) l[i] = kEmptyM;
          m8 = fmaxf(m8, l[i]);
        }
        const float f = fast_exp2(M - m8);
        M = m8;
        den *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (l[i] <= kEmptyM) continue;
          const float w = fast_exp2(l[i] - M);
          den += w;
          weighted(acc, w, o[i]);
        }
      }
      put(e, j, d, M, den, acc, true, 0);
    }
  }
}

// ----------------------------------------------------------------------------- launch
template <typename CT, typename QT, int D, bool MQ, bool ROWS>
static cudaError_t launch_bs_t(const DecodeParams& p, const CUtensorMap& tm, dim3 grid,
                               cudaStream_t st, MmaConfig* cfg) {
  constexpr int NW = kMmaWarps;
  constexpr int dyn = bs_smem_bytes<D, NW>();
  auto kern = decode_bs_kernel<CT, QT, D, MQ, ROWS, NW>;
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

template <typename CT, bool ROWS>
static cudaError_t launch_bs_any(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                                 cudaStream_t st, MmaConfig* cfg) {
  const bool mq = p.q_len > 1;
  auto with_q = [&](auto q_tag) -> cudaError_t {
    using QT = decltype(q_tag);
    if (p.D == 128)
      return mq ? launch_bs_t<CT, QT, 128, true, ROWS>(p, tm, grid, st, cfg)
                : launch_bs_t<CT, QT, 128, false, ROWS>(p, tm, grid, st, cfg);
    if (p.D == 64)
      return mq ? launch_bs_t<CT, QT, 64, true, ROWS>(p, tm, grid, st, cfg)
                : launch_bs_t<CT, QT, 64, false, ROWS>(p, tm, grid, st, cfg);
    return cudaErrorInvalidValue;
  };
  if (q_dtype == kBF16) return with_q(__nv_bfloat16{});
  if (q_dtype == kF16) return with_q(__half{});
  return cudaErrorInvalidValue;
}

}  // namespace pd
