// Tensor-core decode of a 4-bit KV cache: e2m1 codes, two dims a byte, with a scale per row and block
// of SB dims: e4m3 (SB 16) or a power of two, e8m0 (SB 32).
//
//   K_rd = c_rd ks_r,d/SB k_scale,  s_r = sm_scale log2(e) q.K_r,  out = sum_r 2^(s_r) V_r / sum_r 2^(s_r)
//
// The work split and the schedule are those of the other tensor-core decodes (decode_common.cuh): every
// warp is an independent worker on its share of the pages; shares of a segment are merged by its block
// (decode_parts.cuh).
//
// What bounds it: the codes and scales are 9/16 of a byte per dim (17/32 with power-of-two scales), so
// the copy rate leaves an SM about 98 cycles for a 16-row tile of D 128, K and V; the tile takes about
// 250 instructions, of which 64 turn codes to f16 and 64 multiply the scales in (each on a pipe of half
// rate), 16 bring the codes of two rows of V side by side, 23 copy, 16 are products.  The loop issues 2.4
// instructions a cycle (the schedulers' four warps-slots wait for fixed latencies and those two pipes), so
// it takes 105 cycles; what is measured above that is the start (3 us from the first instruction to the
// first tile), the merge and the launch.  The steps that carried it (256 sequences of 300 to 4200 rows /
// eight contexts of 32K to 128K rows, us): tiles by bulk copies of a lane 163 / 181; by 16-byte
// asynchronous copies of all lanes (a bulk copy takes uniform registers, so lanes took turns) 136 / 141;
// masks and rare paths out of the loop 128 / 137; one block of twelve warps an SM, in which the older
// warps of a scheduler do not run ahead of the younger (three blocks of four: 128 / 137; sixteen warps of
// 128 registers: 121 / 145) and merges by the whole block at the end 117 / 130; power-of-two scales two at
// a time 117 / 127; weights of two columns an instruction, nothing of a segment's end worked out before its loop
// 117 / 123.  The copies alone take 97 us and 94 us.
//   Measured on one GB300 (of the 6791 GB/s copy rate): 256 sequences, 64 heads, e4m3 scales 117 us (82 %),
// eight long contexts, power-of-two scales 123 us (81 %), 32 sequences of 512 to 4096 rows 21.9 us (48 %),
// 24 sequences with four queries, D 64 18.9 us (36 %), one of 300 rows 6.5 us (launch and latency); seven short
// ones with F32 Q, D 256, in pages of 20 rows 17.2 us (13 %: bound by its start and its few warps).  256
// sequences in other forms: bf16 D 256 217 us (88 %; its rows gathered one by one 257), F32 Q 164 us (59 %;
// gathered 186; each product twice), pages of 20 rows 144 us.
//
// Arithmetic (mma.sync m16n8k16, fp32 accumulation: at most 8 query columns share a KV head's tile, an
// eighth of the rows of a tcgen05 tile, whose 4-bit products would want Q in 4 bits too and cannot scale
// single rows of V):
//   - a code times its scale has at most 6 significant bits and is exact in f16.
//   - Q is scaled per column by a power of two into the upper f16 range: a bf16 or f16 value keeps all
//     its bits unless it is below 2^-28 of the column's largest.  F32 Q goes as hi + lo (22 bits).
//   - the denominator is held in fp32; the weights of P.V go to f16 once, times 2^7 against a lazy running
//     maximum (F32 Q: hi + lo): the largest lies between 2^7 and 2^15.  They are taken from differences to the
//     maximum, and partial states carry the maximum, so that only those differences matter, at any size.
//   - the products' own sum is cut off towards zero: it holds at most kSumTiles tiles (F32 Q: one), and such
//     sums are added by rounded additions.
//   - rows that do not count get scores of -inf and zero scales of V; a NaN scale of a row that counts
//     makes NaN what attends it.
#pragma once

#include <cfloat>

#include "decode_mma.cuh"
#include "decode_parts.cuh"

namespace pd {

constexpr float kLazyMaxMx = 8.f;   // the running maximum moves when exceeded by more than 2^8 ...
constexpr float kWeightUp = 7.f, kWeightDown = 0x1p-7f;  // ... and a weight is held times 2^7: at most 2^15 in f16
// How many stages ahead of another warp of its scheduler a warp lets it catch up, and for how long (ns);
// 3 to 12 stages and 200 to 1000 ns measure the same.
constexpr int kLead = 6, kNap = 500;

// ----------------------------------------------------------------------------- geometry
template <int SB, int D, bool ROWS>
struct MxTile {
  static constexpr int RB = D / 2;                  // code bytes per row
  static constexpr int NB = D / SB;                 // scale bytes per row
  static constexpr int SR = ROWS && NB < 4 ? 4 : NB;  // of a row in shared memory (ROWS: whole words are copied)
  static constexpr int KT = D / 16;                 // k-tiles of QK, m-tiles of PV
  static constexpr int KB = D == 64 ? 8 : 16;       // K bytes a thread reads at once
  static constexpr int KCH = RB / (4 * KB);         // times per row
  static constexpr int VB = RB / 8;                 // V bytes per row and thread
  static constexpr int RL = D / 8;                  // V dims per row and thread
  static constexpr int kCodes = 16 * RB;            // one tile of K (or V) codes
  static constexpr int kScales = 16 * SR;           // and of its scales
  static constexpr int kPair = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
  static constexpr int NQ = D == 64 ? 4 : 2;        // tiles computed together
  static constexpr int NST = 2;                     // ring stages per warp, of NQ tiles each
  static constexpr int kStage = NQ * kPair;
  static constexpr int kState = kMaxGroupPerCta * D * 4;  // a partial state's outputs, fp32
  static constexpr int kRing = (NST * kStage > kState ? NST * kStage : kState);
  static_assert(D == 64 || D == 128 || D == 256, "head dim");
};
template <int SB, int D, bool ROWS, int NW>
constexpr int mx_smem_bytes() { return NW * (MxTile<SB, D, ROWS>::kRing + MxTile<SB, D, ROWS>::kState) + 128; }

// 16-bit Q: tiles whose products are summed in the accumulators, which cut every sum off (by 5e-8 of it a tile).
// Such sums are added, rounded to nearest, in local memory: the cutting adds up to 6e-6, however long the share.
// (64 tiles at a time would be 2e-6, but cost D 256 10 %: the local memory has left L2 when it is next touched.)
constexpr int kSumTiles = 256;

// Row of the tile that fragment row g (0..7; g + 8: the row + 8) holds, and byte offset of the 16-byte
// chunk c of row r of a tile in shared memory.  Chosen so that the rows of K that one phase of lanes
// reads (those of g = 2i, 2i + 1; D 64: of four g), and the rows of V that the quad lanes read (those
// of g = 0, 2, 4, 6, or of 1, 3, 5, 7), fall on different banks.
template <int D>
__device__ __forceinline__ int mx_row(int g) {
  constexpr uint32_t order = D == 64 ? 0x53427160u : D == 128 ? 0x65217430u : 0x36147250u;
  return (order >> (4 * g)) & 7;
}
template <int D>
__device__ __forceinline__ int mx_chunk(int r, int c) {
  return r * (D / 2) + ((D == 64 ? c : D == 128 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4);
}

// Two scales as f16.
template <int SB>
__device__ __forceinline__ uint32_t mx_scales(uint32_t a, uint32_t b) {
  if constexpr (SB == 16) return e4m3x2_to_f16x2((uint16_t)(a | (b << 8)));
  // 2^(x - 127): exponent x - 112 for 2^-14 to 2^13, 0 below; above, where a code times it would
  // overflow, NaN (141 has 29 in the exponent: 0x7400 + 0xbff).  On both halves at once.
  const uint32_t x = __vminu2(__vmaxu2(a | (b << 16), 0x00700070u), 0x008d008du);
  constexpr uint32_t c = (112u * 1024u + 140u * 0xbffu) * 0x10001u;
  return x * 1024u + __vmaxu2(x, 0x008c008cu) * 0xbffu - c;
}

// eight codes (four bytes) -> f16x2 of each byte, exact
__device__ __forceinline__ void mx_codes(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// f16 times one half of a pair
__device__ __forceinline__ uint32_t mul_lo(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_hi(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// (x + n) c + w of two columns side by side, each step rounded as alone
__device__ __forceinline__ float2 scaled_sums(float x0, float x1, float2 n, float2 c, float w) {
  float2 r;
  asm("{\n .reg .b64 x, n, c, w;\n mov.b64 x, {%2, %3};\n mov.b64 n, {%4, %5};\n mov.b64 c, {%6, %7};\n mov.b64 w, {%8, %8};\n"
      " add.rn.f32x2 x, x, n;\n fma.rn.f32x2 x, x, c, w;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x0), "f"(x1), "f"(n.x), "f"(n.y), "f"(c.x), "f"(c.y), "f"(w));
  return r;
}
__device__ __forceinline__ const uint8_t* shfl_ptr(const uint8_t* x, int from) {
  return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x), from));
}
// 8x8 transpose of 16-bit elements across the warp: from row lane / 4, columns 2 (lane % 4) + {0, 1}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <int N>
__device__ __forceinline__ void cp_async_n(uint32_t dst, const uint8_t* src) {
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but this thread's N most recent groups of copies have landed.
template <int N>
__device__ __forceinline__ void cp_async_group_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
template <int N>  // N bytes of shared memory as words
__device__ __forceinline__ void lds_words(const uint8_t* src, uint32_t (&w)[N / 4]) {
  if constexpr (N == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

// ----------------------------------------------------------------------------- kernel
// SPLIT: F32 Q; Q and the weights then go as a sum of two f16 parts, each product twice.  Else Q is
// F16 or BF16 (p.q_bf16).
// ROWS: tiles of 16 consecutive attended rows of any pages, gathered row by row; else tiles are 16
// rows of one page (page size a multiple of 16), copied whole.
template <int SB, bool SPLIT, int D, bool MQ, bool ROWS, int NW, int BLOCKS>
__global__ void __launch_bounds__(NW * 32, BLOCKS) decode_mx_kernel(const __grid_constant__ DecodeParams p) {
  using T = MxTile<SB, D, ROWS>;
  constexpr int NT = NW * 32;
  constexpr int KT = T::KT, KCH = T::KCH, KB = T::KB, VB = T::VB, RL = T::RL, NQ = T::NQ, NST = T::NST;
  constexpr int RB = T::RB, NB = T::NB, SR = T::SR;
  constexpr int KW = KB / 4;  // words
  extern __shared__ uint8_t s_raw[];
  // of each warp's partial states (first, last segment), by column: maximum and sum, factor
  __shared__ float2 s_pmd[NW][2][kMaxGroupPerCta];
  __shared__ float s_pcs[NW][2][kMaxGroupPerCta];
  __shared__ SegmentMerge s_merge[NW + 4];
  __shared__ int s_n_merge, s_done[NW];             // s_done: stages each warp has computed
  __shared__ WorkerStart s_start[NW];
  // of each tile of two batches of 32 (ROWS: of a stage): which rows count (bit r: row r), and the
  // attended index of row 0; of rows with two scale bytes that were copied one by one, which half of
  // the copied word holds K's and V's
  constexpr int NM = ROWS ? NQ : 32;
  __shared__ __align__(8) uint16_t s_rows[NW][2][NM];
  __shared__ int s_r0[MQ ? NW : 1][2][NM];
  __shared__ uint16_t s_half[ROWS && NB < 4 ? NW : 1][2][NST][NQ];
  constexpr int NH = NQ / 2;  // pairs of tiles

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* const rings = s_raw + (((smem_u32(s_raw) + 127u) & ~127u) - smem_u32(s_raw));
  uint8_t* const my_ring = rings + warp * T::kRing;
  const uint32_t ring = smem_u32(my_ring);
  // the rings' space before the first fill: scratch of the start-up scan; after a warp's last
  // tile, its part: the state of its last segment
  static_assert(NW * T::kRing >= (NT + 1) * 8, "scratch");
  auto state_of = [&](int w, int side) -> float* {
    return reinterpret_cast<float*>(side ? rings + w * T::kRing : rings + NW * T::kRing + w * T::kState);
  };
  if (threadIdx.x == 0) {
    prefetch_l2_share(p.Q, (size_t)p.B * p.q_len * p.H_qo * D * (SPLIT ? 4 : 2), blockIdx.x, gridDim.x);
    if (p.values) prefetch_l2_share(p.values, (size_t)p.nnz_pages * sizeof(int32_t), blockIdx.x, gridDim.x);
  }
  // With a host plan the start-up reads launch parameters alone and runs under the tail of the
  // kernel before; otherwise, as everywhere, nothing of the caller's is read before it completes.
  bool waited = false;
  if (!p.early_inputs && !p.hp_B) {
    pdl_wait();
    pdl_release();
    waited = true;
  }
  line_starts<NT, NW>(p, s_start, reinterpret_cast<long long*>(rings));
  if (lane == 0) s_done[warp] = 0;
  if (threadIdx.x == 0) s_n_merge = 0;
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

  // this thread's fragment rows (+ 8: the second half), and the byte offsets of what it reads of them
  const int kr = mx_row<D>(g_id);
  const int vr[2] = {mx_row<D>(2 * q4), mx_row<D>(2 * q4 + 1)};
  int koff[KCH], voff[2];
#pragma unroll
  for (int c = 0; c < KCH; ++c) {
    const int x = KB * (4 * c + q4);
    koff[c] = mx_chunk<D>(kr, x >> 4) + (x & 15);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) voff[j] = T::kCodes + mx_chunk<D>(vr[j], VB * g_id >> 4) + (VB * g_id & 15);

  // Where this lane's chunk of a tile's codes goes, and of its scales which tile it copies, from where
  // (V's lie behind K's as its codes do) and to where; CS: chunks of a tile's K (or V) scales
  constexpr int CS = T::kScales / 16, TPC = CS < 16 ? 16 / CS : 1;  // (TPC: tiles whose scales go at once)
  static_assert(ROWS || (CS <= 16 && (NQ <= TPC || NQ % TPC == 0) && T::kCodes % 512 == 0), "a warp's copies");
  [[maybe_unused]] const int my_chunk = mx_chunk<D>(16 * lane / RB, 16 * lane % RB / 16);
  [[maybe_unused]] const int my_stile = lane / (2 * CS) % (NQ < TPC ? NQ : TPC);
  [[maybe_unused]] const int my_sdst = my_stile * T::kPair + 2 * T::kCodes + 16 * (lane % (2 * CS));
  [[maybe_unused]] const long long v_codes = (long long)p.H_kv * P * RB;
  [[maybe_unused]] const long long my_sbyte =
      lane % (2 * CS) < CS ? 16 * (lane % CS) : (long long)p.H_kv * P * NB + 16 * (lane % CS);

  // The ring: NQ tiles at a time are computed from stage `cst`, which then takes the ones that follow
  // the other stage's; one group of copies a stage.
  static_assert(NST == 2 && NST * NQ <= 16, "two stages, well within a batch of 32 tiles");
  int cst = 0, stages = 0;
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

  // Raw Q of column g_id at this lane's B-fragment dims (2 KB of them from 2 KB (4 c + q4)), loaded first
  const bool have_q = g_id < hcount;
  constexpr int QV = SPLIT ? KB / 2 : KB / 4;  // 16-byte loads per chunk
  uint4 qraw[KCH][QV];
  {
    constexpr int QB = SPLIT ? 4 : 2;
    const uint8_t* qrow = reinterpret_cast<const uint8_t*>(p.Q) +
                          col_row<MQ>(p, sg.b, hk, c0 + (have_q ? g_id : 0)) * (D * QB);
#pragma unroll
    for (int c = 0; c < KCH; ++c)
#pragma unroll
      for (int i = 0; i < QV; ++i)
        qraw[c][i] = have_q ? __ldg(reinterpret_cast<const uint4*>(qrow + 2 * KB * QB * (4 * c + q4)) + i)
                            : make_uint4(0u, 0u, 0u, 0u);
  }
  int lim0 = 0, lim1 = 0, lim_all = INT_MAX;  // attended-row limits of this lane's score columns, and the least
  if constexpr (MQ) {
    const int cc = c0 + 2 * q4;
    lim_all = sg.seq.L - p.q_len + 1;
    lim0 = lim_all + cc / p.group;
    lim1 = lim_all + (cc + 1) / p.group;
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
  [[maybe_unused]] const int r_first = n_a ? a_lo : b_lo - pcs.shift;  // attended index of the share's first row
  auto tile_at = [&](int k) { return k < n_a ? ((a_lo >> 4) + k) << 4 : ((b_lo >> 4) + k - n_a) << 4; };  // offset
  auto load_page = [&](int k) -> int {  // page id of tile k, unchecked; -1 out of the table
    if (k >= n_tiles) return -1;
    const int pidx = tile_at(k) / P;
    return pidx < sg.seq.npages && (long long)sg.seq.page_begin + pidx < p.nnz_pages
               ? __ldg(p.values + sg.seq.page_begin + pidx) : -1;
  };
  // of this lane's tile: its K codes and scales; of the batch: tiles of which every row counts for every
  // column
  const uint8_t* t_codes = nullptr;
  const uint8_t* t_scales = nullptr;
  int page_next = ROWS ? -1 : load_page(lane);
  unsigned full = 0;
  auto load_batch = [&](int k0) {  // tiles k0 .. k0 + 31
    const int k = k0 + lane, page = page_next;
    page_next = load_page(k + 32);
    const int o = tile_at(k);
    const bool in_a = k < n_a;
    auto below = [&](int end) { return (1 << min(max(end - o, 0), 16)) - 1; };  // the tile's rows before it
    int rows = below(in_a ? a_hi : b_hi) & ~below(in_a ? a_lo : b_lo);
    const int r0 = in_a ? o : o - pcs.shift;
    long long row = ((long long)page * 2 * p.H_kv + hk) * P + o % P;
    if (k >= n_tiles || page < 0 || page >= p.max_pages) {  // no such tile, or its rows do not count
      if (k < n_tiles) set_error(p.err, kErrBadPage);
      rows = 0;
      row = 0;  // (what is copied in its place)
    }
    t_codes = reinterpret_cast<const uint8_t*>(p.pages) + row * RB;
    t_scales = p.mx_scales + row * NB;
    s_rows[warp][(k0 >> 5) & 1][lane] = (uint16_t)rows;
    if constexpr (MQ) s_r0[warp][(k0 >> 5) & 1][lane] = r0;
    full = __ballot_sync(0xffffffffu, rows == 0xffff && (!MQ || r0 + 16 <= lim_all));
  };
  // ROWS: the page (unchecked; -1 out of the table) and slot of a lane's rows 32 h + lane of the
  // stage that starts with tile k, loaded one stage ahead
  int rw_page[NH], rw_slot[NH];
  auto load_rows = [&](int k) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
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
  // its rows -> stage st: RB / 16 lanes copy a row's 16-byte chunks, the row's own lane its scales
  auto issue_rows = [&](int k, int st) {
    constexpr int CPR = RB / 16, RPI = 32 / CPR;  // chunks per row, rows per instruction
    const long long to_v = (long long)p.H_kv * P;  // rows
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int page = rw_page[h], slot = rw_slot[h];
      const bool ok = page >= 0 && page < p.max_pages;
      if (slot >= 0 && !ok) set_error(p.err, kErrBadPage);  // its row does not count
      const unsigned rows = __ballot_sync(0xffffffffu, ok);
      const long long row = ((long long)page * 2 * p.H_kv + hk) * P + slot;  // of K
      const uint32_t tile = ring + st * T::kStage + (2 * h + (lane >> 4)) * T::kPair;
      if (lane < 2) {
        s_rows[warp][st][2 * h + lane] = (uint16_t)(rows >> (16 * lane));
        if constexpr (MQ) s_r0[warp][st][2 * h + lane] = r_first + (k + 2 * h + lane) * 16;
      }
      if constexpr (NB < 4) {  // the aligned word that holds the row's two bytes
        const unsigned kh = __ballot_sync(0xffffffffu, ok && (row & 1));
        const unsigned vh = __ballot_sync(0xffffffffu, ok && ((row + to_v) & 1));
        if (lane < 2) {
          s_half[warp][0][st][2 * h + lane] = (uint16_t)(kh >> (16 * lane));
          s_half[warp][1][st][2 * h + lane] = (uint16_t)(vh >> (16 * lane));
        }
      }
      if (ok) {
        const uint32_t dst = tile + 2 * T::kCodes + (lane & 15) * SR;
        const long long kw = NB < 4 ? row >> 1 : row, vw = NB < 4 ? (row + to_v) >> 1 : row + to_v;
        cp_async_n<SR>(dst, p.mx_scales + kw * SR);
        cp_async_n<SR>(dst + T::kScales, p.mx_scales + vw * SR);
      }
#pragma unroll
      for (int it = 0; it < CPR; ++it) {
        const int r = it * RPI + lane / CPR, x = lane % CPR * 16;  // row of the 32, byte of it
        const long long src_row = __shfl_sync(0xffffffffu, row, r);
        if ((rows >> r) & 1) {
          const uint8_t* src = reinterpret_cast<const uint8_t*>(p.pages) + src_row * RB + x;
          const uint32_t dst = ring + st * T::kStage + (2 * h + (r >> 4)) * T::kPair + mx_chunk<D>(r & 15, x >> 4);
          cp_async_chunk(dst, src);
          cp_async_chunk(dst + T::kCodes, src + to_v * RB);
        }
      }
    }
    load_rows(k + NQ);
  };
  // tiles k .. k + NQ - 1 (the next in order; their lanes side by side) -> stage st
  auto issue = [&](int k, int st) {
    if constexpr (ROWS) return issue_rows(k, st);
    if ((k & 31) == 0) load_batch(k);
    const uint32_t to = ring + st * T::kStage;
    const int first = k & 31;
    // codes: a tile's are contiguous, of K and of V, and go a 16-byte chunk a lane at a time
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const uint8_t* src = shfl_ptr(t_codes, first + t) + 16 * lane;
      const uint32_t dst = to + t * T::kPair;
      // (D 256: 512 bytes are four rows, which turn bit 2 of a chunk's place over)
      auto at = [&](int j) { return 512 * j + (D == 256 && (j & 1) ? my_chunk ^ 64 : my_chunk); };
#pragma unroll
      for (int j = 0; j < T::kCodes / 512; ++j) cp_async_chunk(dst + at(j), src + 512 * j);
      src += v_codes;
#pragma unroll
      for (int j = 0; j < T::kCodes / 512; ++j) cp_async_chunk(dst + T::kCodes + at(j), src + 512 * j);
    }
    // scales: of TPC tiles at once
#pragma unroll
    for (int t = 0; t < NQ; t += TPC) {
      const uint8_t* src = shfl_ptr(t_scales, first + t + my_stile) + my_sbyte;
      if (NQ >= TPC || lane < NQ * 2 * CS) cp_async_chunk(to + t * T::kPair + my_sdst, src);
    }
  };

  if (!waited) {  // pages and scales may still be written by the previous kernel until here
    pdl_wait();
    pdl_release();
    waited = true;
  }
  // tiles are computed NQ at a time: the last few may be empty ones
  const int k_end = (n_tiles + NQ - 1) / NQ * NQ;
  int k_issued = 0;
#pragma unroll 1
  for (; k_issued < NST * NQ; k_issued += NQ) {
    if (k_issued < k_end) issue(k_issued, k_issued == 0 ? cst : cst ^ 1);
    cp_async_group();
  }

  // ---------------------------------------------------------------- Q^T B fragments
  // k-tile kt = 2 (KW c + w) + h: dims 2 KB (4 c + q4) + 8 w + 4 h + {0, 1} and + {2, 3} of column g_id,
  // times 2^(14 - e), e the exponent of the column's largest magnitude, and the sign of sm_scale
  uint32_t qf[KT][2];
  [[maybe_unused]] uint32_t ql[SPLIT ? KT : 1][2];
  float cs0, cs1;  // column factors of this lane's score columns: 2^(e - 14) |sm_scale| log2(e) k_scale
  {
    float q[KT][4];  // this lane's four dims of each k-tile
    auto unpack = [&](auto tag) {
      using QT = decltype(tag);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const int c = kt / (2 * KW), i = kt % (2 * KW);
        if constexpr (SPLIT) {
          const uint4 v = qraw[c][i];
          q[kt][0] = __uint_as_float(v.x), q[kt][1] = __uint_as_float(v.y);
          q[kt][2] = __uint_as_float(v.z), q[kt][3] = __uint_as_float(v.w);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 f = unpack2<QT>(comp(qraw[c][i >> 1], 2 * (i & 1) + h));
            q[kt][2 * h] = f.x, q[kt][2 * h + 1] = f.y;
          }
        }
      }
    };
    if (p.q_bf16) unpack(__nv_bfloat16{});
    else unpack(__half{});
    float amax = 0.f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(q[kt][i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^(14 - e) and its inverse, both normal: e is kept in [-100, 126]
    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255) - 127, -100), 126);
    const float up = copysignf(__uint_as_float((unsigned)(127 + 14 - e) << 23), p.score_scale);
    // (at least the least normal float, so that the -inf of a row that does not count stays one, and finite, so
    // that the maximum's difference of 0 does)
    const float cs = fminf(fmaxf(__uint_as_float((unsigned)(127 - 14 + e) << 23) * fabsf(p.score_scale), FLT_MIN), FLT_MAX);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = q[kt][2 * h] * up, y = q[kt][2 * h + 1] * up;
        if constexpr (SPLIT) split2<__half>(x, y, qf[kt][h], ql[kt][h]);
        else qf[kt][h] = pack2<__half>(x, y);
      }
    cs0 = __shfl_sync(0xffffffffu, cs, 8 * q4);      // column 2 q4
    cs1 = __shfl_sync(0xffffffffu, cs, 8 * q4 + 4);  // column 2 q4 + 1
  }

  // The running maxima m are of the products before the column's factor cs (> 0); weights are
  // 2^(cs (s - m) + kWeightUp): by differences, which are finite and exact next to the maximum however large
  // cs and m are.  They move when a product is above th.
  float st_n[2] = {FLT_MAX, FLT_MAX}, st_d[2] = {0.f, 0.f};  // (st_n: -m)
  float th[2] = {-FLT_MAX, -FLT_MAX};
  float oacc[KT][4];
#pragma unroll
  for (int i = 0; i < KT; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;

  [[maybe_unused]] unsigned full_left = 0;  // `full` from tile k on

  // this lane's accumulators' sums of the share so far, kSumTiles tiles at a time, against the maxima -sums_n
  [[maybe_unused]] float4 sums_local[SPLIT ? 1 : KT];
  [[maybe_unused]] float4* sums = sums_local;
  if constexpr (!SPLIT) asm volatile("" : "+l"(sums));  // (kept out of the registers)
  [[maybe_unused]] float sums_n[2] = {FLT_MAX, FLT_MAX};

#pragma unroll 1
  for (int k = 0; k < k_end;) {
  // NQ tiles from the ring: their chains of loads, products and exponentials are independent and
  // overlap in the warp, and share the vote and the rescale
  const int k_next = SPLIT ? k_end : min(k + kSumTiles, k_end);
#pragma unroll 1
  for (; k < k_next; k += NQ) {
    cp_async_group_wait<NST - 1>();
    __syncwarp();  // every lane's copies, and what was written beside them
    const uint8_t* const stage = my_ring + cst * T::kStage;
    float sc[NQ][4];
    // a row's scale bytes in shared memory (v: of V)
    auto scales_at = [&](int i, int r, bool v) -> const uint8_t* {
      const uint8_t* at = stage + i * T::kPair + 2 * T::kCodes + (v ? T::kScales : 0) + r * SR;
      if constexpr (ROWS && NB < 4) at += ((s_half[warp][v ? 1 : 0][cst][i] >> r) & 1) * NB;
      return at;
    };
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      // -------------------------------------------------------------- S^T = K Q^T
      const uint8_t* const tile = stage + i * T::kPair;
      const uint8_t* sa = scales_at(i, kr, false);
      const uint8_t* sb = scales_at(i, kr + 8, false);
      sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
      for (int c = 0; c < KCH; ++c) {
        uint32_t ka[KW], kb[KW];
        lds_words<KB>(tile + koff[c], ka);
        lds_words<KB>(tile + 8 * RB + koff[c], kb);
        constexpr int BPC = 2 * KB > SB ? 2 * KB / SB : 1;  // blocks of a chunk
        const int blk = 2 * KB * (4 * c + q4) / SB;
        // their scales: of row kr (low halves) and kr + 8 (high halves); of two blocks, a pair each
        uint32_t fa, fb;
        if constexpr (BPC == 2) {
          if constexpr (SB == 16) {  // (both bytes at once)
            fa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sa + blk));
            fb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sb + blk));
          } else {
            fa = mx_scales<SB>(sa[blk], sa[blk + 1]);
            fb = mx_scales<SB>(sb[blk], sb[blk + 1]);
          }
        } else {
          fa = fb = mx_scales<SB>(sa[blk], sb[blk]);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t ra[4], rb[4];
          mx_codes(ka[w], ra);
          mx_codes(kb[w], rb);
          const bool second = BPC == 2 && 2 * w >= KW;
          auto of_a = [&](uint32_t x) { return second ? mul_hi(x, fa) : mul_lo(x, fa); };
          auto of_b = [&](uint32_t x) { return BPC == 1 || second ? mul_hi(x, fb) : mul_lo(x, fb); };
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kt = 2 * (KW * c + w) + h;
            const uint32_t a[4] = {of_a(ra[2 * h]), of_b(rb[2 * h]), of_a(ra[2 * h + 1]), of_b(rb[2 * h + 1])};
            Mma<__half>::run(sc[i], a, qf[kt][0], qf[kt][1]);
            if constexpr (SPLIT) Mma<__half>::run(sc[i], a, ql[kt][0], ql[kt][1]);
          }
        }
      }
    }
    // ---------------------------------------------------------------- online softmax (log2)
    bool whole;  // every row of the stage counts for every column
    if constexpr (ROWS) {
      whole = !MQ || s_r0[warp][cst][NQ - 1] + 16 <= lim_all;
#pragma unroll
      for (int i = 0; i < NQ; ++i) whole = whole && s_rows[warp][cst][i] == 0xffff;
    } else {
      if ((k & 31) == 0) full_left = full;  // (the batch of k is the last one loaded: fewer than 32 tiles are ahead)
      whole = (full_left & ((1u << NQ) - 1)) == (1u << NQ) - 1;
      full_left >>= NQ;
    }
    if (!whole) {
      // Rarely (warp-uniform).  Rows that do not count get scores of -inf, and zeros for V's scales,
      // which may be anything there.  A row that some of the queries alone attend must not reach the
      // others by a NaN scale of V: such scales go to the outputs of those that attend it.
      const int m_at = ROWS ? cst : (k >> 5) & 1, m_i = ROWS ? 0 : k & 31;  // the tiles' masks
      int ln;  // (the lane's number, read here: nothing of this branch is worked out in every stage)
      asm volatile("mov.u32 %0, %%laneid;" : "=r"(ln)::"memory");
      auto is_nan = [](uint8_t b) { return SB == 16 ? (b & 0x7f) == 0x7f : b > 127 + 13; };
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const unsigned rows = s_rows[warp][m_at][m_i + i];
        const int r0 = MQ ? s_r0[warp][m_at][m_i + i] : 0;
        // whether row r counts for this lane's column 2 q4 + h
        auto counts = [&](int r, int h) { return ((rows >> r) & 1) && (!MQ || r0 + r < (h ? lim1 : lim0)); };
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!counts(mx_row<D>(ln >> 2) + (e >> 1) * 8, e & 1)) sc[i][e] = -INFINITY;
        uint8_t* const vs = const_cast<uint8_t*>(stage) + i * T::kPair + 2 * T::kCodes + T::kScales;
        bool nan = false;
        for (int x = ln; x < T::kScales; x += 32) {
          if (!((rows >> (x / SR)) & 1)) vs[x] = 0;
          nan = nan || is_nan(vs[x]);
        }
        if (MQ && __any_sync(0xffffffffu, nan)) {
          constexpr int VBL = RL > SB ? RL / SB : 1;
#pragma unroll
          for (int b = 0; b < VBL; ++b) {
            bool bad[2] = {false, false};
#pragma unroll 1
            for (int r = 0; r < 16; ++r) {
              if (!is_nan(scales_at(i, r, true)[RL * g_id / SB + b])) continue;
              bad[0] = bad[0] || counts(r, 0);
              bad[1] = bad[1] || counts(r, 1);
            }
#pragma unroll
            for (int mt = b * KT / VBL; mt < (b + 1) * KT / VBL; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (bad[h]) oacc[mt][h] = oacc[mt][h + 2] = __int_as_float(0x7fc00000);
          }
          __syncwarp();
          for (int x = ln; x < T::kScales; x += 32)
            if (is_nan(vs[x])) vs[x] = 0;
        }
      }
      __syncwarp();
    }
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      t0 = fmaxf(t0, fmaxf(sc[i][0], sc[i][2]));
      t1 = fmaxf(t1, fmaxf(sc[i][1], sc[i][3]));
    }
    if (__any_sync(0xffffffffu, t0 > th[0] || t1 > th[1])) {
      const float mn0 = fmaxf(-st_n[0], max_over_groups(t0)), mn1 = fmaxf(-st_n[1], max_over_groups(t1));
      const float a0 = fast_exp2((-st_n[0] - mn0) * cs0), a1 = fast_exp2((-st_n[1] - mn1) * cs1);
      st_d[0] *= a0;
      st_d[1] *= a1;
      st_n[0] = -mn0;
      st_n[1] = -mn1;
      // (rounded down: never more than 2^kLazyMaxMx above the maximum; a column without a row so far keeps its own)
      if (mn0 != -FLT_MAX) th[0] = __fadd_rd(mn0, kLazyMaxMx / cs0);
      if (mn1 != -FLT_MAX) th[1] = __fadd_rd(mn1, kLazyMaxMx / cs1);
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) {
        oacc[mt][0] *= a0;
        oacc[mt][1] *= a1;
        oacc[mt][2] *= a0;
        oacc[mt][3] *= a1;
      }
    }
    uint32_t pb[NQ][2];
    [[maybe_unused]] uint32_t pl[SPLIT ? NQ : 1][2];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 x = scaled_sums(sc[i][e], sc[i][e + 1], make_float2(st_n[0], st_n[1]), make_float2(cs0, cs1), kWeightUp);
        pr[e] = fast_exp2(x.x);
        pr[e + 1] = fast_exp2(x.y);
      }
      st_d[0] += pr[0] + pr[2];
      st_d[1] += pr[1] + pr[3];
      // P^T as a B fragment: rows 2 q4, 2 q4 + 1 (+ 8) of column g_id
      if constexpr (SPLIT) {
        uint32_t hi, lo;
        split2<__half>(pr[0], pr[1], hi, lo);
        pb[i][0] = transpose8(hi);
        pl[i][0] = transpose8(lo);
        split2<__half>(pr[2], pr[3], hi, lo);
        pb[i][1] = transpose8(hi);
        pl[i][1] = transpose8(lo);
      } else {
        pb[i][0] = transpose8(pack2<__half>(pr[0], pr[1]));
        pb[i][1] = transpose8(pack2<__half>(pr[2], pr[3]));
      }
    }
    // ---------------------------------------------------------------- O^T += V^T P^T
    // m-tile mt: rows g_id / g_id + 8 are dims RL g_id + 2 mt / + 1
    constexpr int VBL = RL > SB ? RL / SB : 1;  // blocks of a thread's dims
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const uint8_t* const tile = stage + i * T::kPair;
      uint32_t v[4][VB / 4];  // rows vr[0], vr[1], vr[0] + 8, vr[1] + 8
      uint32_t sv[2][VBL];    // scales of rows (vr[0], vr[1]) and of the same + 8
#pragma unroll
      for (int j = 0; j < 4; ++j) lds_words<VB>(tile + voff[j & 1] + 8 * RB * (j >> 1), v[j]);
#pragma unroll
      for (int b = 0; b < VBL; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int blk = RL * g_id / SB + b;
          sv[j][b] = mx_scales<SB>(scales_at(i, vr[0] + 8 * j, true)[blk], scales_at(i, vr[1] + 8 * j, true)[blk]);
        }
#pragma unroll
      for (int w = 0; w < VB / 4; ++w) {
        // codes of rows (0, 1) and (2, 3) side by side in a byte: even dims, odd dims
        constexpr uint32_t M = 0x0f0f0f0fu;
        uint32_t ev[2][4], od[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t x = v[2 * j][w], y = v[2 * j + 1][w];
          mx_codes((x & M) | ((y << 4) & ~M), ev[j]);
          mx_codes(((x >> 4) & M) | (y & ~M), od[j]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int mt = 4 * w + u, b = mt * VBL / KT;
          const uint32_t a[4] = {mul_h2(ev[0][u], sv[0][b]), mul_h2(od[0][u], sv[0][b]),
                                 mul_h2(ev[1][u], sv[1][b]), mul_h2(od[1][u], sv[1][b])};
          if constexpr (SPLIT) {
            // (the products' own sum is cut off at 24 bits, which adds up over hundreds of tiles: a tile's
            // are summed from zero, and rounded to nearest into the output)
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            Mma<__half>::run(part, a, pl[i][0], pl[i][1]);
            Mma<__half>::run(part, a, pb[i][0], pb[i][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[mt][e] += part[e];
          } else {
            Mma<__half>::run(oacc[mt], a, pb[i][0], pb[i][1]);
          }
        }
      }
    }
    // every lane has its codes in registers: the stage takes the next tiles
    __syncwarp();
    if (k_issued < k_end) issue(k_issued, cst);
    k_issued += NQ;
    cp_async_group();
    cst ^= 1;
    // A scheduler's older warps run ahead of its younger ones, which then end alone and leave it idle:
    // a warp that is kLead stages ahead of another of its scheduler lets it catch up for a moment.
    ++stages;
    if constexpr (NW > 4) {
      if ((stages & 3) == 0) {
        if (lane == 0) *(volatile int*)&s_done[warp] = stages;
        int least = INT_MAX;
#pragma unroll
        for (int i = 4; i < NW; i += 4) least = min(least, *(volatile int*)&s_done[warp + i < NW ? warp + i : warp + i - NW]);
        if (stages > least + kLead) __nanosleep(kNap);
      }
    }
  }
  if constexpr (!SPLIT) {
    if (__builtin_expect(k_end > kSumTiles, 0)) {
      const bool first = k <= kSumTiles;
      const float a0 = fast_exp2((st_n[0] - sums_n[0]) * cs0), a1 = fast_exp2((st_n[1] - sums_n[1]) * cs1);
      sums_n[0] = st_n[0];
      sums_n[1] = st_n[1];
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) {
        float4 x = first ? make_float4(0.f, 0.f, 0.f, 0.f) : sums[mt];
        x = make_float4(fmaf(x.x, a0, oacc[mt][0]), fmaf(x.y, a1, oacc[mt][1]), fmaf(x.z, a0, oacc[mt][2]), fmaf(x.w, a1, oacc[mt][3]));
        if (k < k_end) {
          sums[mt] = x;
          x = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        oacc[mt][0] = x.x, oacc[mt][1] = x.y, oacc[mt][2] = x.z, oacc[mt][3] = x.w;
      }
    }
  }
  }
  st_d[0] = sum_over_groups(st_d[0]);
  st_d[1] = sum_over_groups(st_d[1]);

  // ---------------------------------------------------------------- finish the segment
  int ln;  // (the lane's number, read here: nothing that follows is worked out before the loop)
  asm volatile("mov.u32 %0, %%laneid;" : "=r"(ln)::"memory");
  const int gf = ln >> 2, qf4 = ln & 3;
  // This thread holds columns 2 qf4 (o0, o2) and 2 qf4 + 1 (o1, o3), dims RL gf .. + RL - 1.
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float inv = st_d[h] == 0.f ? 0.f : p.out_scale / st_d[h];
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) oacc[mt][h] *= inv, oacc[mt][h + 2] *= inv;
  }
  const bool mine = ua == 0 && ub == sg.n;  // the whole segment: this warp writes the output
  if (!mine) {
    // its state to shared memory; the first of the block's warps that share the segment notes it for the
    // block to merge (lane i looks at warp i's range)
    const int side = sg.off > ws.x0;
    float* const o = state_of(warp, side);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 2 * qf4 + h;
      if (j >= hcount) continue;
#pragma unroll
      for (int x = 0; x < RL / 4; ++x)
        reinterpret_cast<float4*>(o + j * D + RL * gf)[x] =
            make_float4(oacc[2 * x][h], oacc[2 * x][h + 2], oacc[2 * x + 1][h], oacc[2 * x + 1][h + 2]);
      if (gf == 0) {
        s_pmd[warp][side][j] = make_float2(-st_n[h], st_d[h] * kWeightDown);
        s_pcs[warp][side][j] = h ? cs1 : cs0;
      }
    }
    const int wi = lane < NW && lane % zg == warp % zg ? lane : -1;
    const long long w0 = wi >= 0 ? s_start[wi].x0 : 0, w1 = wi >= 0 ? s_start[wi].x1 : 0;
    const int units = wi >= 0 ? units_within(sg.off, C, sg.n, w0, w1) : 0;
    const int in_block = __reduce_add_sync(0xffffffffu, units);
    const unsigned from = __ballot_sync(0xffffffffu, units > 0), late = __ballot_sync(0xffffffffu, units > 0 && sg.off > w0);
    if (lane == 0 && warp == __ffs(from) - 1) {
      const PartMerge e{sg.off, ws.U, sg.b, sg.hz, sg.n, hk, c0, hcount, C, zg};
      s_merge[atomicAdd(&s_n_merge, 1)] =
          SegmentMerge{e, in_block == sg.n ? SegmentBlocks{} : blocks_of(e), in_block, from, late};
    }
  }
  if (mine) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 2 * qf4 + h;
      if (j >= hcount) continue;
      const size_t row = col_row<MQ>(p, sg.b, hk, c0 + j);
      const bool empty = st_d[h] == 0.f;
      float inv = 1.f, lse = empty ? kEmptyM : fmaf(-st_n[h], h ? cs1 : cs0, log2f(st_d[h]) - kWeightUp);
      if (p.sink) {
        const SinkAdj sa = apply_sink(p, col_head<MQ>(p, hk, c0 + j), lse, empty);
        inv = sa.scale;
        lse = sa.lse;
      }
#pragma unroll
      for (int x = 0; x < RL / 4; ++x)
        store_four(p, row * D + RL * gf + 4 * x,
                   make_float4(oacc[2 * x][h] * inv, oacc[2 * x][h + 2] * inv, oacc[2 * x + 1][h] * inv,
                               oacc[2 * x + 1][h + 2] * inv));
      if (gf == 0) p.lse[row] = lse;
    }
  }
  }  // ua < ub
  if (sg.off + C + sg.n >= cx1 || !next_segment(p, sg, C)) break;
  }  // segments
  if (!waited) pdl_wait();  // (a worker without units: what the block merges may still follow it)
  if (lane == 0) *(volatile int*)&s_done[warp] = INT_MAX / 2;
  merge_states<D, MQ, NW>(p, s_merge, s_n_merge, s_pmd, s_pcs, state_of);
}

// ----------------------------------------------------------------------------- launch
template <int SB, bool SPLIT, int D, bool MQ, bool ROWS>
static cudaError_t launch_mx_t(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  constexpr int NW = mx_warps(SPLIT, D);
  constexpr int BLOCKS = 1;
  constexpr int dyn = mx_smem_bytes<SB, D, ROWS, NW>();
  auto kern = decode_mx_kernel<SB, SPLIT, D, MQ, ROWS, NW, BLOCKS>;
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
  return launch_pdl(kern, grid, dim3(NW * 32), dyn, st, p);
}

template <int SB, bool SPLIT, int D, bool ROWS>
static cudaError_t launch_mx_q(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  return p.q_len > 1 ? launch_mx_t<SB, SPLIT, D, true, ROWS>(p, grid, st, cfg)
                     : launch_mx_t<SB, SPLIT, D, false, ROWS>(p, grid, st, cfg);
}

template <int SB, bool SPLIT, bool ROWS>
static cudaError_t launch_mx(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  switch (p.D) {
    case 64: return launch_mx_q<SB, SPLIT, 64, ROWS>(p, grid, st, cfg);
    case 128: return launch_mx_q<SB, SPLIT, 128, ROWS>(p, grid, st, cfg);
    case 256: return launch_mx_q<SB, SPLIT, 256, ROWS>(p, grid, st, cfg);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pd
