// Pieces shared by the decodes of caches with scales (decode_bs.cuh, decode_mx.cuh): the mbarrier of
// a warp's ring, asynchronous copies, output stores, and the merge of the partial states that the
// workers of a block and the blocks of a segment leave.
#pragma once

#include <cfloat>
#include <type_traits>

#include "decode_common.cuh"

namespace pd {

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
__device__ __forceinline__ void cp_async_chunk(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_scale(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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

// ----------------------------------------------------------------------------- line starts
// The start of each of the block's NW workers on the cost line, as worker_starts (decode_common.cuh)
// gives it, by a binary search over the sequences' places: those of a host plan, or sums made here by
// the whole block (each thread those of `per` consecutive sequences).  Ends with a block barrier.
template <int NT, int NW>
__device__ __forceinline__ void line_starts(const DecodeParams& p, WorkerStart* s_ws, long long* s_pre) {
  __shared__ long long s_warp[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, C = p.seg_cost;
  const int zg = p.mode == kSchedBalanced ? p.zg : 1, HZ = p.H_kv * p.n_z / zg;
  const int per = p.hp_B ? 1 : (p.B + NT - 1) / NT;
  auto cost = [&](int b) { return units_of(load_seq(p, b), p.P) + C; };
  if (p.mode == kSchedBalanced && !p.hp_B) {
    long long mine = 0;
    for (int b = min(tid * per, p.B); b < min((tid + 1) * per, p.B); ++b) mine += cost(b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_warp[wid] = incl;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < wid; ++i) incl += s_warp[i];
    s_pre[tid] = incl - mine;
    if (tid == NT - 1) s_pre[NT] = incl;
    __syncthreads();
  }
  if (tid < NW) {
    WorkerStart s{};
    s.b = -1;
    if (p.mode == kSchedBalanced) {
      const int parts = p.hp_B ? p.B : NT;  // places known: of each sequence, or of each thread's
      auto place = [&](int i) { return p.hp_B ? (long long)p.hp[i] : s_pre[i]; };
      const long long W = (long long)gridDim.x * NW / zg, w = ((long long)blockIdx.x * NW + tid) / zg;
      s.U = place(parts) * HZ;
      s.x0 = div_floor(w * s.U, W);
      s.x1 = div_floor((w + 1) * s.U, W);
      if (s.x0 < s.x1) {
        int lo = 0, hi = parts - 1;  // last i with place(i) * HZ <= x0
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (place(mid) * HZ <= s.x0) lo = mid;
          else hi = mid - 1;
        }
        long long first = place(lo);
        int b = lo, n;
        if (p.hp_B) {
          n = p.hp[lo + 1] - p.hp[lo];
        } else {
          b = lo * per;
          while ((first + (n = cost(b))) * HZ <= s.x0) {
            first += n;
            ++b;
          }
        }
        s.b = b;
        s.hz = (int)div_floor(s.x0 - first * HZ, n);
        s.off = first * HZ + (long long)s.hz * n;
        s.hz = s.hz * zg + tid % zg;  // (NW is a multiple of zg)
      }
    } else if (p.mode == kSchedPerBlock) {
      s.b = (int)(blockIdx.x / HZ);
      s.hz = (int)(blockIdx.x - (unsigned)s.b * HZ);
      s.U = units_of(load_seq(p, s.b), p.P);
      s.x0 = tid * s.U / NW;
      s.x1 = (tid + 1) * s.U / NW;
      if (s.x0 == s.x1) s.b = -1;
    } else {
      const long long w = (long long)blockIdx.x * NW + tid;
      s.U = (long long)p.B * HZ;
      if (w < s.U) {
        s.b = (int)(w / HZ);
        s.hz = (int)(w - (long long)s.b * HZ);
        s.x1 = LLONG_MAX;
      }
    }
    s_ws[tid] = s;
  }
  __syncthreads();
}

// ----------------------------------------------------------------------------- merges at the block's end
// A warp leaves its part of a segment that it shares as a state (per column normalised outputs, the maximum m of
// the products before the column's factor cs, and d = sum 2^(cs (s - m))) in shared memory and goes on.  At its
// end the block merges its states of each such segment (M = max m_s, w_s = d_s 2^(cs (m_s - M)), out = sum w_s
// o_s / sum w_s), all segments at once.  Differences of maxima stand where a log-sum-exp would be rounded to
// the size of the scores; a state without rows has d = 0 and m = -FLT_MAX.  If the block
// holds all units of a segment that is the result; else it publishes the state and adds its units to the
// segment's counter, and the block that completes the count merges the blocks' states.  Such code runs
// once, from a cold instruction cache, and each dependent step costs its latency: it is kept short, and
// its steps are shared by all segments (a warp that merged its own segments from its registers took 16 %
// longer for 24 sequences with four queries, 9 % for 32 sequences and 4 % less for 256).
struct PartMerge {
  long long off, U;  // the segment's place on the cost line, and the line's length
  int b, hz, n, hk, c0, hcount, C, zg;
};

// The units of a segment at line position off within the positions [x0, x1).
__device__ __forceinline__ int units_within(long long off, int C, int n, long long x0, long long x1) {
  return (int)(min(max(x1 - off - C, 0ll), (long long)n) - min(max(x0 - off - C, 0ll), (long long)n));
}

// The first block that holds units of a segment, how many blocks do, and the slot of one's state:
// two per block and slice of side-by-side columns, for the segment that the block's range starts in
// (or at) and the one that it ends in.
struct SegmentBlocks {
  long long first;
  int n;
  bool ends_in;  // the first block's range does not start in the segment
};
__device__ __forceinline__ SegmentBlocks blocks_of(const PartMerge& e) {
  const long long G = gridDim.x;
  SegmentBlocks s;
  s.first = share_of(e.off + e.C, e.U, G);
  s.n = (int)(share_of(e.off + e.C + e.n - 1, e.U, G) - s.first + 1);
  s.ends_in = e.off > div_floor(s.first * e.U, G);
  return s;
}
__device__ __forceinline__ long long slot_of(const PartMerge& e, const SegmentBlocks& s, int i) {
  return ((2 * (s.first + i) + (i == 0 && s.ends_in)) * e.zg + (e.zg > 1 ? e.hz % e.zg : 0)) * kMaxGroupPerCta;
}
// Whether block first + i has units: with fewer positions than blocks some between have none.
__device__ __forceinline__ bool holds_units(const PartMerge& e, const SegmentBlocks& s, int i) {
  const long long G = gridDim.x;
  return e.U >= G || div_floor((s.first + i) * e.U, G) < div_floor((s.first + i + 1) * e.U, G);
}

struct SegmentMerge {
  PartMerge e;
  SegmentBlocks blocks;
  int in_block;         // its units in the block
  unsigned from, late;  // the warps that hold states of it, and those whose state is that of their last segment
};
template <int NW>
struct MergeScratch {
  float weight[NW + 4][NW][kMaxGroupPerCta];  // of a segment's states, by column
  float2 md[NW + 4][kMaxGroupPerCta];         // of the block's state
  float cs[NW + 4][kMaxGroupPerCta];
  bool all[NW + 4];  // the segment is complete, and its blocks' states are to be merged
};
// (s_merge, s_n: the segments; state_of(warp, side), s_pmd, s_pcs: the states, of a warp's first and last segment.
// A published state's m and d lie in p.part_lse, a pair a column: two slots per block and slice side by side, where
// the workspace has two per warp.)
template <int D, bool MQ, int NW, typename StateOf>
__device__ __forceinline__ void merge_states(const DecodeParams& p, const SegmentMerge (&s_merge)[NW + 4], const int& s_n,
                                           const float2 (&s_pmd)[NW][2][kMaxGroupPerCta],
                                           const float (&s_pcs)[NW][2][kMaxGroupPerCta], StateOf state_of) {
  constexpr int NT = NW * 32, G8 = kMaxGroupPerCta, kItems = G8 * (D / 4);  // of a segment: a column and four dims each
  static_assert(NW >= 8, "room for the published pairs: at most four slices side by side");
  __shared__ MergeScratch<NW> s;
  const int tid = threadIdx.x;
  __syncthreads();
  const int n = s_n;
  if (n == 0) return;
  float2* const part_md = reinterpret_cast<float2*>(p.part_lse);
  auto put = [&](int w, int j, int d, float4 o, float2 md, bool final) {
    const PartMerge& e = s_merge[w].e;
    if (final) {
      const bool empty = md.y == 0.f;
      float l = kEmptyM;
      if ((p.sink || d == 0) && !empty) l = fmaf(md.x, s.cs[w][j], log2f(md.y));
      if (p.sink) {
        const SinkAdj sa = apply_sink(p, col_head<MQ>(p, e.hk, e.c0 + j), l, empty);
        o = make_float4(o.x * sa.scale, o.y * sa.scale, o.z * sa.scale, o.w * sa.scale);
        l = sa.lse;
      }
      const size_t row = col_row<MQ>(p, e.b, e.hk, e.c0 + j);
      store_four(p, row * D + d, o);
      if (d == 0) p.lse[row] = l;
    } else {
      const SegmentBlocks& sb = s_merge[w].blocks;
      const long long at = slot_of(e, sb, (int)(blockIdx.x - sb.first)) + j;
      *reinterpret_cast<float4*>(p.part_o + at * D + d) = o;
      if (d == 0) part_md[at] = md;
    }
  };
  // the block's own states: their weights, then the sums
  for (int x = tid; x < n * G8; x += NT) {
    const int w = x / G8, j = x % G8;
    const unsigned from = s_merge[w].from, late = s_merge[w].late;
    const int one = __ffs(from) - 1;
    const float cs = s_pcs[one][(late >> one) & 1][j];
    float2 md[NW];
    float M = -FLT_MAX, den = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      md[i] = (from >> i) & 1 ? s_pmd[i][(late >> i) & 1][j] : make_float2(-FLT_MAX, 0.f);
      M = fmaxf(M, md[i].x);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      md[i].y *= fast_exp2((md[i].x - M) * cs);
      den += md[i].y;
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int i = 0; i < NW; ++i) s.weight[w][i][j] = md[i].y * inv;
    s.md[w][j] = make_float2(M, den);
    s.cs[w][j] = cs;
  }
  __syncthreads();
  for (int x = tid; x < n * kItems; x += NT) {
    const int w = x / kItems, j = x % kItems / (D / 4), d = x % (D / 4) * 4;
    if (j >= s_merge[w].e.hcount) continue;
    const unsigned from = s_merge[w].from, late = s_merge[w].late;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < NW; ++i) {
      if (!((from >> i) & 1)) continue;
      const float x_ = s.weight[w][i][j];
      const float4 o = *reinterpret_cast<const float4*>(state_of(i, (late >> i) & 1) + j * D + d);
      acc = make_float4(fmaf(x_, o.x, acc.x), fmaf(x_, o.y, acc.y), fmaf(x_, o.z, acc.z), fmaf(x_, o.w, acc.w));
    }
    put(w, j, d, acc, s.md[w][j], s_merge[w].in_block == s_merge[w].e.n);
  }
  if (p.mode != kSchedBalanced) return;
  __syncthreads();
  // the counts of the segments' units (the fence follows the whole block's stores)
  if (tid < n) {
    const PartMerge& e = s_merge[tid].e;
    const int in_block = s_merge[tid].in_block;
    bool all = false;
    if (in_block < e.n) {
      fence_acq_rel_gpu();
      int* cnt = p.counters + (size_t)e.b * p.H_kv * p.n_z + e.hz;
      all = atomicAdd(cnt, in_block) + in_block == e.n;
      if (all) *cnt = 0;  // every other block's units have arrived: reset for reuse
      fence_acq_rel_gpu();
    }
    s.all[tid] = all;
  }
  __syncthreads();
  // the blocks' states
#pragma unroll 1
  for (int x = tid; x < n * kItems; x += NT) {
    const int w = x / kItems, j = x % kItems / (D / 4), d = x % (D / 4) * 4;
    const PartMerge& e = s_merge[w].e;
    if (j >= e.hcount || !s.all[w]) continue;
    const SegmentBlocks sb = s_merge[w].blocks;
    const float cs = s.cs[w][j];
    float M = -FLT_MAX, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // four states' sums and rows in flight together (eight, twice the cold code: 32 sequences 22.4 us for 21.7)
#pragma unroll 1
    for (int i0 = 0; i0 < sb.n; i0 += 4) {
      float2 md[4];
      float4 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long at = slot_of(e, sb, min(i0 + i, sb.n - 1)) + j;
        md[i] = __ldcg(part_md + at);
        o[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + d));
      }
      float m = M;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= sb.n || !holds_units(e, sb, i0 + i)) md[i] = make_float2(-FLT_MAX, 0.f);
        m = fmaxf(m, md[i].x);
      }
      const float f = fast_exp2((M - m) * cs);
      M = m;
      den *= f;
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (md[i].y == 0.f) continue;  // (of a block without units: not written)
        const float x_ = md[i].y * fast_exp2((md[i].x - M) * cs);
        den += x_;
        acc = make_float4(fmaf(x_, o[i].x, acc.x), fmaf(x_, o[i].y, acc.y), fmaf(x_, o[i].z, acc.z), fmaf(x_, o[i].w, acc.w));
      }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    put(w, j, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), make_float2(M, den), true);
  }
}

// ----------------------------------------------------------------------------- states in shared memory
// A segment's states within the block are merged first (lse = M + log2 sum 2^(lse_s - M), out =
// sum 2^(lse_s - M) o_s / sum 2^(lse_s - M)).  If the block holds all of its units that is the
// result; else the block publishes one state and adds its units to the segment's counter, and
// the block that completes the count merges the blocks' states.  So a segment split over the
// four warps of a block never leaves it, and one over several blocks costs a state per block.
// Called by the whole block, after every warp has written its entries; s0: the block's first start.
// (The 8-bit decode's: four warps and log-sum-exps, segment after segment.  merge_states above rounds in another
// order, so this one stays, and with it that decode's results bit for bit.)
template <int D, bool MQ, int NW, typename StateOf>
__device__ __forceinline__ void merge_parts(const DecodeParams& p, PartEntry (&s_part)[NW][2],
                                            float (&s_plse)[NW][2][kMaxGroupPerCta], int (&s_last)[2 * NW],
                                            const WorkerStart& s0, int C, int zg, StateOf state_of) {
  constexpr int NT = NW * 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  const long long U = s0.U, G = gridDim.x;
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
    const long long to = all ? 0 : slot_of(blockIdx.x, e.off > s0.x0, e.hz);  // (x0: the block's)
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

}  // namespace pd
