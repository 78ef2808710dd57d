// Pieces shared by the decodes of caches with scales (decode_bs.cuh, decode_mx.cuh): the mbarrier of
// a warp's ring, asynchronous copies, output stores, and the merge of the partial states that the
// workers of a block and the blocks of a segment leave.
#pragma once

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

// ----------------------------------------------------------------------------- partial states
// A segment's states within the block are merged first (lse = M + log2 sum 2^(lse_s - M), out =
// sum 2^(lse_s - M) o_s / sum 2^(lse_s - M)).  If the block holds all of its units that is the
// result; else the block publishes one state and adds its units to the segment's counter, and
// the block that completes the count merges the blocks' states.  So a segment split over the
// four warps of a block never leaves it, and one over several blocks costs a state per block.
// Called by the whole block, after every warp has written its entries; s0: the block's first start.
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
