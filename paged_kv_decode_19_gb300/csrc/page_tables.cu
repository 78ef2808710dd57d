// build_page_tables: the tables that a step's append and decode read, from the requests' lengths and
// the numbers of tokens they bring (or give back), on the device.
//
// With len_b the rows held, n_b the change, P rows a page, pages(x) = ceil(x / P):
//   indptr, append_indptr   exclusive sums of pages(len_b + n_b) and max(n_b, 0)
//   grown_b = max(0, pages(len_b + n_b) - pages(len_b)) pages come from the ring of free pages, at
//     head + (exclusive sum of grown) + j; freed_b = max(0, pages(len_b) - pages(len_b + n_b)) go to
//     tail + (exclusive sum of freed) + j.  The ring holds every page of the pool, so what is taken
//     and what is given back never share a place, and one pass does both.
//
// Bound by latency: two dependent loads (lengths, then a page id) around a block-wide scan; the bytes
// (8 per page, 12 per token) count from some 10^5 pages on.  So every block makes the scan of all
// requests itself, in shared memory, and fills its share of the outputs without waiting for another:
// each output finds its request by a binary search over the sums.  lengths and the ring's state, which
// every block reads, are moved on by the last block to have read them (a ticket in `state`).  Measured
// on one GB300, a call: one request 3.8 us, 256 requests 4.9 us, 61 requests with 230,000 pages and
// 75,000 new tokens 5.2 us (one page a thread at a time, and the ticket before the outputs: 7.2 us).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace pd {

namespace {
constexpr int kThreads = kTableThreads;

// Inclusive sum over the block of three counts and of one that saturates at `most` (>= 0, at most 2^30).
struct Sums {
  int pages, grown, freed, tokens;
};
__device__ __forceinline__ Sums plus(const Sums& a, const Sums& b, int most) {
  return {a.pages + b.pages, a.grown + b.grown, a.freed + b.freed, min(a.tokens + b.tokens, most)};
}
__device__ Sums block_scan(Sums x, int most, Sums* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y = {__shfl_up_sync(0xffffffffu, x.pages, o), __shfl_up_sync(0xffffffffu, x.grown, o),
                    __shfl_up_sync(0xffffffffu, x.freed, o), __shfl_up_sync(0xffffffffu, x.tokens, o)};
    if (lane >= o) x = plus(x, y, most);
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x = plus(x, s_warp[w], most);
  return x;
}

// The last b < n with at[b] <= i (at[0] = 0 <= i, non-decreasing; empty requests are passed over).
__device__ __forceinline__ int request_of(const int* at, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
}  // namespace

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const __grid_constant__ TableParams a) {
  extern __shared__ int s_dyn[];
  __shared__ Sums s_warp[kThreads / 32];
  __shared__ int s_flag;
  const int B = a.B, P = a.P, tid = threadIdx.x;
  int* const s_len = s_dyn;              // [B] rows held (0 for a request that is not taken)
  int* const s_pages = s_len + B;        // [B + 1] exclusive sums
  int* const s_grown = s_pages + B + 1;
  int* const s_freed = s_grown + B + 1;
  int* const s_tok = s_freed + B + 1;
  pdl_wait();  // inputs and state are the previous kernel's to write until it completes
  pdl_release();

  const long long head = a.state[0], tail = a.state[1];
  const int most = a.most_tokens + 1;
  // each thread counts `per` requests one after the other
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  auto count = [&](int b, int& len, int& n) -> Sums {
    len = a.lengths[b];
    n = a.new_tokens[b];
    const long long now = (long long)len + n;
    if (len < 0 || len > a.max_rows || now < 0 || now > a.max_rows) {
      set_error(a.err, kErrBadLength);
      len = -1;
      n = 0;
      return {0, 0, 0, 0};
    }
    const int held = (len + P - 1) / P, need = ((int)now + P - 1) / P;
    return {need, a.ring ? max(need - held, 0) : 0, a.ring ? max(held - need, 0) : 0, min(max(n, 0), most)};
  };
  Sums mine = {0, 0, 0, 0};
  int len1 = 0, n1 = 0;  // of the thread's last request
  for (int b = b0; b < b1; ++b) mine = plus(mine, count(b, len1, n1), most);
  const Sums incl = block_scan(mine, most, s_warp);
  // the place before its first request: what the inclusive sum holds less the thread's own (the
  // saturated one from the warps' sums would differ past `most`, where the step is not taken)
  Sums at = {incl.pages - mine.pages, incl.grown - mine.grown, incl.freed - mine.freed,
             max(incl.tokens - mine.tokens, 0)};
  for (int b = b0; b < b1; ++b) {
    int len = len1, n = n1;
    const Sums c = per == 1 ? mine : count(b, len, n);
    s_len[b] = max(len, 0);
    s_pages[b] = at.pages;
    s_grown[b] = at.grown;
    s_freed[b] = at.freed;
    s_tok[b] = at.tokens;
    at = plus(at, c, most);
  }
  if (b1 == B && (b0 < B || tid == 0)) {  // (one thread: the last with a request; B = 0: the first)
    s_pages[B] = at.pages;
    s_grown[B] = at.grown;
    s_freed[B] = at.freed;
    s_tok[B] = at.tokens;
  }
  __syncthreads();
  int n_pages = s_pages[B], n_tok = s_tok[B];
  const int n_grown = s_grown[B], n_freed = s_freed[B];
  const bool long_ = n_pages > a.values_cap || n_tok > a.most_tokens;
  const long long spare = tail - head;
  // (spare + freed within the ring: what is given back then lies behind all that may be taken)
  const bool short_ = a.ring && (head < 0 || spare < 0 || n_grown > spare || spare + n_freed > a.C);
  const bool ok = !long_ && !short_;  // else nothing is taken, and the tables describe empty sequences
  // Every read of lengths and state is behind the barriers above: the last block to come here may move
  // them on.  Its last thread asks for the ticket; the answer is looked at when the outputs are written.
  if (tid == kThreads - 1) {
    if (!ok) set_error(a.err, long_ ? kErrBadLength : kErrNoPages);
    unsigned long long before = 0;
    if (gridDim.x > 1) {
      fence_acq_rel_gpu();
      before = atomicAdd(reinterpret_cast<unsigned long long*>(a.state) + 2, 1ull);
    }
    s_flag = before == gridDim.x - 1;
  }
  const long long first = (long long)blockIdx.x * kThreads + tid, step = (long long)gridDim.x * kThreads;
  for (long long b = first; b <= B; b += step) {
    a.indptr[b] = ok ? s_pages[b] : 0;
    if (a.append_indptr) a.append_indptr[b] = ok ? s_tok[b] : 0;
    if (b == B) break;
    const int need = ok ? s_pages[b + 1] - s_pages[b] : 0;
    int now = 0;
    if (need) {
      // rows after the step: all of those held and new, of a request that shrinks what its input says
      const int grow = s_tok[b + 1] - s_tok[b];
      now = grow ? s_len[b] + grow : s_len[b] + min(a.new_tokens[b], 0);
    }
    a.length_info[b] = need ? now - (need - 1) * P : 0;
    if (a.window) {
      const bool cut = now > (long long)a.window + a.sinks;
      a.length_info[B + b] = cut ? now - a.window : 0;
      a.length_info[2 * B + b] = cut ? a.sinks : 0;
    }
  }
  if (!ok) n_pages = n_tok = 0;
  const int C = a.C;
  auto place = [&](long long x) { return x >> 32 ? (int)(x % C) : (int)((unsigned)x % (unsigned)C); };
  const int head_at = ok && n_grown ? place(head) : 0, tail_at = ok && n_freed ? place(tail) : 0;
  auto wrap = [&](int at0, int i) {  // (at0 + i) mod C, i <= C
    const long long x = (long long)at0 + i;
    return (int)(x >= C ? x - C : x);
  };
  auto held_of = [&](int b) { return (s_len[b] + P - 1) / P; };
  // four pages a thread at a time: one search, and the loads of all four under way together
  for (long long i0 = 4 * first; i0 < n_pages; i0 += 4 * step) {
    int b = request_of(s_pages, B, (int)i0), at[4], page[4];
    bool taken[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = (int)min(i0 + x, n_pages - 1ll);
      while (i >= s_pages[b + 1]) ++b;
      const int k = i - s_pages[b], held = held_of(b);
      at[x] = b;
      taken[x] = a.ring && k >= held;
      page[x] = taken[x] ? a.ring[wrap(head_at, s_grown[b] + k - held)] : a.table[b * a.table_stride + k];
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (i0 + x >= n_pages) break;
      a.values[i0 + x] = page[x];
      if (taken[x]) a.table[at[x] * a.table_stride + (i0 + x - s_pages[at[x]])] = page[x];
    }
  }
  if (ok) {
    for (long long i = first; i < n_freed; i += step) {
      const int b = request_of(s_freed, B, (int)i), k = s_pages[b + 1] - s_pages[b] + (int)i - s_freed[b];
      a.ring[wrap(tail_at, (int)i)] = a.table[b * a.table_stride + k];
    }
  }
  if (a.slots || a.positions) {
    for (long long t = first; t < a.T; t += step) {
      long long slot = -1;
      int o = 0;
      if (t < n_tok) {
        const int b = request_of(s_tok, B, (int)t);
        o = s_len[b] + (int)t - s_tok[b];
        const int k = o / P;
        const int held = held_of(b);
        const int page = a.ring && k >= held ? a.ring[wrap(head_at, s_grown[b] + k - held)] : a.table[b * a.table_stride + k];
        if (page < 0) set_error(a.err, kErrBadPage);  // (a table that does not hold the row: skipped)
        else slot = (long long)page * P + (o - k * P);
      }
      if (a.slots) a.slots[t] = slot;
      if (a.positions) a.positions[t] = o;
    }
  }
  __syncthreads();
  if (!s_flag) return;
  if (ok) {
    for (int b = tid; b < B; b += kThreads) {
      const int n = a.new_tokens[b], len = a.lengths[b];
      const long long now = (long long)len + n;
      if (len >= 0 && len <= a.max_rows && now >= 0 && now <= a.max_rows) a.lengths[b] = (int)now;
    }
  }
  if (tid == 0) {
    if (ok) {
      a.state[0] = head + n_grown;
      a.state[1] = tail + n_freed;
    }
    if (gridDim.x > 1) a.state[2] = 0;
  }
}

constexpr int smem_bytes(int B) { return (B + 4 * (B + 1)) * (int)sizeof(int); }

// The shared memory of the largest batch is allowed once per device: a limit set by every call to its own size could
// fall, between another thread's and its launch, below what that one asks for.
cudaError_t prepare_page_tables() {
  return cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxTableB));
}

cudaError_t launch_page_tables(const TableParams& a, int num_sms, cudaStream_t st) {
  // four outputs a thread, at most one block an SM
  const long long items = std::max<long long>(std::min<long long>(a.values_cap, (long long)a.B * a.max_pages),
                                                  a.slots || a.positions ? a.T : 0);
  const long long blocks = std::min<long long>(num_sms, std::max<long long>(1, (items + 4 * kThreads - 1) / (4 * kThreads)));
  return launch_pdl(page_tables_kernel, dim3((unsigned)blocks), dim3(kThreads), smem_bytes(a.B), st, a);
}

}  // namespace pd
