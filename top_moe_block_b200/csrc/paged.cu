// Paged KV cache bookkeeping: the block tables and slot maps of one serving
// step, and the write of the step's keys and values into their pages.
//
// Plan.  Rows b = 0 .. B-1 are the requests of the step, P the page size,
// pages(x) = ceil(x / P):
//   free stack   F = free_list[0 .. n_free) ++ the pages of the rows' former
//                requests (drop_len), row by row; top = |F|
//   new pages    need_b = pages(ctx_b + new_b) - pages(ctx_b); the j-th page
//                needed, row by row, is F[top - 1 - j]
//   tokens       cu = exclusive prefix sum of new_len; token t of row b sits at
//                position ctx_b + t - cu_b, in slot table[b][pos / P] * P + pos % P
// Everything follows from three prefix sums over the rows, so each CTA scans
// the (at most 4096) lengths itself into shared memory and then takes its
// share of the dropped pages, the new pages and the tokens, each of which
// finds its row by a binary search.  A small step is one CTA's; a large one
// takes two launches over the whole GPU, since dropped pages must be on the
// stack before they are handed out again: 1024 rows and 131072 tokens in
// 12.2 us (calls in a row), against 29 us in one cluster of eight CTAs.
// All or nothing: every page id that the step drops, pops or goes on with is looked
// at before any is handed out.  Until then only places of the stack above its top are
// written, and the second launch records no fault of its own: the status word that
// its CTAs read is the first launch's.
//
// Store.  kv[slot] = (k, v) of every token with a slot, as bf16 or as E4M3
// bytes (nearest, ties to even, saturating).  A thread moves 16-byte chunks of K
// and the same chunks of V, which it reads before it knows their slot.  Bound by
// HBM (16384 tokens into E4M3 pages: 6.2 us, 3.8 TB/s) or, for a decode step, by
// the launch and two round trips to memory (64 tokens: 2.1 us).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace zaya {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 4;                            // consecutive rows a thread scans
constexpr int kPlanMaxRows = kPlanThreads * kPlanRows;
constexpr uint32_t kSat = 1u << 30;                     // prefix sums saturate here (past any limit they are checked against)

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// Exclusive prefix sums of three values per thread over the CTA; `total` gets the sums.
__device__ __forceinline__ void scan3(uint32_t (&v)[3], uint32_t (&total)[3], uint32_t (*warp_sums)[3]) {
  const int lane = lane_id(), warp = warp_id();
  uint32_t inc[3] = {v[0], v[1], v[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] = sat_add(inc[k], a);
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < 3; ++k) warp_sums[warp][k] = inc[k];
  }
  __syncthreads();
  // every warp scans the 32 warp sums for itself
  uint32_t w[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) w[k] = warp_sums[lane][k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, w[k], o);
      if (lane >= o) w[k] = sat_add(w[k], a);
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    total[k] = __shfl_sync(0xffffffffu, w[k], 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w[k], warp > 0 ? warp - 1 : 0);
    const uint32_t prev = __shfl_up_sync(0xffffffffu, inc[k], 1);
    v[k] = sat_add(warp > 0 ? before : 0u, lane > 0 ? prev : 0u);
  }
}

// The row whose half-open range [pre[r], pre[r + 1]) holds x (x < pre[n]).
__device__ __forceinline__ int find_row(const uint32_t* pre, int n, uint32_t x) {
  int lo = 0, hi = n;   // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Tokens up to which one CTA does the whole step (two a thread): 4.2 to 4.5 us at 64 rows
// and tokens, where the second launch alone would add 2 to 3 us.
constexpr int kPlanOneCta = 2 * kPlanThreads;

enum PlanPart {
  PLAN_ALL,    // everything, one CTA
  PLAN_DROP,   // many CTAs: the page ids are checked, the dropped pages go above the stack's top
  PLAN_REST    // many CTAs, behind PLAN_DROP: the table, the lengths, the tokens
};

template <int PART>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedPlanParams p) {
  extern __shared__ uint32_t plan_sm[];
  uint32_t* s_cu = plan_sm;                // [B + 1] first token of each row
  uint32_t* s_need = s_cu + p.B + 1;       // [B + 1] new pages before each row
  uint32_t* s_gone = s_need + p.B + 1;     // [B + 1] dropped pages before each row
  __shared__ uint32_t warp_sums[kPlanThreads / 32][3];
  griddep_begin();
  const int tid = threadIdx.x;
  const int me = blockIdx.x * kPlanThreads + tid, all = gridDim.x * kPlanThreads;
  const int sh = p.page_shift, pm = (1 << sh) - 1;
  const long long room = (long long)p.max_pages << sh;
  // n_free_out may be n_free_in: its old value reaches PLAN_REST through the workspace
  const int n_free = PART == PLAN_REST ? *p.n_free_old : *p.n_free_in;

  // Ids are pages, but that a dropped entry may be -1 (no page).  On the stack of an earlier step or
  // in the page a row goes on with, -1 would be a page that its tokens' keys never reach.
  auto outside = [&](int id, int least = 0) { return id < least || id >= p.n_pages; };
  uint32_t v[3] = {0, 0, 0}, mine[kPlanRows][3];
  bool bad = status_peek(p.status) != 0;   // a fault earlier in the step: nothing is handed out
#pragma unroll
  for (int u = 0; u < kPlanRows; ++u) {
    const int b = tid * kPlanRows + u;
    mine[u][0] = mine[u][1] = mine[u][2] = 0;
    if (b < p.B) {
      const int ctx = p.ctx_len[b], fresh = p.new_len[b], drop = p.drop_len ? p.drop_len[b] : 0;
      const bool off = ctx < 0 || fresh < 0 || drop < 0 || (drop > 0 && ctx > 0) || (long long)ctx + fresh > room || drop > room;
      bad |= off;
      if (!off) {
        mine[u][0] = min((uint32_t)fresh, kSat);
        mine[u][1] = (uint32_t)((((long long)ctx + fresh + pm) >> sh) - (((long long)ctx + pm) >> sh));
        mine[u][2] = (uint32_t)(((long long)drop + pm) >> sh);
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = sat_add(v[k], mine[u][k]);
  }
  uint32_t total[3];
  scan3(v, total, warp_sums);
#pragma unroll
  for (int u = 0; u < kPlanRows; ++u) {
    const int b = tid * kPlanRows + u;
    if (b <= p.B) {
      s_cu[b] = v[0];
      s_need[b] = v[1];
      s_gone[b] = v[2];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = sat_add(v[k], mine[u][k]);
  }
  if (tid == kPlanThreads - 1 && p.B == kPlanMaxRows) {
    s_cu[p.B] = total[0];
    s_need[p.B] = total[1];
    s_gone[p.B] = total[2];
  }
  const uint32_t top = (uint32_t)max(n_free, 0) + total[2];
  bad |= n_free < 0 || top > (uint32_t)p.n_pages || total[1] > top || total[0] > (uint32_t)p.T;
  bad = __syncthreads_or(bad);
  if (PART == PLAN_DROP && me == 0) *p.n_free_old = n_free;

  // a token's row and position, and the id of its page: pages the row already held come from
  // its table, new ones from the stack (another thread may be writing their table entries)
  auto token = [&](int t, int& b, int& pos, bool& dropped) {
    b = find_row(s_cu, p.B, (uint32_t)t);
    const int ctx = p.ctx_len[b];
    pos = ctx + (int)((uint32_t)t - s_cu[b]);
    const int have = (int)(((long long)ctx + pm) >> sh), j = pos >> sh;
    const uint32_t at = top - 1 - (s_need[b] + (uint32_t)(j - have));
    dropped = j >= have && at >= (uint32_t)n_free;
    return j < have ? p.block_table[(size_t)b * p.max_pages + j] : p.free_list[at];
  };
  constexpr int kMine = kPlanOneCta / kPlanThreads;
  int row[kMine], pos[kMine], id[kMine];   // PLAN_ALL: this thread's tokens
  if (PART != PLAN_REST && !bad) {
    auto goes_on = [&](int b) {   // the page that holds some of row b's tokens and takes more
      const int ctx = b < p.B ? p.ctx_len[b] : 0;
      return (ctx & pm) && p.new_len[b] > 0 ? p.block_table[(size_t)b * p.max_pages + (ctx >> sh)] : 0;
    };
    const int first = PART == PLAN_DROP ? goes_on(me) : 0;   // on its way beside the dropped ones
    for (uint32_t k = me; k < total[2]; k += all) {   // former requests' pages go above the stack's top
      const int b = find_row(s_gone, p.B, k);
      const int x = p.block_table[(size_t)b * p.max_pages + (k - s_gone[b])];
      bad |= outside(x, -1);
      p.free_list[(uint32_t)n_free + k] = x;
    }
    if (PART == PLAN_ALL) {   // every page popped or gone on with is some token's
      if (total[2]) __syncthreads();
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int t = tid + u * kPlanThreads;
        row[u] = pos[u] = id[u] = -1;
        bool dropped = true;
        if ((uint32_t)t < total[0]) id[u] = token(t, row[u], pos[u], dropped);
        bad |= outside(id[u], dropped ? -1 : 0);
      }
    } else {
      for (long long k = (long long)top - total[1] + me; k < n_free; k += all) bad |= outside(p.free_list[k]);
      bad |= outside(first);
      for (int b = me + all; b < p.B; b += all) bad |= outside(goes_on(b));
    }
    bad = __syncthreads_or(bad);
  }
  if (bad) {   // nothing happens: no token has a slot, the table and the stack stay as they are
    if (PART != PLAN_REST && tid == 0) set_status(p.status, ZAYA_ERR_DEVICE_RANGE);   // keeps an earlier fault
    if (PART == PLAN_DROP) return;
    if (me == 0) {
      *p.n_free_out = n_free;
      p.cu_new[p.B] = 0;
    }
    for (int b = me; b < p.B; b += all) {
      p.cu_new[b] = 0;
      p.seq_len[b] = p.ctx_len[b];
    }
    for (int t = me; t < p.T; t += all) {
      p.slot_map[t] = -1;
      p.positions[t] = -1;
      p.token_row[t] = -1;
    }
    return;
  }
  if (PART == PLAN_DROP) return;
  // From here on page ids of the step come from the stack, and the table is written at
  // entries of dropped pages and of new ones only, each by one thread.
  if (me == 0) *p.n_free_out = (int)(top - total[1]);
  for (uint32_t k = me; k < total[2]; k += all) {   // dropped entries that no new page takes
    const int b = find_row(s_gone, p.B, k);
    const uint32_t j = k - s_gone[b];
    if (j >= s_need[b + 1] - s_need[b]) p.block_table[(size_t)b * p.max_pages + j] = -1;
  }
  for (uint32_t k = me; k < total[1]; k += all) {   // new pages come off it
    const int b = find_row(s_need, p.B, k);
    const int have = (int)(((long long)p.ctx_len[b] + pm) >> sh);
    p.block_table[(size_t)b * p.max_pages + have + (k - s_need[b])] = p.free_list[top - 1 - k];
  }
  for (int b = me; b <= p.B; b += all) {
    p.cu_new[b] = (int)s_cu[b];
    if (b < p.B) p.seq_len[b] = p.ctx_len[b] + p.new_len[b];
  }
  auto put = [&](int t, int b, int at, int page) {
    p.slot_map[t] = b < 0 ? -1 : page * (pm + 1) + (at & pm);
    p.positions[t] = at;
    p.token_row[t] = b;
  };
  if (PART == PLAN_ALL) {
#pragma unroll
    for (int u = 0; u < kMine; ++u)
      if (tid + u * kPlanThreads < p.T) put(tid + u * kPlanThreads, row[u], pos[u], id[u]);
  } else {
    for (int t = me; t < p.T; t += all) {
      int b = -1, at = -1;
      bool dropped;
      const int page = (uint32_t)t < total[0] ? token(t, b, at, dropped) : -1;
      put(t, b, at, page);
    }
  }
}

__device__ __forceinline__ uint2 e4m3x8(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 a = unpack_bf2(w[2 * h]), c = unpack_bf2(w[2 * h + 1]);
    o[h] = (uint32_t)pack_e4m3x2(a.x, a.y) | ((uint32_t)pack_e4m3x2(c.x, c.y) << 16);
  }
  return make_uint2(o[0], o[1]);
}

__global__ void __launch_bounds__(256) paged_store_kernel(const PagedStoreParams p, int tokens) {
  griddep_begin();
  if (status_peek(p.status)) return;
  const int vph = p.d / 8, vpr = p.n_kv * vph;   // 16-byte chunks per head / per token
  const int t0 = blockIdx.x * tokens, n = min(tokens, p.T - t0) * vpr;
  const int pm = (1 << p.page_shift) - 1;
  for (int i0 = threadIdx.x; i0 < n; i0 += 512) {
    int slot[2], c[2];
    uint4 kx[2], vx[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {   // all loads under way before the slots are looked at
      const int i = i0 + u * 256;
      slot[u] = -1;
      if (i >= n) continue;
      const int t = t0 + i / vpr;
      c[u] = i % vpr;
      slot[u] = p.slot_map[t];
      kx[u] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k) + (size_t)t * p.k_stride)[c[u]];
      vx[u] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + (size_t)t * p.v_stride)[c[u]];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (slot[u] < 0) continue;
      const int page = slot[u] >> p.page_shift;
      if (page >= p.n_pages) {
        set_status(p.status, ZAYA_ERR_DEVICE_RANGE);
        continue;
      }
      const size_t row = (((size_t)page * p.n_kv + c[u] / vph) << p.page_shift) + (slot[u] & pm);
      const size_t dst = row * vph + c[u] % vph;
      if (p.fp8) {
        static_cast<uint2*>(p.k_pages)[dst] = e4m3x8(kx[u]);
        static_cast<uint2*>(p.v_pages)[dst] = e4m3x8(vx[u]);
      } else {
        static_cast<uint4*>(p.k_pages)[dst] = kx[u];
        static_cast<uint4*>(p.v_pages)[dst] = vx[u];
      }
    }
  }
}

}  // namespace

int paged_plan_max_rows() { return kPlanMaxRows; }
int paged_plan_launches(int T) { return T <= kPlanOneCta ? 1 : 2; }

int launch_paged_plan(const PagedPlanParams& p, int num_sms, cudaStream_t st) {
  const size_t smem = (size_t)3 * (p.B + 1) * 4;
  auto go = [&](void (*kern)(PagedPlanParams), int grid) {
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * (kPlanMaxRows + 1) * 4) != cudaSuccess)
      return false;
    return launch_k(kern, dim3(grid), dim3(kPlanThreads), smem, st, nullptr, 0, p) == cudaSuccess;
  };
  if (paged_plan_launches(p.T) == 1) return go(paged_plan_kernel<PLAN_ALL>, 1) ? ZAYA_OK : ZAYA_ERR_CUDA;
  const long long ids = (p.drop_len ? (long long)p.B * p.max_pages : 0) + p.B + (p.T >> p.page_shift);   // at most
  const int drop = (int)std::min<long long>(num_sms, (ids + kPlanThreads - 1) / kPlanThreads);
  const int rest = std::min(num_sms, (p.T + kPlanThreads - 1) / kPlanThreads);
  return go(paged_plan_kernel<PLAN_DROP>, drop) && go(paged_plan_kernel<PLAN_REST>, rest) ? ZAYA_OK : ZAYA_ERR_CUDA;
}

int launch_paged_store(const PagedStoreParams& p, cudaStream_t st) {
  if (p.T <= 0) return ZAYA_OK;
  // 16 tokens a CTA (two chunks a thread in flight at 2 key heads of 128): 6.2 us for 16384 tokens,
  // against 7.8 with one chunk a thread; a decode step's 64 tokens are spread wider: 2.1 us against 2.3
  const int tokens = p.T >= 4096 ? 16 : 4, blocks = (p.T + tokens - 1) / tokens;
  const cudaError_t e = launch_k(paged_store_kernel, dim3(blocks), dim3(256), 0, st, nullptr, 0, p, tokens);
  return e == cudaSuccess ? ZAYA_OK : ZAYA_ERR_CUDA;
}

}  // namespace zaya
