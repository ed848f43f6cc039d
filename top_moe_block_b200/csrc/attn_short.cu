// Attention of few tokens over few keys: what attn_ragged.cu computes, without its
// pipeline, whose chain from the lengths to the first output is 10 us.
//
// A CTA per (token, key head), a group of LPK lanes per key: the group's lanes hold
// 8 to 32 bytes of a key row each, for all the query heads of the key head at once,
// in fp32, weights included.  Every group runs over its own keys (every 32nd or so)
// with a running maximum and sum, keys and values of BATCH of them on their way at a
// time; the groups are added across the warp and then over the warps in shared memory,
// in a fixed order.  Bound by latency: lengths, page ids, then a round trip and the
// products and shuffles of four keys a group, 2.7 us for 128 keys of 4 heads of 128.
// 7 packed prompts of about 73 tokens, window 32: 8.3 us against 11.6; 64 rows decoding
// over 251 keys: 10.5 us against 20.9, E4M3 10.2 against 22.9; one over 31: 6.7 against 10.1.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace zaya {

namespace {

constexpr int kWarps = 8;
// A call takes this kernel up to a number of keys that a token may see (the table's width or the
// window, the less; the lengths are on the device).  Where its CTAs fit the SMs at once, by the query
// heads of a key head: 1, 2, 4, 8 of 64, 8 of 128.  The border lies lower with few CTAs than where
// most SMs have one, since there the other kernel's query tiles are cut.  Here against the other
// kernel, us, bf16, one row: 1 head x 1000 keys 15.0 / 17.4; 2 x 500 11.7 / 16.8, x 1000 20.4 / 15.9;
// 4 x 440 13.9 / 16.4, x 570 16.5 / 15.7; 8 of 64 x 280 12.7 / 14.2; 8 of 128 x 60 9.0 / 9.7,
// x 80 10.5 / 10.0, x 280 20.8 / 15.5.  140 CTAs: 2 x 1000 25.6 / 31.2, 4 x 570 17.7 / 26.5, 8 of
// 128 x 100 12.4 / 11.7, x 180 16.4 / 20.7, x 280 21.5 / 22.6.  E4M3: ahead wherever bf16 is.
constexpr int kFewCtas[5] = {1024, 800, 560, 288, 72}, kMostCtas[5] = {1024, 1024, 576, 288, 288};
// Up to four times as many CTAs of small heads (300 rows x 120 keys of 4 heads of 64: 11.4 / 17.6,
// E4M3 11.0 / 19.6).
constexpr int kManyKeys = 128;
constexpr int kMaxPages = 1024 / 16 + 1;

// N consecutive values of a key or value row as floats.
template <int N, bool F8>
struct Piece {
  static constexpr int BYTES = N * (F8 ? 1 : 2);
  alignas(BYTES < 16 ? BYTES : 16) uint32_t u[BYTES / 4];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const uint8_t* s = static_cast<const uint8_t*>(base) + at * (F8 ? 1 : 2);
    if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(u) = __ldcg(reinterpret_cast<const uint2*>(s));
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) reinterpret_cast<uint4*>(u)[i] = __ldcg(reinterpret_cast<const uint4*>(s) + i);
    }
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float2 f;
      if (F8) {
        const uint32_t h = e4m3x2_to_f16x2((uint16_t)(u[i / 4] >> (i % 4 * 8)));
        f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      } else {
        f = unpack_bf2(u[i / 2]);
      }
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
};

// BATCH: keys of a group under way at once; one, in fewer registers, where CTAs share an SM.
template <int D, int REP, bool PAGED, bool F8, int BATCH>
__global__ void __launch_bounds__(32 * kWarps, BATCH == 1 ? 3 : 1) attn_short_kernel(const __grid_constant__ RaggedAttnParams p) {
  // dims of a lane: queries and outputs are 2 x REP x DPL registers
  constexpr int DPL = REP < 8 && (D == 128 || (F8 && (BATCH > 1 || REP < 4))) ? 16 : 8;
  constexpr int LPK = D / DPL, KPW = 32 / LPK;                // lanes of a key, keys a warp takes at once
  constexpr int ROUND = kWarps * KPW;
  __shared__ int s_row, s_bad, s_page[kMaxPages];
  __shared__ float s_max[kWarps][REP], s_sum[kWarps][REP], s_o[kWarps][REP][D];
  griddep_begin();
  const int t = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int status0 = status_peek(p.status);
  if (tid == 0) s_row = -1;
  // the token's row, and the lengths' checks
  const long long room = PAGED ? min(1LL << 30, (long long)p.max_pages << p.page_shift) : 0;
  bool bad = tid == 0 && p.cu[0] < 0;
  int mine = -1;
  for (int r = tid; r < p.B; r += 32 * kWarps) {
    const int first = p.cu[r], end = p.cu[r + 1], ctx = PAGED ? p.seq_len[r] - (end - first) : 0;
    bad |= end < first || end > p.T || (PAGED && (ctx < 0 || (long long)ctx + (end - first) > room));
    if (first <= t && t < end) mine = r;
  }
  if (tid == 0) s_bad = status0;
  bad = __syncthreads_or(bad);
  if (mine >= 0) s_row = mine;
  if (bad && tid == 0) set_status(p.status, ZAYA_ERR_DEVICE_RANGE);
  __syncthreads();
  const int b = s_row;
  if (bad || s_bad || b < 0) return;   // a fault, or a token behind the last row
  const int first = p.cu[b], n = p.cu[b + 1] - first;
  const int pos = (PAGED ? p.seq_len[b] - n : 0) + (t - first), lo = max(0, pos - p.window + 1), sh = p.page_shift;
  if (PAGED) {
    for (int i = tid; i <= (pos >> sh) - (lo >> sh); i += 32 * kWarps) {
      int id = p.block_table[(size_t)b * p.max_pages + (lo >> sh) + i];
      if ((unsigned)id >= (unsigned)p.n_pages) {
        set_status(p.status, ZAYA_ERR_DEVICE_RANGE);
        id = -1;
      }
      s_page[i] = id;
    }
  }
  const int sub = lane / LPK, d0 = lane % LPK * DPL;
  float q[REP][DPL];
  const float scale = p.scale * 1.4426950408889634f;
#pragma unroll
  for (int h = 0; h < REP; ++h) {
    Piece<DPL, false> x;
    x.load(p.q, (size_t)t * p.q_stride + (g * REP + h) * D + d0);
    x.get(q[h]);
#pragma unroll
    for (int i = 0; i < DPL; ++i) q[h][i] *= scale;
  }
  __syncthreads();
  const int keys = pos - lo + 1;
  // element offset of a key's row, or false
  auto at = [&](int i, int stride, size_t& off) -> bool {
    if (i >= keys) return false;
    const int j = lo + i;
    if (!PAGED) {
      off = (size_t)(first + j) * stride + g * D + d0;
      return true;
    }
    const int id = s_page[(j >> sh) - (lo >> sh)];
    off = ((((size_t)id * p.n_kv + g) << sh) + (j & ((1 << sh) - 1))) * D + d0;
    return id >= 0;
  };
  float m[REP], l[REP], o[REP][DPL];
#pragma unroll
  for (int h = 0; h < REP; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < DPL; ++i) o[h][i] = 0.f;
  }
#pragma unroll 1
  for (int i0 = warp * KPW + sub; i0 - (warp * KPW + sub) < keys; i0 += BATCH * ROUND) {   // the same rounds for all
    Piece<DPL, F8> k[BATCH], v[BATCH];
    bool in[BATCH];
#pragma unroll
    for (int r = 0; r < BATCH; ++r) {
      size_t off;
      in[r] = at(i0 + r * ROUND, p.k_stride, off);
      if (in[r]) k[r].load(p.k, off);
    }
#pragma unroll
    for (int r = 0; r < BATCH; ++r) {
      size_t off;
      if (at(i0 + r * ROUND, p.v_stride, off)) v[r].load(p.v, off);
    }
    float s[BATCH][REP];
#pragma unroll
    for (int r = 0; r < BATCH; ++r) {
      float x[DPL];
      k[r].get(x);
#pragma unroll
      for (int h = 0; h < REP; ++h) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < DPL; ++i) a = fmaf(q[h][i], x[i], a);
#pragma unroll
        for (int w = 1; w < LPK; w <<= 1) a += __shfl_xor_sync(0xffffffffu, a, w);
        s[r][h] = in[r] ? a : -INFINITY;
      }
    }
#pragma unroll
    for (int h = 0; h < REP; ++h) {
      float mn = m[h];
#pragma unroll
      for (int r = 0; r < BATCH; ++r) mn = fmaxf(mn, s[r][h]);
      const float f = l[h] == 0.f ? 0.f : exp2f(m[h] - mn);
      m[h] = mn;
      l[h] *= f;
#pragma unroll
      for (int i = 0; i < DPL; ++i) o[h][i] *= f;
    }
#pragma unroll
    for (int r = 0; r < BATCH; ++r) {
      if (!in[r]) continue;
      float x[DPL];
      v[r].get(x);
#pragma unroll
      for (int h = 0; h < REP; ++h) {
        const float e = s[r][h] == -INFINITY ? 0.f : exp2f(s[r][h] - m[h]);
        l[h] += e;
#pragma unroll
        for (int i = 0; i < DPL; ++i) o[h][i] = fmaf(e, x[i], o[h][i]);
      }
    }
  }
  // over the warp's key groups, then over the warps
#pragma unroll
  for (int h = 0; h < REP; ++h) {
    const float M = warp_max(m[h]);
    const float f = l[h] == 0.f ? 0.f : exp2f(m[h] - M);   // 0: no visible key (NaN counts)
    l[h] *= f;
#pragma unroll
    for (int a = LPK; a < 32; a <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], a);
#pragma unroll
    for (int i = 0; i < DPL; ++i) {
      o[h][i] *= f;
#pragma unroll
      for (int a = LPK; a < 32; a <<= 1) o[h][i] += __shfl_xor_sync(0xffffffffu, o[h][i], a);
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < DPL; ++i) s_o[warp][h][d0 + i] = o[h][i];
    }
    if (lane == 0) {
      s_max[warp][h] = M;
      s_sum[warp][h] = l[h];
    }
  }
  __syncthreads();
  for (int i = tid; i < REP * D; i += 32 * kWarps) {
    const int h = i / D, d = i % D;
    float M = -INFINITY, sum = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_max[w][h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_sum[w][h] == 0.f ? 0.f : exp2f(s_max[w][h] - M);
      sum += f * s_sum[w][h];
      y += f * s_o[w][h][d];
    }
    static_cast<__nv_bfloat16*>(p.out)[(size_t)t * p.out_stride + (g * REP + h) * D + d] = f2bf(sum != 0.f ? y / sum : 0.f);
  }
}

template <int D, int REP, int BATCH>
cudaError_t launch(const RaggedAttnParams& p, cudaStream_t st) {
  const dim3 grid(p.T, p.n_kv), block(32 * kWarps);
  if (!p.seq_len) return launch_k(attn_short_kernel<D, REP, false, false, BATCH>, grid, block, 0, st, nullptr, 0, p);
  if (p.fp8) return launch_k(attn_short_kernel<D, REP, true, true, BATCH>, grid, block, 0, st, nullptr, 0, p);
  return launch_k(attn_short_kernel<D, REP, true, false, BATCH>, grid, block, 0, st, nullptr, 0, p);
}

template <int D>
cudaError_t launch_one_wave(const RaggedAttnParams& p, cudaStream_t st) {
  switch (p.n_q / p.n_kv) {
    case 1: return launch<D, 1, 4>(p, st);
    case 2: return launch<D, 2, 4>(p, st);
    case 4: return launch<D, 4, 4>(p, st);
    default: return launch<D, 8, 2>(p, st);
  }
}

cudaError_t launch_many(const RaggedAttnParams& p, cudaStream_t st) {   // d x rep at most 256
  const int rep = p.n_q / p.n_kv;
  if (p.d == 128) return rep == 1 ? launch<128, 1, 1>(p, st) : launch<128, 2, 1>(p, st);
  return rep == 1 ? launch<64, 1, 1>(p, st) : rep == 2 ? launch<64, 2, 1>(p, st) : launch<64, 4, 1>(p, st);
}

}  // namespace

bool attn_short_fits(const RaggedAttnParams& p, int num_sms) {
  const long long len = p.seq_len ? (long long)p.max_pages << p.page_shift : p.T;
  const long long keys = len < p.window ? len : p.window, ctas = (long long)p.T * p.n_kv;
  const int rep = p.n_q / p.n_kv;
  const int heads = rep == 1 ? 0 : rep == 2 ? 1 : rep == 4 ? 2 : p.d == 64 ? 3 : 4;
  if (ctas <= num_sms) return keys <= (ctas * 8 < num_sms * 7LL ? kFewCtas : kMostCtas)[heads];
  return ctas <= 4LL * num_sms && keys <= kManyKeys && p.d * rep <= 256;
}

int launch_attn_short(const RaggedAttnParams& p, int num_sms, cudaStream_t st) {
  const bool one = (long long)p.T * p.n_kv <= num_sms;
  const cudaError_t e = !one ? launch_many(p, st) : p.d == 128 ? launch_one_wave<128>(p, st) : launch_one_wave<64>(p, st);
  return e == cudaSuccess ? ZAYA_OK : ZAYA_ERR_CUDA;
}

}  // namespace zaya
