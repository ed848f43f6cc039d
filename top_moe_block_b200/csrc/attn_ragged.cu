// Causal sliding-window grouped-query attention over ragged rows, on the
// 5th-generation tensor cores (tcgen05 + TMEM).  Each row's new tokens (a chunk
// of a prompt, a whole prompt, or one token) attend over the row's keys, which
// lie in cache pages found through a block table (bf16, or E4M3 bytes), or
// packed one row after the other.
//
//   out_i = sum_j softmax_j(scale q_i . k_j) v_j   over 0 <= p_i - j < window,
//   p_i = length - new + i, the position of the row's i-th new token.
//
// Tiles.  An MMA tile is 128 query rows: 128 / rep consecutive tokens times
// the rep query heads of one key head, so every key tile is loaded once for
// all of them, and a decoding row's rep heads share one pass over its keys.
// Key tiles are 128 keys.  A CTA works in two lanes, each a softmax warpgroup
// with its own S / P and O in tensor memory:
//   a tile of more than 128 rows: the lanes hold its two halves and share the
//     key tiles (K and V read from shared memory once per 256 query rows);
//   a tile of at most 128 rows (a decoding row): both lanes hold the same
//     queries and take the key tiles in turn; their (max, sum, O) are merged.
// While one lane's softmax runs, the tensor pipe works for the other.
//
// Work.  The (row, key head, query tile, key tile) steps of the whole call, in
// that order, weighted by what they cost, form one sequence that is cut into
// equal shares, one for each SM; the lengths are on the device, so every CTA
// finds its share itself from a scan over the rows (closed form per row).  A
// query tile cut between CTAs is finished by whichever of them comes last: the
// others have written (max, sum, O) in fp32, and the parts are added in order, so
// the result does not depend on which that was.  No CTA ever waits for another.
// One launch, whatever the lengths: balanced for one long context as for many
// short ones.
//
// Roles: warp 0 loads by TMA (Q once per query tile, K and V tiles into one
// ring, the page ids a batch ahead, a lane a box); one thread of warp 1 issues
// the MMAs; warp 2 walks the share and hands its segments to the others through a
// small ring, ahead of them (a segment's arithmetic, 1 to 3 us of 64-bit steps,
// used to sit between two segments); warps 4-7 and 8-11 are the lanes' softmax,
// a thread per query row (its TMEM lane); with E4M3 pages warps 12-15 expand the
// raw tiles in their slots (exact), K to bf16 and V to f16.
// P goes back over S, as bf16 (a weight off by up to 2^-8 of itself, while the sum
// keeps the unrounded ones) or for E4M3 pages as f16 (2^-11 of itself, or 2^-32 of the
// row's largest so far), in two halves: the first
// half's product runs while the second's exponentials are taken.  O is rescaled
// only when the running maximum grows by more than 2^8, which leaves the result
// as it is.
//
// What bounds it (times of calls in a row, 8 query and 2 key heads of 128):
//   long prompts and chunks: the lane's cycle of softmax and MMAs (tensor pipe 46 %
//     busy at 16k keys, special-function unit 46 %, about 5 cycles an
//     instruction).  8192 tokens after 24576: 0.92 to 0.98 ms (0.98 to 1.04
//     PFLOP/s; the card is at its power limit); a prompt of 4096: 59 us.
//     E4M3 pages: 1.05 ms for the chunk, 81 us for 12 ragged ones (bf16 72).
//   decoding: the HBM, once the pipe is full.  64 rows, window 4096: 61 to 64 us (4.2 to
//     4.4 TB/s with its start and end; 1.6 us a key tile between them, 6 TB/s), E4M3
//     71 us (the expansion's instructions and shared-memory traffic).
//   small calls: the chain of dependent steps (lengths, share, page ids, first
//     tile, softmax, output), 10 us for one row over 31 keys, 21 for 64 over 250
//     (128 query tiles, which 148 shares cut).
// Code size counts: with few warps and many roles, straight-line code waits for
// its instructions.  Loops over halves of a tile that read S twice beat one pass
// over all of it with S in registers (decode 65 -> 61 us, E4M3 77 -> 72 us), E4M3
// expansion one chunk at a time beats eight (105 -> 78 us).  Tried and slower:
// exponentials partly as polynomials on the FMA pipes (858 -> 1018 us at the half
// of them, chunk as above), S in halves of 64 keys by separate MMAs (846 -> 1030),
// whichever lane is ready served first (1304).
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace zaya {

namespace {

constexpr int kRows = 128;   // query rows of an MMA tile
constexpr int kKeys = 128;   // keys of a key tile
constexpr int kMaxCtas = ZAYA_ATTENTION_CLEAR / 16;   // four counters each
constexpr int kFlat = 4;     // CTAs of a query tile up to which one of them merges all
// Weight a CTA takes at least: below one short query tile's, so that short rows are not put together.
// Decoding calls with 8, 12 and 16 (us): 1 row x 31 keys 10.4, 15.1, 15.1; 1 x 1100 15.4, 18.7, 19.2;
// 4 x 300 15.5, 18.1, 20.9; 16 x 1100 18.2, 19.7, 22.3.  12 is ahead for 1 x 32768 (24.2, 22.9, 25.7) and
// 64 x 250 (20.8, 15.4, 21.7).
constexpr int kMinShare = 8;
// What a key tile costs a query tile of up to 128 rows, and of more (measured over bf16 pages with 8
// query and 2 key heads of 128: 1.6 to 1.9 us, bound by the loads, against 2.3; used for every head
// and page type); and what a query tile costs beside its key tiles.
constexpr int kKeyCost = 3, kKeyCostTwo = 4, kTileCost = 6;
constexpr int kSegs = 4;     // ring of segments
constexpr float kRescaleLog2 = 8.0f;
// Up to this maximum (in log2) the exponent is one fma of the logit: the product
// is not rounded, so its distance from the rounded maximum is off by up to 2^-24
// of the maximum, 2^-8 here.  Beyond it both are rounded alike.
constexpr float kFusedMax = 65536.0f;
// E4M3 pages: the running maximum is kept this far below the true one, so that the f16 weights lie
// between 2^-24 and 2^(8 + 7) of it.  With its top at 1, weights under 2^-25 of the largest came to
// nothing while the sum counted them: under one strong key, half of what 4000 others hold was lost.
constexpr float kHeadroom = 7.0f;
constexpr int kCvtWarps = 2;   // warps that expand an E4M3 tile together
constexpr int kNoBox = -1;
constexpr int kMaxLen = 1 << 30;   // keys of a row

template <int D, bool F8>
struct Cfg {
  static constexpr int SUB = D / 64;                   // 64-wide swizzle atoms along d
  static constexpr int ATOM = 128 * 128;               // [128 rows][64] bf16
  static constexpr int TILE = SUB * ATOM;              // Q, K or V tile
  // An E4M3 tile lands in its slot and is expanded in place: for d = 128 its rows
  // lie where the second half of the bf16 rows goes; for d = 64 behind the tile.
  static constexpr int RAW_OFF = D == 128 ? ATOM : TILE;
  static constexpr int SLOT = TILE + (F8 && D == 64 ? kKeys * D : 0);
  static constexpr int RING = D == 128 ? 5 : 8;
  // Barriers of the raw tiles, position p's at p % RAWS.  A parity wait tells a phase from its neighbours
  // only, so whoever waits at p must have seen p - RAWS land.  The two expanding groups take positions in
  // turn: with an odd ring and a barrier a slot, the slot's last use is the other group's, and a copy
  // that overtakes others would let a tile be expanded before it is there.
  static constexpr int RAWS = RING % 2 ? 2 * RING : RING;
  static constexpr int FULLS = F8 ? RAWS : RING;       // barriers that the copies arrive on
  static constexpr int WARPS = F8 ? 16 : 12;
  static constexpr int THREADS = 32 * WARPS;
  // registers: the launch gives every thread 168 (E4M3: 128); the first warpgroup
  // hands some of its own to the softmax (the sum stays at or below the launch's)
  static constexpr int REGS_IO = F8 ? 72 : 80;
  static constexpr int REGS_CVT = 88;
  static constexpr int REGS_SOFTMAX = F8 ? 176 : 208;
  static_assert(kFlat == 4, "the merge in tensor memory takes up to four parts");
  static_assert(F8 ? REGS_IO + REGS_CVT + 2 * REGS_SOFTMAX <= 4 * 128 : REGS_IO + 2 * REGS_SOFTMAX <= 3 * 168, "registers");
  static constexpr int SMEM = 1024 + 2 * TILE + RING * SLOT + 768;
  static_assert(SMEM <= 232448 - 1024, "shared memory");
  static constexpr uint32_t IDESC_QK = idesc_bf16_f32(kRows, kKeys);
  // E4M3: P and V in f16, which V's codes fit as they are (A and B type fields 0: f16)
  static constexpr uint32_t IDESC_PV = F8 ? idesc_bf16_f32_bmn(kRows, D) & ~((1u << 7) | (1u << 10)) : idesc_bf16_f32_bmn(kRows, D);
  static constexpr uint32_t S_COL = 0, O_COL = 256;    // lane x: S at 128 x, O at 256 + 128 x
};

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Pairs of floats, two operations an instruction.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// A 3-D tensor-map box into shared memory.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Two E4M3 bytes as a bf16 pair, exactly (through f16, which holds every code, NaN too).
__device__ __forceinline__ uint32_t e4m3x2_to_bf2(uint16_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf2(f.x, f.y);
}

// ------------------------------------------------------------------ the sequence of steps
__device__ __forceinline__ long long div_pos(long long a, long long b) {   // a >= 0, b > 0
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// sum over i < m of floor((a + i * 2^tsh) / 128), a >= 0
__device__ __forceinline__ long long floor_sum(int a, int m, int tsh) {
  if (m <= 0) return 0;
  if (tsh >= 7) return (long long)m * (a >> 7) + (((long long)m * (m - 1) / 2) << (tsh - 7));
  const int R = 1 << (7 - tsh);
  long long s = 0;
  for (int r = 0; r < R && r < m; ++r) {
    const long long c = (m - r + R - 1) >> (7 - tsh);   // i = r, r + R, ...
    s += c * ((a + (r << tsh)) >> 7) + c * (c - 1) / 2;
  }
  return s;
}

// One row of the call: n new tokens after ctx cached ones, in m query tiles of
// up to 2^tsh tokens (256 query rows).
struct Row {
  int first, n, ctx, m;
};

// Query tile i of a row.
struct QTile {
  int tok0, ntok;   // its tokens within the row
  int two;          // more than 128 query rows
  int lo, hi;       // keys some token of the tile sees
  int kb, nt;       // first key tile, key tiles
};

struct Steps {
  int window, tsh;
  __device__ __forceinline__ QTile tile(const Row& r, int i) const {
    QTile t;
    t.tok0 = i << tsh;
    t.ntok = min(1 << tsh, r.n - t.tok0);
    t.two = t.ntok > (1 << (tsh - 1));
    t.hi = r.ctx + t.tok0 + t.ntok;
    t.lo = max(0, r.ctx + t.tok0 - window + 1);
    t.kb = t.lo >> 7;
    t.nt = ((t.hi - 1) >> 7) - t.kb + 1;
    return t;
  }
  // key tiles of the first i query tiles, all of them full
  __device__ __forceinline__ long long before(const Row& r, int i) const {
    const int c0 = r.ctx - window + 1;   // lo of tile i' is max(0, c0 + i' * 2^tsh)
    const int i0 = c0 >= 0 ? 0 : (int)(((long long)-c0 + (1 << tsh) - 1) >> tsh);
    return floor_sum(r.ctx + (1 << tsh) - 1, i, tsh) - (i > i0 ? floor_sum(c0 + (i0 << tsh), i - i0, tsh) : 0) + i;
  }
  // weight of a row's first i query tiles
  __device__ __forceinline__ long long weight_before(const Row& r, int i) const { return kKeyCostTwo * before(r, i) + (long long)i * kTileCost; }
  // weight of a row for one key head
  __device__ __forceinline__ long long weight(const Row& r) const {
    if (r.m == 0) return 0;
    const QTile t = tile(r, r.m - 1);
    return (r.m > 1 ? weight_before(r, r.m - 1) : 0) + kTileCost + (long long)t.nt * (t.two ? kKeyCostTwo : kKeyCost);
  }
};

// What the roles need of a segment, the part of one query tile that falls into a
// CTA's share: key tiles kt0 .. kt0 + n - 1.  n = 0 ends the share.
struct Seg {
  int tok, ntok, pos0;   // the query tile's first token, tokens, and its first position
  int lo, hi;            // keys some of them see
  int kt0, n, two;
  int g, b, first;       // key head, row, the row's first token
  int cf, cl;            // first and last CTA of the query tile
};

// A CTA's place in the sequence.
struct Walk {
  const RaggedAttnParams* p;
  Steps st;
  long long q, r;            // shares: q steps, one more for the first r CTAs
  long long lo, hi;          // this CTA's
  int b, g, i;               // position
  Row row;
  long long start;           // weight before the current query tile

  __device__ __forceinline__ Row load(int x) const {
    Row y;
    y.first = p->cu[x];
    y.n = p->cu[x + 1] - y.first;
    y.ctx = p->seq_len ? p->seq_len[x] - y.n : 0;
    y.m = (y.n + (1 << st.tsh) - 1) >> st.tsh;
    return y;
  }
  __device__ __forceinline__ int owner(long long u) const {
    const long long head = r * (q + 1);
    return (int)(u < head ? div_pos(u, q + 1) : r + div_pos(u - head, q));
  }
  // from row r0, whose steps begin at weight base (base <= lo) and weigh w for one key head
  __device__ __forceinline__ void begin(int r0, long long base, long long w) {
    b = r0;
    row = load(b);
    const long long off = lo - base;
    g = (int)div_pos(off, w);
    const long long rest = off - (long long)g * w;
    long long before = 0;
    int a = 0, e = row.m;   // the largest i in [a, e) with weight_before(i) <= rest, 32 tries at a time
    while (e - a > 1) {
      const int step = (e - a + 31) / 32;
      const int at = a + lane_id() * step;
      const long long w_at = st.weight_before(row, at);
      const int n = __popc(__ballot_sync(0xffffffffu, at < e && w_at <= rest));   // at least lane 0's
      before = __shfl_sync(0xffffffffu, w_at, n - 1);
      a += (n - 1) * step;
      e = min(e, a + step);
    }
    i = a;
    start = base + (long long)g * w + before;
  }
  // The segment at the current position, which moves on to the next query tile;
  // n = 0 behind the share's end.
  __device__ __forceinline__ Seg next() {
    Seg s;
    s.n = 0;
    while (start < hi && s.n == 0) {
      const QTile t = st.tile(row, i);
      const int w = t.two ? kKeyCostTwo : kKeyCost;
      const long long keys = start + kTileCost, end = keys + (long long)t.nt * w;
      // a key tile is the CTA's whose share has its first step
      const int k0 = lo > keys ? (int)div_pos(lo - keys + w - 1, w) : 0;
      const int k1 = end > hi ? (int)div_pos(max(0LL, hi - keys + w - 1), w) : t.nt;
      s.tok = row.first + t.tok0; s.ntok = t.ntok; s.pos0 = row.ctx + t.tok0;
      s.lo = t.lo; s.hi = t.hi; s.kt0 = t.kb + k0; s.n = max(0, k1 - k0); s.two = t.two;
      s.g = g; s.b = b; s.first = row.first;
      s.cf = lo > keys ? owner(keys) : blockIdx.x;   // of the first key tile's first step
      s.cl = end > hi ? owner(end - w) : blockIdx.x;   // of the last key tile's first step
      start = end;
      if (++i == row.m) {
        i = 0;
        if (++g == p->n_kv) {
          g = 0;
          if (start < hi) {
            do row = load(++b);
            while (row.m == 0);   // a share that goes on has a row that does
          }
        }
      }
    }
    return s;
  }
};

// Ring positions of a segment of n key tiles: K(0), then K(j + 1) (if there is
// one) and V(j) for every j.
__device__ __forceinline__ uint32_t pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t pos_v(int j, int n) { return min(2 * j + 2, 2 * n - 1); }

// The ring of segments, seen by one of its readers (a warp).
struct SegRing {
  const Seg* segs;
  uint64_t *full, *empty;
  uint32_t at;
  __device__ __forceinline__ bool next(Seg& s, const WaitCtx& wc) {
    const uint32_t slot = at % kSegs;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], (at / kSegs) & 1, wc))) return false;
    s = segs[slot];
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&empty[slot]);
    ++at;
    return s.n != 0;
  }
};

// A list of partial results of one query tile: CTA c = c0 + (i >> nzl) * step, lane z0 (+ i & 1).
struct Parts {
  const float* o;    // [sub][D / 4][128 rows][4]
  const float* ml;   // [sub][max | sum][128 rows]
  int c0, step, cf, whole_slot;   // whole_slot >= 0: the slot of a tile that one CTA holds
  int n, z0, nzl;   // nzl: log2 of the lanes a CTA has in the list
  __device__ __forceinline__ int sub(int i) const {
    const int c = c0 + (i >> nzl) * step;
    // slots: 2 c for the tile a CTA goes on with, 2 c + 1 for the one it leaves to the next
    const int slot = whole_slot >= 0 ? whole_slot : c > cf ? 2 * c : 2 * c + 1;
    return slot * 2 + z0 + (i & nzl);
  }
};

// Loads that stay where they are written, ahead of the branches behind them.
__device__ __forceinline__ float ld_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cg4(const float* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// One thread's columns (float4 col + k * stride) of row rr over parts i0, i0 + di, ..
// in order: acc, the maximum M and the sum L.
template <int D, int COLS, int U>
__device__ __forceinline__ void merge_cols(const Parts& ps, int rr, int col, int stride, int i0, int di, float4 (&acc)[COLS],
                                           float& M, float& L) {
  M = -INFINITY;
  L = 0.f;
#pragma unroll
  for (int k = 0; k < COLS; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1   // run once or twice a launch: less code to fetch
  for (int i = i0; i < ps.n; i += di * U) {
    float m[U], l[U];
    float4 o[U][COLS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = i + u * di < ps.n;
      const int sb = ps.sub(in ? i + u * di : i);
      const float* ml = ps.ml + (size_t)sb * 2 * kRows + rr;
      m[u] = ld_cg(ml);
      l[u] = ld_cg(ml + kRows);
      if (!in) l[u] = 0.f;
      const float* src = ps.o + (size_t)sb * kRows * D + rr * 4;
#pragma unroll
      for (int k = 0; k < COLS; ++k) o[u][k] = ld_cg4(src + (size_t)(col + k * stride) * kRows * 4);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (l[u] == 0.f) continue;   // no visible key in this part (NaN counts), or none at all
      const float Mn = fmaxf(M, m[u]);
      const float f = L == 0.f ? 0.f : ex2_approx(M - Mn), w = ex2_approx(m[u] - Mn);
      M = Mn;
      L = L * f + w * l[u];
#pragma unroll
      for (int k = 0; k < COLS; ++k) {
        acc[k].x = fmaf(w, o[u][k].x, acc[k].x * f);
        acc[k].y = fmaf(w, o[u][k].y, acc[k].y * f);
        acc[k].z = fmaf(w, o[u][k].z, acc[k].z * f);
        acc[k].w = fmaf(w, o[u][k].w, acc[k].w * f);
      }
    }
  }
}

// Merges a list over `live` rows with the 256 softmax threads.  Rows side by
// side (their float4s are neighbours in memory); with few rows, the threads left
// over share the list and add up across lanes.  done(row, column, value, M, L).
template <int D, class F>
__device__ __forceinline__ void merge_parts(const Parts& ps, int live, int st_id, F&& done) {
  int rp = 1;   // rows side by side: a power of two
  while (rp < live) rp <<= 1;
  const int combos = rp * (D / 4);
  if (combos <= 256) {
    const int ng = 256 / combos, g = st_id & (ng - 1), idx = st_id / ng, rr = idx & (rp - 1), col = idx / rp;
    const int row = min(rr, live - 1);   // every lane takes part in the shuffles
    float4 a[1];
    float M, L;
    merge_cols<D, 1, 4>(ps, row, col, 0, g, ng, a, M, L);
    for (int o = 1; o < ng; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
      float4 b;
      b.x = __shfl_xor_sync(0xffffffffu, a[0].x, o);
      b.y = __shfl_xor_sync(0xffffffffu, a[0].y, o);
      b.z = __shfl_xor_sync(0xffffffffu, a[0].z, o);
      b.w = __shfl_xor_sync(0xffffffffu, a[0].w, o);
      const float Mn = fmaxf(M, m2);
      const float f = L == 0.f ? 0.f : ex2_approx(M - Mn), w = l2 == 0.f ? 0.f : ex2_approx(m2 - Mn);
      M = Mn;
      L = L * f + l2 * w;
      a[0] = make_float4(a[0].x * f + b.x * w, a[0].y * f + b.y * w, a[0].z * f + b.z * w, a[0].w * f + b.w * w);
    }
    if (g == 0 && rr < live) done(rr, col, a[0], M, L);
  } else {
    const int rr = st_id & (rp - 1), stride = 256 / rp;
    if (rr >= live) return;
    int col = st_id / rp;
    if (combos >= 256 * 8) {
      for (; col < D / 4; col += 8 * stride) {
        float4 a[8];
        float M, L;
        merge_cols<D, 8, 2>(ps, rr, col, stride, 0, 1, a, M, L);
#pragma unroll
        for (int k = 0; k < 8; ++k) done(rr, col + k * stride, a[k], M, L);
      }
    } else {
      for (; col < D / 4; col += 2 * stride) {
        float4 a[2];
        float M, L;
        merge_cols<D, 2, 4>(ps, rr, col, stride, 0, 1, a, M, L);
#pragma unroll
        for (int k = 0; k < 2; ++k) done(rr, col + k * stride, a[k], M, L);
      }
    }
  }
}

template <int D, bool PAGED, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::THREADS, 1)
    attn_ragged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ RaggedAttnParams p) {
  using C = Cfg<D, F8>;
  constexpr int RING = C::RING;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                        // [2] Q tiles
  uint8_t* sKV = sQ + 2 * C::TILE;           // [RING] K / V tiles
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + RING * C::SLOT);
  uint64_t* q_full = bars;                   // [2]
  uint64_t* q_empty = q_full + 2;            // [2]
  uint64_t* kv_full = q_empty + 2;           // [RING]
  uint64_t* kv_empty = kv_full + RING;       // [RING]
  uint64_t* s_full = kv_empty + RING;        // [2] S of the lane's next key tile is there (and its last PV done)
  uint64_t* p_full = s_full + 2;             // [2][2] lane, half: P is over it
  uint64_t* o_full = p_full + 4;             // [2] O of the segment is complete
  uint64_t* o_free = o_full + 2;             // [2] and has been read
  uint64_t* seg_full = o_free + 2;           // [kSegs]
  uint64_t* seg_empty = seg_full + kSegs;    // [kSegs]
  uint64_t* sm_sync = seg_empty + kSegs;     // the softmax warps among themselves
  uint64_t* mdrain = sm_sync + 1;            // the MMA thread's last commit
  uint64_t* raw_full = mdrain + 1;           // [RAWS] E4M3 bytes are there
  Seg* segs = reinterpret_cast<Seg*>(raw_full + (F8 ? C::RAWS : 0));   // [kSegs]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(segs + kSegs);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 1);
  __shared__ long long s_sum[C::WARPS], s_base, s_weight;
  __shared__ int s_row, s_skip;

  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  if (warp == 0 && lane == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&p_full[2 * x + h], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_free[x], 4);
    }
    for (int s = 0; s < RING; ++s) {
      mbar_init(&kv_full[s], F8 ? kCvtWarps : 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; F8 && s < C::RAWS; ++s) mbar_init(&raw_full[s], 1);
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], C::WARPS - 2);   // every warp but the walker and the idle one
    }
    mbar_init(sm_sync, 8);
    mbar_init(mdrain, 1);
    fence_barrier_init();
    fence_proxy_async();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_begin();   // the prologue above overlaps the previous kernel; global memory only from here

  // ---------------- the share: a scan of the rows' weights
  // the header's loads under way while the rows' are
  const int status0 = status_peek(p.status);
  const uint64_t limit0 = *reinterpret_cast<const volatile uint64_t*>(p.status + 2);
  Walk wk;
  wk.p = &p;
  wk.st = Steps{p.window, 8 - p.rep_shift};
  const int c = blockIdx.x;
  const int per = (p.B + C::THREADS - 1) / C::THREADS;
  const int r0 = min(p.B, tid * per);
  int r1 = min(p.B, r0 + per);
  long long mine = 0, base = 0;
  bool bad = tid == 0 && p.cu[0] < 0, work = false;
  WaitCtx wc;
  const long long room = PAGED ? min((long long)kMaxLen, (long long)p.max_pages << p.page_shift) : 0;
  // first the weights, then, in the thread whose rows hold the share's first step, that row
  // (one loop for both: code that runs once costs its fetch)
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += a;
      }
      if (lane == 31) s_sum[warp] = inc;
      if (tid == 0) s_skip = status0 != 0;   // one reading for the whole CTA
      bad = __syncthreads_or(bad);
      wc = wait_ctx(p.status, status0, limit0);
      if (bad && tid == 0) set_status(p.status, ZAYA_ERR_DEVICE_RANGE);
      long long sums = lane < C::WARPS ? s_sum[lane] : 0;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += a;
      }
      const long long total = __shfl_sync(0xffffffffu, sums, 15);
      base = inc - mine + (warp > 0 ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
      const int G = (int)max(1LL, min((long long)gridDim.x, total / kMinShare));
      work = !bad && !s_skip && total > 0 && c < G;   // the same for every thread of the CTA
      if (!work) break;
      wk.q = div_pos(total, G);
      wk.r = total - wk.q * G;
      wk.lo = c * wk.q + min((long long)c, wk.r);
      wk.hi = wk.lo + wk.q + (c < wk.r ? 1 : 0);
      if (wk.lo < base || wk.lo >= base + mine) r1 = r0;
    }
    for (int r = r0; r < r1; ++r) {
      const Row x = wk.load(r);
      const bool off = x.n < 0 || p.cu[r + 1] > p.T || (PAGED && (x.ctx < 0 || (long long)x.ctx + x.n > room));
      const long long w = off ? 0 : wk.st.weight(x);
      bad |= off;
      if (pass == 0) {
        mine += w * p.n_kv;
      } else if (wk.lo < base + w * p.n_kv) {
        s_row = r;
        s_base = base;
        s_weight = w;
        break;
      } else {
        base += w * p.n_kv;
      }
    }
  }
  __syncthreads();
  SegRing ring{segs, seg_full, seg_empty, 0};
  Seg sg;

  if (warp < 4) {
    regs_dec<C::REGS_IO>();
    if (!work) {
    } else if (warp == 2) {
      // ---------------- the walk
      wk.begin(s_row, s_base, s_weight);
      uint32_t at = 0;
      bool more = true;
      while (more) {
        const Seg s = wk.next();
        more = s.n != 0;
        const uint32_t slot = at % kSegs;
        if (!__all_sync(0xffffffffu, mbar_wait(&seg_empty[slot], ((at / kSegs) & 1) ^ 1u, wc))) break;
        if (lane == 0) {
          segs[slot] = s;
          mbar_arrive(&seg_full[slot]);
        }
        ++at;
      }
    } else if (warp == 0) {
      // ---------------- TMA: Q once per segment, K and V tiles through the ring (the whole warp, a box a lane)
      uint32_t pos = 0;
      uint32_t q_use[2] = {0, 0};
      int half = 0;
      bool ok = true;
      uint64_t* full = F8 ? raw_full : kv_full;
      const int P = 1 << p.page_shift;
      const int box = PAGED ? min(P, kKeys) : kKeys;        // rows of a box
      const int n_box = kKeys / box;                        // boxes of a key tile (per 64 columns)
      const int my_box = lane % n_box, my_sub = lane / n_box, batch = 32 / n_box;
      constexpr int SUBS = F8 ? 1 : C::SUB;                 // an E4M3 row is one box wide
      constexpr int ROW = F8 ? D : 128;                     // bytes of a box's row
      const bool loads = my_sub < SUBS;
      while (ok && ring.next(sg, wc)) {
        for (int x = 0; ok && x <= sg.two; ++x) {   // Q
          const int h = half ^ x;
          ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[h], (q_use[h] & 1) ^ 1u, wc));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[h], C::TILE);
            for (int s = 0; s < C::SUB; ++s)
              tma_load_3d(sQ + h * C::TILE + s * C::ATOM, &tmQ, &q_full[h], s * 64, sg.g << p.rep_shift,
                          sg.tok + (x << (wk.st.tsh - 1)));
          }
          ++q_use[h];
        }
        if (!sg.two) half ^= 1;
        // Page ids, a lane a box, `batch` key tiles at a time; kNoBox: no token of the query
        // tile sees any of the box, which is not loaded.
        auto pages = [&](int j0) -> int {
          const int j = j0 + lane / n_box, key = ((sg.kt0 + j) << 7) + (lane % n_box) * box;
          if (j >= sg.n || key >= sg.hi || key + box <= sg.lo) return kNoBox;
          if (!PAGED) return 0;
          const int id = p.block_table[(size_t)sg.b * p.max_pages + (key >> p.page_shift)];
          if ((unsigned)id < (unsigned)p.n_pages) return id;
          set_status(p.status, ZAYA_ERR_DEVICE_RANGE);
          return kNoBox;
        };
        int ids = pages(0), ids_more = sg.n > batch ? pages(batch) : kNoBox, j_ids = 0;
        // this lane's page of key tile j (called for each j once, in order)
        auto page_of = [&](int j) -> int {
          if (j == j_ids + batch) {
            j_ids = j;
            ids = ids_more;
            if (j + batch < sg.n) ids_more = pages(j + batch);
          }
          const int id = __shfl_sync(0xffffffffu, ids, (j - j_ids) * n_box + my_box);
          return loads ? id : kNoBox;
        };
        int id_next = page_of(0);
        // one K or V tile, a box a lane
        auto load = [&](const CUtensorMap* map, int j, int page) -> bool {
          const uint32_t slot = pos % RING;
          if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[slot], ((pos / RING) & 1) ^ 1u, wc))) return false;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, page != kNoBox));
          uint64_t* landed = &full[pos % C::FULLS];
          if (lane == 0) mbar_arrive_expect_tx(landed, boxes * (uint32_t)(box * ROW));
          __syncwarp();
          if (page != kNoBox) {
            uint8_t* dst = sKV + slot * C::SLOT + (F8 ? C::RAW_OFF : my_sub * C::ATOM) + my_box * box * ROW;
            const int key = ((sg.kt0 + j) << 7) + my_box * box;
            if (PAGED) tma_load_3d(dst, map, landed, my_sub * 64, (sg.g << p.page_shift) + (key & (P - 1)), page);
            else tma_load_3d(dst, map, landed, my_sub * 64, sg.g, sg.first + key);
          }
          ++pos;
          return true;
        };
        ok = ok && load(&tmK, 0, id_next);
        for (int j = 0; ok && j < sg.n; ++j) {
          const int id = id_next;
          if (j + 1 < sg.n) {
            id_next = page_of(j + 1);
            ok = load(&tmK, j + 1, id_next);
          }
          ok = ok && load(&tmV, j, id);
        }
      }
      // every copy started must land before the CTA may exit
      for (int h = 0; h < 2; ++h)
        if (q_use[h]) mbar_drain(&q_full[h], (q_use[h] - 1) & 1, p.status);
      for (uint32_t q = pos > RING ? pos - RING : 0; q < pos; ++q) mbar_drain(&full[q % C::FULLS], (q / C::FULLS) & 1, p.status);
    } else if (warp == 1) {
      // ---------------- MMA issuer: one thread (the warp reads the segments together)
      const bool leader = elect_one();
      // P comes in halves of 64 keys: the first's product runs while the softmax
      // works on the second, and S of the lane's next key tile (which takes P's
      // place) waits for the second's product alone.
      uint32_t base_pos = 0, q_use0 = 0, q_use1 = 0, tiles0 = 0, tiles1 = 0, o_cnt0 = 0, o_cnt1 = 0;
      int half = 0;
      bool ok = true;
      while (ok && ring.next(sg, wc)) {
        if (leader) {
          const int n = sg.n, two = sg.two;
          // S of key tile j for lane x (a constant at every call)
          auto qk = [&](int x, int j) -> bool {
            const uint32_t pk = base_pos + pos_k(j), slot = pk % RING;
            const int qh = two ? half ^ x : half;
            if (j == 0 && !mbar_wait(&q_full[qh], (qh ? q_use1 : q_use0) & 1, wc)) return false;   // the first use of a Q tile
            if ((!two || x == 0) && !mbar_wait(&kv_full[slot], (pk / RING) & 1, wc)) return false;
            tc_fence_after();
            const uint32_t qa = smem_u32(sQ + qh * C::TILE), ka = smem_u32(sKV + slot * C::SLOT);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::ATOM + (kk & 3) * 32;
              tc_mma_bf16(tmem_base + C::S_COL + x * 128, smem_desc_sw128(qa + off, 16, 1024),
                          smem_desc_sw128(ka + off, 16, 1024), C::IDESC_QK, kk > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[x]);
            if (!two || x == 1) tc_commit(&kv_empty[slot]);
            if (j == n - 1) {   // the last use
              tc_commit(&q_empty[qh]);
              if (qh) ++q_use1;
              else ++q_use0;
            }
            return true;
          };
          // O of lane x += P V over half h of key tile j
          auto pv = [&](int x, int j, int h) -> bool {
            const uint32_t p_v = base_pos + pos_v(j, n), slot = p_v % RING;
            const bool first = h == 0 && j == (two ? 0 : x);   // the lane's first product of the segment overwrites O
            if (h == 0 && (!two || x == 0) && !mbar_wait(&kv_full[slot], (p_v / RING) & 1, wc)) return false;
            if (!mbar_wait(&p_full[2 * x + h], (x ? tiles1 : tiles0) & 1, wc)) return false;
            if (first) {
              if (!mbar_wait(&o_free[x], ((x ? o_cnt1 : o_cnt0) & 1) ^ 1u, wc)) return false;
              if (x) ++o_cnt1;
              else ++o_cnt0;
            }
            tc_fence_after();
            const uint32_t va = smem_u32(sKV + slot * C::SLOT) + h * 4 * 2048, pa = tmem_base + C::S_COL + x * 128 + h * 64;
#pragma unroll
            for (int kk = 0; kk < kKeys / 32; ++kk)
              tc_mma_bf16_ts(tmem_base + C::O_COL + x * 128, pa + kk * 8, smem_desc_sw128(va + kk * 2048, C::ATOM, 1024),
                             C::IDESC_PV, (!first || kk > 0) ? 1u : 0u);
            if (h == 1) {
              if (!two || x == 1) tc_commit(&kv_empty[slot]);
              if (x) ++tiles1;
              else ++tiles0;
            }
            return true;
          };
          // key tile j of lane x, and S of the lane's next
          auto step = [&](int x, int j, int next) -> bool {
            if (!pv(x, j, 0) || !pv(x, j, 1)) return false;
            if (next < n) return qk(x, next);
            tc_commit(&o_full[x]);
            return true;
          };
          if (two) {
            ok = qk(0, 0) && qk(1, 0);
            for (int j = 0; ok && j < n; ++j) ok = step(0, j, j + 1) && step(1, j, j + 1);
          } else {
            ok = qk(0, 0) && (n == 1 || qk(1, 1));
            for (int j = 0; ok && j < n; j += 2) ok = step(0, j, j + 2) && (j + 1 == n || step(1, j + 1, j + 3));
          }
          base_pos += 2 * n;
          if (!two) half ^= 1;
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (leader) {
        tc_commit(mdrain);   // on every path: arrives once every MMA above is done
        mbar_drain(mdrain, 0, p.status);
      }
    }
  } else if (warp < 12) {
    regs_inc<C::REGS_SOFTMAX>();
    // ---------------- softmax: lane x of the CTA, a thread per query row
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int qrow = quarter * 32 + lane;
    const uint32_t tl = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tS = tl + C::S_COL + x * 128, tO = tl + C::O_COL + x * 128;
    const float sl2 = p.scale * 1.4426950408889634f;
    const int rsh = p.rep_shift, tokens_half = 1 << (7 - rsh);
    const int st_id = (warp - 4) * 32 + lane;
    float* part = static_cast<float*>(p.part);
    float* part_ml = part + (size_t)gridDim.x * 6 * kRows * D;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && p.out_stride % 16 == 0;   // 32-byte stores
    uint32_t s_cnt = 0, o_cnt = 0, base_pos = 0, sync_cnt = 0;   // key tiles, segments, ring positions, barriers so far
    // all eight softmax warps; false when the wait ran out, and the warp leaves
    auto sync_all = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(sm_sync);
      const bool got = __all_sync(0xffffffffu, mbar_wait(sm_sync, sync_cnt & 1, wc));
      ++sync_cnt;
      return got;
    };
    // Who comes last of `n` at a counter (left zero)?  What the CTA's softmax threads
    // wrote before is visible to the one that does, and the others' writes to all its threads.
    auto last_of = [&](int* ctr, int n, bool& last) -> bool {
      if (!sync_all()) return false;
      if (st_id == 0) {
        __threadfence();
        *s_last = atomicInc(reinterpret_cast<unsigned*>(ctr), (unsigned)(n - 1)) == (unsigned)(n - 1);
        __threadfence();
      }
      if (!sync_all()) return false;
      last = *s_last != 0;
      return true;
    };
    while (work && ring.next(sg, wc)) {
      const int n = sg.n, two = sg.two;
      const int nx = two ? n : (n - x + 1) >> 1;   // this lane's key tiles
      const int half0 = two ? x * tokens_half : 0;
      const int t_w0 = half0 + ((quarter * 32) >> rsh), t_w1 = half0 + ((quarter * 32 + 31) >> rsh);   // the warp's tokens
      const int tok = half0 + (qrow >> rsh);
      const int pos = sg.pos0 + tok;
      const bool valid = tok < sg.ntok;
      const bool dead = t_w0 >= sg.ntok;   // none of the warp's rows is a token's
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      for (int k = 0; k < nx; ++k) {
        const int j = two ? k : 2 * k + x;
        const int key0 = (sg.kt0 + j) << 7;
        // every wait that guards a .sync.aligned TMEM access is made warp-uniform
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x], s_cnt & 1, wc));
        if (!ok) break;
        ++s_cnt;
        tc_fence_after();
        if (!F8 && (!two || x == 0) && (key0 < sg.lo || key0 + kKeys > sg.hi)) {
          // values of keys no token of the tile sees may be anything (not loaded, behind the row's
          // end): zero, so that their zero weights count; the MMA waits for all four warps' P, and takes
          // the lanes' key tiles in order
          const uint32_t p_v = base_pos + pos_v(j, n), slot = p_v % RING;
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[slot], (p_v / RING) & 1, wc));
          if (!ok) break;
          const int key = key0 + qrow;
          if (key < sg.lo || key >= sg.hi) {
            uint8_t* v = sKV + slot * C::SLOT + qrow * 128;
#pragma unroll
            for (int s = 0; s < C::SUB; ++s)
#pragma unroll
              for (int q = 0; q < 8; ++q) reinterpret_cast<uint4*>(v + s * C::ATOM)[q] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        // P's first half is handed over before the second is begun
        auto hand = [&](int h) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + h]);
        };
        if (dead) {
          hand(0);
          hand(1);
          continue;
        }
        // Both passes run over halves of 64 keys, as loops, and read S from tensor memory each time:
        // half the registers and half the code of one pass over all 128.
        const int e = pos - key0, a = e - p.window;   // visible: a < i <= e
        const bool behind = key0 + kKeys - 1 > sg.pos0 + t_w0, left = sg.pos0 + t_w1 - key0 >= p.window;   // of some token of the warp
        auto load = [&](int h, float (&v)[64]) {
          tmem_ld32(tS + h * 64, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_ld32(tS + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tmem_ld_wait();
          if (behind) {
            const int hi = e - h * 64;
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = i <= hi ? v[i] : -INFINITY;
          }
          if (left) {
            const int lo = a - h * 64;
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = i > lo ? v[i] : -INFINITY;
          }
        };
        float tmax = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float v[64];
          load(h, v);
          float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int i = 4; i < 60; i += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], v[i + q], v[i + 4 + q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], v[60 + q]);
          tmax = fmaxf(max3(mx[0], mx[1], tmax), fmaxf(mx[2], mx[3]));
        }
        // a NaN logit is no maximum, and spoils the sum below
        const float top = tmax * sl2, m_new = fmaxf(m_used, F8 && fabsf(top) < kFusedMax ? top - kHeadroom : top);
        // move the running maximum when it grew by more than 2^8, the whole
        // warp at once (the rescale is a warp-wide TMEM access); rows of no token, whose
        // logits may come from whatever lies behind the row's keys, have no say
        if (__any_sync(0xffffffffu, valid && m_new - m_used > kRescaleLog2)) {   // the difference is exact, a sum would not be
          const bool finite_new = m_new != -INFINITY;
          const float f = (m_used == -INFINITY || !finite_new) ? 1.f : exp2f(m_used - m_new);
          if (k > 0 && __any_sync(0xffffffffu, m_used != -INFINITY)) {
            // O is complete up to the last key tile: S was issued behind its PV
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + q * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(tO + q * 32, o);
            }
          }
          l *= f;
          if (finite_new) m_used = m_new;
        }
        const float nb = (m_used == -INFINITY) ? 0.f : -m_used;
        const bool apart = __any_sync(0xffffffffu, valid && fabsf(nb) > kFusedMax);
        const uint64_t s2 = apart ? f2(1.f, 1.f) : f2(sl2, sl2), b2 = apart ? f2(0.f, 0.f) : f2(nb, nb);
        uint64_t ls[2] = {0, 0};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float v[64];
          load(h, v);
          if (apart) {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = __fadd_rn(__fmul_rn(v[i], sl2), nb);
          }
#pragma unroll
          for (int i = 0; i < 64; i += 2) unf2(fma2(f2(v[i], v[i + 1]), s2, b2), v[i], v[i + 1]);
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = ex2_approx(v[i]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float x = v[q * 32 + i], y = v[q * 32 + i + 1];
              pk[i >> 1] = F8 ? pack_h2(x, y) : pack_bf2(x, y);
            }
            tmem_st16(tS + h * 64 + q * 16, pk);
          }
#pragma unroll
          for (int i = 0; i < 64; i += 2) ls[(i >> 1) & 1] = add2(ls[(i >> 1) & 1], f2(v[i], v[i + 1]));
          tmem_st_wait();
          hand(h);
        }
        float la, lb;
        unf2(add2(ls[0], ls[1]), la, lb);
        l += la + lb;
      }
      if (!ok) break;
      base_pos += 2 * n;

      // ---------------- the segment's end: O / l, or a partial
      const bool have = nx > 0;
      if (have) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_full[x], o_cnt & 1, wc))) break;
        ++o_cnt;
        tc_fence_after();
      }
      const bool whole = sg.cf == sg.cl;
      const int n_cta = sg.cl - sg.cf + 1;
      __nv_bfloat16* dst = out + (size_t)(sg.tok + tok) * p.out_stride + ((sg.g << rsh) + (qrow & ((1 << rsh) - 1))) * D;
      auto release_o = [&] {
        tc_fence_before();
        __syncwarp();
        if (have && lane == 0) mbar_arrive(&o_free[x]);
      };
      auto store32 = [&](int q, const uint32_t (&o)[32], float inv) {   // 32 columns, whole sectors at a time
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = pack_bf2(__uint_as_float(o[16 * u + 2 * i]) * inv, __uint_as_float(o[16 * u + 2 * i + 1]) * inv);
          __nv_bfloat16* at = dst + q * 32 + u * 16;
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                         "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          } else {
            reinterpret_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      };
      if (whole && (two || n == 1)) {   // this lane alone holds the rows' result
        if (have && !dead) {
          const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
          for (int q = 0; q < D / 32; q += 2) {
            uint32_t o[64];
            tmem_ld32(tO + q * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
            tmem_ld32(tO + q * 32 + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
            tmem_ld_wait();
            if (valid) {
              store32(q, *reinterpret_cast<uint32_t(*)[32]>(o), inv);
              store32(q + 1, *reinterpret_cast<uint32_t(*)[32]>(o + 32), inv);
            }
          }
        }
        release_o();
        continue;
      }
      // partial slots: three a CTA (see Parts; the third, 2 G + c, for a tile of
      // its own that only its lanes share), two sub-slots each, one a lane
      Parts ps;
      ps.o = part;
      ps.ml = part_ml;
      ps.whole_slot = whole ? 2 * (int)gridDim.x + c : -1;
      ps.cf = sg.cf;
      ps.step = 1;
      ps.c0 = c;
      ps.n = 1;
      ps.nzl = 0;
      ps.z0 = x;
      const int sub = ps.sub(0);
      auto write_part = [&] {
        if (have && !dead) {
          float* po = part + (size_t)sub * kRows * D;
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + q * 32, o);
            tmem_ld_wait();
            if (valid) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                __stcg(reinterpret_cast<float4*>(po) + (size_t)(q * 8 + u) * kRows + qrow,
                       make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]), __uint_as_float(o[4 * u + 2]),
                                   __uint_as_float(o[4 * u + 3])));
            }
          }
        }
        if (valid) {
          __stcg(part_ml + (size_t)sub * 2 * kRows + qrow, have ? m_used : -INFINITY);
          __stcg(part_ml + (size_t)sub * 2 * kRows + kRows + qrow, have ? l : 0.f);
        }
      };
      if (two && n_cta <= kFlat) {
        // A full tile cut in a few parts: whoever comes last keeps its own in tensor memory and
        // adds the others', each thread its row.  The CTA that began the tile works on it at its
        // share's end, mostly after the others, and looks whether they are done before it writes.
        int* ctr = p.ctr + 4 * sg.cf + 1;
        bool last = false;
        if (c == sg.cf) {
          if (st_id == 0) {
            const bool done = atomicAdd(ctr, 0) == n_cta - 1;
            __threadfence();
            if (done) *ctr = 0;
            s_last[1] = done;
          }
          if (!sync_all()) break;
          last = s_last[1] != 0;
        }
        if (!last) {
          write_part();
          if (!last_of(ctr, n_cta, last)) break;
        }
        if (last && !dead) {
          float w[kFlat], lq[kFlat], M = -INFINITY, L = 0.f;
          const float* src[kFlat];
#pragma unroll
          for (int q = 0; q < kFlat; ++q) {
            const int cc = min(sg.cf + q, sg.cl);
            const int sb = (cc > sg.cf ? 2 * cc : 2 * cc + 1) * 2 + x;
            src[q] = part + (size_t)sb * kRows * D + qrow * 4;
            w[q] = ld_cg(part_ml + (size_t)sb * 2 * kRows + qrow);
            lq[q] = ld_cg(part_ml + (size_t)sb * 2 * kRows + kRows + qrow);
            if (cc == c) {
              w[q] = m_used;
              lq[q] = l;
            }
          }
#pragma unroll
          for (int q = 0; q < kFlat; ++q)
            if (q < n_cta) M = fmaxf(M, w[q]);
#pragma unroll
          for (int q = 0; q < kFlat; ++q) {
            if (q < n_cta) {
              w[q] = lq[q] == 0.f ? 0.f : exp2f(w[q] - M);   // 0: no visible key in this part (NaN counts)
              L += w[q] * lq[q];
            }
          }
          const float inv = L != 0.f ? 1.f / L : 0.f;
          const int me = c - sg.cf;
#pragma unroll 1
          for (int q = 0; q < D / 32; q += 2) {   // 64 columns at a time
            float acc[64], y[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.f;
#pragma unroll 1
            for (int s = 0; s < n_cta; ++s) {
              const float ws = s == 0 ? w[0] : s == 1 ? w[1] : s == 2 ? w[2] : w[3];
              if (s == me) {
                tmem_ld32(tO + q * 32, *reinterpret_cast<uint32_t(*)[32]>(y));
                tmem_ld32(tO + q * 32 + 32, *reinterpret_cast<uint32_t(*)[32]>(y + 32));
                tmem_ld_wait();
              } else {
                const float* from = s == 0 ? src[0] : s == 1 ? src[1] : s == 2 ? src[2] : src[3];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                  const float4 z = ld_cg4(from + (size_t)(q * 8 + u) * kRows * 4);
                  y[4 * u] = z.x;
                  y[4 * u + 1] = z.y;
                  y[4 * u + 2] = z.z;
                  y[4 * u + 3] = z.w;
                }
              }
              if (ws != 0.f) {
#pragma unroll
                for (int i = 0; i < 64; ++i) acc[i] = fmaf(ws, y[i], acc[i]);
              }
            }
            if (valid) {
              store32(q, *reinterpret_cast<uint32_t(*)[32]>(acc), inv);
              store32(q + 1, *reinterpret_cast<uint32_t(*)[32]>(acc + 32), inv);
            }
          }
        }
        release_o();
        continue;
      }
      write_part();
      release_o();
      // The tile's parts: up to kFlat CTAs' are merged by whoever comes last;
      // more in groups of about the square root of their number, each by its last
      // CTA into its first one's slot, and the groups by the last of all.
      const int gs = n_cta <= kFlat ? n_cta : (int)ceilf(sqrtf((float)n_cta));
      const int n_grp = (n_cta + gs - 1) / gs, grp = (c - sg.cf) / gs, g0 = sg.cf + grp * gs;
      const int g_cta = min(gs, sg.cl - g0 + 1);
      bool last = true;
      if (g_cta > 1) {
        if (!last_of(p.ctr + 4 * g0 + (g0 > sg.cf ? 0 : 1), g_cta, last)) break;
      } else if (!sync_all()) {
        break;
      }
      if (last && n_grp > 1) {
        float* gml = part_ml + (size_t)gridDim.x * 6 * 2 * kRows;
        for (int y = 0; y <= two; ++y) {
          ps.c0 = g0;
          ps.nzl = two ? 0 : 1;
          ps.z0 = y;
          ps.n = g_cta << ps.nzl;
          const int dst_sub = ps.sub(0);   // a part that each thread has read before it writes
          float* po = part + (size_t)dst_sub * kRows * D;
          merge_parts<D>(ps, min(kRows, (sg.ntok - y * tokens_half) << rsh), st_id, [&](int rr, int col, const float4& a, float M, float L) {
            __stcg(reinterpret_cast<float4*>(po) + (size_t)col * kRows + rr, a);
            if (col == 0) {
              __stcg(gml + (size_t)dst_sub * 2 * kRows + rr, M);
              __stcg(gml + (size_t)dst_sub * 2 * kRows + kRows + rr, L);
            }
          });
        }
        if (!last_of(p.ctr + 4 * sg.cf + 2, n_grp, last)) break;
        ps.ml = gml;
      }
      if (last) {
        for (int y = 0; y <= two; ++y) {   // a full tile's halves one after the other
          ps.c0 = sg.cf;
          ps.step = n_grp > 1 ? gs : 1;
          ps.nzl = (two || n_grp > 1) ? 0 : 1;
          ps.z0 = two ? y : 0;
          ps.n = (n_grp > 1 ? n_grp : n_cta) << ps.nzl;
          __nv_bfloat16* o0 = out + (size_t)(sg.tok + y * tokens_half) * p.out_stride + (sg.g << rsh) * D;
          merge_parts<D>(ps, min(kRows, (sg.ntok - y * tokens_half) << rsh), st_id, [&](int rr, int col, const float4& a, float M, float L) {
            const float inv = L != 0.f ? 1.f / L : 0.f;
            reinterpret_cast<uint2*>(o0 + (size_t)(rr >> rsh) * p.out_stride + (rr & ((1 << rsh) - 1)) * D)[col] =
                make_uint2(pack_bf2(a.x * inv, a.y * inv), pack_bf2(a.z * inv, a.w * inv));
          });
        }
      }
      if (whole && !sync_all()) break;   // the lanes' slot is free again
    }
  } else {
    // ---------------- E4M3 tiles expanded in their slots (exact), unseen values as zeros
    if constexpr (F8) {
      regs_dec<C::REGS_CVT>();
      // kCvtWarps warps a tile, so that several tiles are under way: what a tile takes is
      // mostly latency (its barrier, shared memory, the proxy fence)
      constexpr int GROUPS = 4 / kCvtWarps;
      static_assert(C::RAWS % GROUPS == 0, "a barrier's uses are all one group's");
      constexpr int CPR = D / 16;             // 16-byte chunks of a raw row
      constexpr int RPI = 32 / CPR;           // rows a warp takes at once
      constexpr int ROUNDS = kKeys / (RPI * kCvtWarps), BATCH = 1;
      const int group = (warp - 12) / kCvtWarps, in_group = (warp - 12) % kCvtWarps;
      // eight threads side by side write four chunks of two rows: all banks once
      const int col = D == 128 ? (lane & 3) | ((lane >> 1) & 4) : lane & 3;
      const int row0 = in_group * RPI + (D == 128 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane >> 2);
      uint32_t pos = 0;
      bool ok = true;
      while (work && ok && ring.next(sg, wc)) {
        const int n = sg.n;
        // ring order: K(0), then K(j + 1) and V(j)
        for (int q = 0; ok && q < 2 * n; ++q, ++pos) {
          if (GROUPS > 1 && pos % GROUPS != (uint32_t)group) continue;
          const bool is_k = q == 0 || ((q & 1) && q < 2 * n - 1);
          const int j = is_k ? (q + 1) >> 1 : (q == 2 * n - 1 ? n - 1 : (q >> 1) - 1);
          const uint32_t slot = pos % RING;
          ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[pos % C::RAWS], (pos / C::RAWS) & 1, wc));
          if (!ok) break;
          const int key0 = (sg.kt0 + j) << 7;
          const bool edge = key0 < sg.lo || key0 + kKeys > sg.hi;
          uint8_t* dst = sKV + slot * C::SLOT + (col >> 2) * C::ATOM;   // 4 raw chunks are one 128-byte row of 16 bits
          const uint8_t* src = sKV + slot * C::SLOT + C::RAW_OFF + col * 16;
          const int c0 = (col & 3) * 2;
          auto expand = [&](auto key) {   // keys as bf16, like the queries; values as f16, like the weights
            constexpr bool K = decltype(key)::value;
#pragma unroll 1
            for (int b = 0; b < ROUNDS; b += BATCH) {
              uint4 w[BATCH];
#pragma unroll
              for (int u = 0; u < BATCH; ++u) w[u] = *reinterpret_cast<const uint4*>(src + ((b + u) * RPI * kCvtWarps + row0) * D);
              __syncwarp();   // d = 128: a row's bytes are read by this warp before it writes over them
#pragma unroll
              for (int u = 0; u < BATCH; ++u) {
                const int r = (b + u) * RPI * kCvtWarps + row0;
                if (!K && edge && (key0 + r < sg.lo || key0 + r >= sg.hi)) w[u] = make_uint4(0, 0, 0, 0);
                const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint16_t lo = (uint16_t)in[i], hi = (uint16_t)(in[i] >> 16);
                  o[2 * i] = K ? e4m3x2_to_bf2(lo) : e4m3x2_to_f16x2(lo);
                  o[2 * i + 1] = K ? e4m3x2_to_bf2(hi) : e4m3x2_to_f16x2(hi);
                }
                uint8_t* d = dst + r * 128;
                *reinterpret_cast<uint4*>(d + (((c0) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(d + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
              }
            }
          };
          if (is_k) expand(std::true_type{});
          else expand(std::false_type{});
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[slot]);
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int D, bool PAGED, bool F8>
int launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const RaggedAttnParams& p, int grid, cudaStream_t st) {
  using C = Cfg<D, F8>;
  auto kern = attn_ragged_kernel<D, PAGED, F8>;
  // the attribute belongs to the current device: set on every call
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return ZAYA_ERR_CUDA;
  const cudaError_t e = launch_k(kern, dim3(grid), dim3(C::THREADS), C::SMEM, st, nullptr, 0, q, k, v, p);
  return e == cudaSuccess ? ZAYA_OK : ZAYA_ERR_CUDA;
}

}  // namespace

size_t attn_ragged_ws_bytes(int n_q, int n_kv, int d) {
  const int sms = std::min(num_sms_current(), kMaxCtas);
  // three slots of two lanes a CTA: O, and (max, sum) of the lane and of its group
  return (size_t)sms * 6 * ((size_t)kRows * d * 4 + 2 * 2 * kRows * 4);
}

int launch_attn_ragged(const RaggedAttnParams& p0, cudaStream_t st) {
  if (attn_short_fits(p0, num_sms_current())) return launch_attn_short(p0, num_sms_current(), st);
  RaggedAttnParams p = p0;
  p.rep_shift = 0;
  while (p.n_kv << p.rep_shift < p.n_q) ++p.rep_shift;
  const bool paged = p.seq_len != nullptr;
  const int rep = 1 << p.rep_shift, tok = kRows >> p.rep_shift;
  CUtensorMap mq, mk, mv;
  int rc = make_tmap_heads(&mq, p.q, p.T, p.n_q, p.d, p.q_stride, rep, tok, 0);
  if (rc) return rc;
  if (paged) {   // [page][head x place][d]: no coordinate passes 32 bits in a pool of any size
    const uint64_t rows = (uint64_t)p.n_kv << p.page_shift;
    const uint32_t box = std::min(1 << p.page_shift, kKeys);
    rc = make_tmap_heads(&mk, p.k, p.n_pages, rows, p.d, rows * p.d, box, 1, p.fp8);
    if (!rc) rc = make_tmap_heads(&mv, p.v, p.n_pages, rows, p.d, rows * p.d, box, 1, p.fp8);
  } else {
    rc = make_tmap_heads(&mk, p.k, p.T, p.n_kv, p.d, p.k_stride, 1, kKeys, 0);
    if (!rc) rc = make_tmap_heads(&mv, p.v, p.T, p.n_kv, p.d, p.v_stride, 1, kKeys, 0);
  }
  if (rc) return rc;
  // no more CTAs than the call can have shares: query tiles x key tiles of the longest row possible
  const long long tiles = (long long)p.n_kv * (p.T / (2 * tok) + std::min(p.B, p.T));
  const long long len = paged ? (long long)p.max_pages << p.page_shift : p.T;
  const long long span = std::min(len, (long long)p.window + 2 * tok) / kKeys + 2;
  const int grid = (int)std::min<long long>(std::min(num_sms_current(), kMaxCtas), tiles * span);
  if (p.d == 128) {
    if (!paged) return launch<128, false, false>(mq, mk, mv, p, grid, st);
    return p.fp8 ? launch<128, true, true>(mq, mk, mv, p, grid, st) : launch<128, true, false>(mq, mk, mv, p, grid, st);
  }
  if (!paged) return launch<64, false, false>(mq, mk, mv, p, grid, st);
  return p.fp8 ? launch<64, true, true>(mq, mk, mv, p, grid, st) : launch<64, true, false>(mq, mk, mv, p, grid, st);
}

}  // namespace zaya
