// attn_q4.cu -- attention of new tokens over the 4-bit KV cache (q4.cuh): over
// each sequence's whole context (with its log-sum-exp, and for the block's
// selection its logits), and over index lists (the sparse layers).
//
// decode_attn_q4: grid of at most kQ4AttnCtas CTAs of four warps.  The contexts' tiles
// of 128 tokens, in the order (sequence, KV head, tile), are cut into equal
// contiguous ranges, one per CTA, so ragged lengths leave no SM idle; every
// CTA works out its range from the lengths.  Each warp owns 32 tokens of a
// tile and a ring of stages of its own, filled by untiled bulk copies of its
// records (never past the sequence's length): no warp waits for another until
// a (sequence, KV head) ends.  There the warps' states are joined and one
// partial (log-sum-exp, normalised o) is written; decode_attn_q4_merge joins
// the partials.
//
// What bounds it: with the arithmetic taken out the copies alone run at 6.6
// TB/s; with it, two contexts of 1M tokens (32 / 4 heads, 1.18 GB) take 227 us =
// 5.2 TB/s, 0.81 of the measured copy rate, in short bursts (260 us under
// sustained load, where the power cap lowers the clock).  Per 16 tokens a warp
// issues 311 instructions, about 140 of them on the integer pipe (one mask per
// pair of codes), where HBM would leave an SM time for about 390 issue slots per
// scheduler quarter.  No pipe is saturated (integer 55%, issue slots 60% busy):
// dependent latencies take part of the rest, and the end of the launch another,
// since an SM's three CTAs do not end together (see Cut).  Three CTAs of four
// warps per SM at 168 registers: two CTAs 286 us, four (128 registers, spills)
// 294 us where three took 266; five warps per CTA 23% slower, six or seven 9%
// to 37%.  Steps of 32 keys rather than 16 (266 against 287 us) give the
// scheduler two independent chains.  Tried and slower: the -8 of V's codes
// through a second MMA on a constant operand (254 against 244 us), the shifts
// as multiply-high (247 against 228), q^T K as e4m3 MMAs with q split in two
// (291 against 228; the legacy FP8 MMA is slow here), the queries' fragments in
// shared memory (equal at 12 warps, 243 against 227 us at 16).
//
// sparse_q4: a cluster of CTAs per (sequence, KV head) splits the list; each
// warp gathers 32 records at a time into a ring of its own by 16-byte
// asynchronous copies, and the cluster joins through distributed shared memory.
// One bulk copy per 144-byte record was limited by the rate at which an SM
// starts bulk copies, about one per 20 cycles (300 x 4 lists of 1152: 100 us,
// against 68 us).  Few short lists are bound by latency (list entry -> record ->
// step -> join).  From some 48 x 2 lists on the steps get slower as warps are
// added (1.7 us a step with one CTA per list, 2.7 us with two), which no single
// counter explains: a warp issues 440 instructions per 16 records (130 more than
// above, for addresses and copies), issue slots 47% and the integer pipe 39%
// busy, and L2 is asked for 9.6 sectors of 32 bytes per record (a copy of 16
// bytes asks for one) where a record covers 5.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace hs2 {

HS2_STATUS_ACCESSOR(status_attn_q4)
HS2_BUDGET_SETTER(budget_attn_q4)

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int NW = 4;                       // warps per CTA
constexpr int WT = 32;                      // tokens per warp and tile
constexpr int TILE = NW * WT;               // tokens per tile
constexpr int STAGES = 2;                   // ring depth per warp (a power of two)
constexpr int STAGE_BYTES = WT * Q4_REC;    // 4608

template <int NT, int W = NW>
struct JoinBuf {  // the warps' states of one (sequence, KV head)
  float m[W][NT * 8], l[W][NT * 8];
  float o[W][NT * 8][128];
};

template <int NT>
constexpr int attn_smem_bytes() {
  return NW * STAGES * STAGE_BYTES + int(sizeof(JoinBuf<NT>)) + 16;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The joined state of W warps for head h, in the form of q4_put: {log-sum-exp,
// weight}, four dims of the normalised output per lane in acc.
template <int NT, int W>
__device__ __forceinline__ float2 joined(const JoinBuf<NT, W>& join, int h, int lane, float4& acc) {
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) M = fmaxf(M, join.m[i][h]);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float w = join.m[i][h] == -INFINITY ? 0.f : fast_exp2(join.m[i][h] - M);
    L += join.l[i][h] * w;
    const float4 v = *reinterpret_cast<const float4*>(&join.o[i][h][4 * lane]);
    acc.x += v.x * w;
    acc.y += v.y * w;
    acc.z += v.z * w;
    acc.w += v.w * w;
  }
  if (L == 0.f) return make_float2(-INFINITY, 0.f);
  const float n = __fdividef(1.f, L);
  acc = make_float4(acc.x * n, acc.y * n, acc.z * n, acc.w * n);
  return make_float2(M + __log2f(L), 1.f);
}

// length of sequence b, clamped to [0, cap]
__device__ __forceinline__ int seq_length(const Q4Lens& lens, int b, int64_t cap) {
  return lens.dev == nullptr ? lens.host[b] : min(max(__ldg(lens.dev + b), 0), int(cap));
}

// s_pre[b] = tiles of one KV head in sequences before b; s_pre[B] = all (times
// Hkv they fit an int: 2^31 tiles would be 39 TB of records)
// (B <= kQ4MaxBatch, 128 threads, a CTA barrier on both sides)
__device__ void tile_prefix(const Q4Lens& lens, int B, int64_t cap, int* s_pre, int* s_sum) {
  constexpr int PER = kQ4MaxBatch / (NW * 32);
  const int tid = threadIdx.x, lane = lane_id();
  int n[PER], mine = 0;
  const int per = (B + NW * 32 - 1) / (NW * 32);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * per + i;
    n[i] = i < per && b < B ? (seq_length(lens, b, cap) + TILE - 1) / TILE : 0;
    // a length outside [0, cap] is reported, and taken as the nearest bound
    if (i < per && b < B && lens.dev != nullptr && unsigned(__ldg(lens.dev + b)) > unsigned(cap))
      set_dev_status(DEV_BAD_INDEX);
    mine += n[i];
  }
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) s_sum[warp_id()] = inc;
  __syncthreads();
  int base = inc - mine;
  for (int w = 0; w < warp_id(); ++w) base += s_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * per + i;
    if (i < per && b < B) s_pre[b] = base;
    base += n[i];
  }
  if (tid == 0) {
    int all = 0;
    for (int w = 0; w < NW; ++w) all += s_sum[w];
    s_pre[B] = all;
  }
  __syncthreads();
}

// a position in the flat order (sequence, KV head, tile)
struct TileAt {
  int b, g, i, nt, len;  // sequence, KV head, tile; that sequence's tiles and length
};

__device__ __forceinline__ TileAt tile_at(int flat, const int* s_pre, const Q4Lens& lens,
                                          int B, int64_t cap, int Hkv) {
  int lo = 0, hi = B;  // largest b with s_pre[b] * Hkv <= flat (its tiles not empty)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_pre[mid] * Hkv <= flat) lo = mid; else hi = mid;
  }
  TileAt a;
  a.b = lo;
  a.nt = s_pre[lo + 1] - s_pre[lo];
  a.len = seq_length(lens, lo, cap);
  const int r = flat - s_pre[lo] * Hkv;
  a.g = r / a.nt;
  a.i = r - a.g * a.nt;
  return a;
}

__device__ __forceinline__ void tile_next(TileAt& a, const int* s_pre, const Q4Lens& lens, int B,
                                          int64_t cap, int Hkv) {
  if (++a.i < a.nt) return;
  a.i = 0;
  if (++a.g < Hkv) return;
  a.g = 0;
  a.nt = 0;
  while (a.nt == 0 && ++a.b < B) a.nt = s_pre[a.b + 1] - s_pre[a.b];
  if (a.b < B) a.len = seq_length(lens, a.b, cap);
}

// The equal ranges that `total` tiles are cut into: range c is [start(c),
// start(c + 1)), none of them empty, so that the ranges of one (sequence, KV
// head) are consecutive and each has written its partial.  An SM's three CTAs
// do not end together (167, 191 and 215 us of 2 x 1M tokens: the first one
// issues first), but shares of 9 : 8 : 7 in the order of launch made SMs end
// apart instead (195 to 227 us), since that order does not tell which CTAs
// share an SM.  Tiles drawn one by one from a counter into a CTA's partial would
// make the order of the sums, and with it the result's last bits, depend on
// timing; drawing fixed chunks with a partial each would not, and is not built.
struct Cut {
  int total, n;
  __device__ Cut(int tiles, int ctas) : total(tiles), n(min(tiles, ctas)) {}
  __device__ int start(int c) const { return int(uint64_t(total) * unsigned(c) / unsigned(n)); }
  // the range that holds tile x: the last c with start(c) <= x
  __device__ int of(int x) const {
    return int((uint64_t(x + 1) * unsigned(n) - 1) / unsigned(total));
  }
};

template <int G, bool LOGITS>
__global__ void __launch_bounds__(NW * 32, G > 8 ? 2 : 3)
    decode_attn_q4(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ cache,
                   const __grid_constant__ Q4Lens lens, int B, int64_t cap, int Hkv,
                   float scale_log2, float* __restrict__ logits, float2* __restrict__ part,
                   float* __restrict__ part_o, int2* __restrict__ where) {
  constexpr int NT = G > 8 ? G / 8 : 1;
  __shared__ int s_pre[kQ4MaxBatch + 1];
  __shared__ int s_sum[NW];
  __shared__ uint64_t full[NW][STAGES];
  __shared__ __align__(16) __nv_bfloat16 s_q[2][G * 128];  // queries: this KV head's, the next one's
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* dsmem = dsmem_raw + ((16u - (smem_u32(dsmem_raw) & 15u)) & 15u);
  JoinBuf<NT>& join = *reinterpret_cast<JoinBuf<NT>*>(dsmem + NW * STAGES * STAGE_BYTES);

  const int warp = warp_id(), lane = lane_id(), gid = lane >> 2, t = lane & 3;
  uint8_t* ring = dsmem + warp * STAGES * STAGE_BYTES;
  grid_trigger();
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[warp][i], 1);
    fence_barrier_init();
  }
  tile_prefix(lens, B, cap, s_pre, s_sum);  // its barriers publish the mbarriers too
  const Cut cut(s_pre[B] * Hkv, gridDim.x);
  if (int(blockIdx.x) >= cut.n) return;
  const int t0 = cut.start(blockIdx.x), t1 = cut.start(blockIdx.x + 1);

  // ---- this warp's records of a range: per (sequence, KV head) some whole
  // parts of WT records and at most one shorter one, copied in order
  struct Run {
    int whole, part;     // whole parts; records of the short one (0: none)
    const uint8_t* src;  // the first
  };
  auto run_of = [&](const TileAt& a, int tiles) {
    const int n = a.len - a.i * TILE - warp * WT;  // tokens from this warp's first part on
    Run r;
    r.whole = min(tiles, n >= WT ? (n - WT) / TILE + 1 : 0);
    r.part = r.whole < tiles ? max(0, min(WT - 1, n - r.whole * TILE)) : 0;
    r.src = cache + ((int64_t(a.b) * Hkv + a.g) * cap + int64_t(a.i) * TILE + warp * WT) * Q4_REC;
    return r;
  };
  auto next_head = [&](TileAt& a) {
    a.i = a.nt - 1;
    tile_next(a, s_pre, lens, B, cap, Hkv);
  };
  TileAt at = tile_at(t0, s_pre, lens, B, cap, Hkv), ahead = at;
  int left = t1 - t0;  // tiles whose copies have not been reached
  Run run{0, 0, nullptr};
  unsigned n_in = 0, n_out = 0;  // stages filled / attended so far
  bool ok = true;
  auto fill = [&]() {  // copies the next part
    while (run.whole == 0 && run.part == 0) {
      if (left == 0) return;
      const int tiles = min(left, ahead.nt - ahead.i);
      run = run_of(ahead, tiles);
      left -= tiles;
      next_head(ahead);
    }
    const uint32_t bytes = (run.whole > 0 ? WT : run.part) * Q4_REC;
    if (run.whole > 0) --run.whole; else run.part = 0;
    if (lane == 0) {
      uint64_t* bar = &full[warp][n_in % STAGES];
      mbar_arrive_expect_tx(bar, bytes);
      bulk_load(ring + (n_in % STAGES) * STAGE_BYTES, run.src, bytes, bar);
    }
    run.src += TILE * Q4_REC;
    ++n_in;
  };
  auto fetch_q = [&](const TileAt& a, int buf) {
    const __nv_bfloat16* src = q + (int64_t(a.b) * Hkv + a.g) * G * 128;
    for (int i = threadIdx.x; i < G * 16; i += NW * 32) cp_async16(&s_q[buf][8 * i], src + 8 * i);
  };
  fetch_q(at, 0);
#pragma unroll 1
  for (int s = 0; s < STAGES; ++s) fill();

  int qbuf = 0;
  for (int tt = t0; tt < t1;) {
    // ---- one (sequence, KV head): its tiles in this CTA's range
    const int b = at.b, g = at.g, i0 = at.i;
    const int tiles = min(t1 - tt, at.nt - at.i);
    const Run mine = run_of(at, tiles);
    if (at.i == 0 && threadIdx.x == 0) {  // where this head's partials will be
      where[int64_t(b) * Hkv + g] =
          make_int2(int(blockIdx.x) + b * Hkv + g, cut.of(tt + at.nt - 1) - int(blockIdx.x) + 1);
    }
    tt += tiles;
    // the head's queries have landed, and every warp is done with the last
    // head's join buffer and queries; the next head's queries set out
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    next_head(at);
    if (tt < t1) fetch_q(at, qbuf ^ 1);
    Q4State<NT> st;
    q4_init<NT>(st, s_q[qbuf], G, scale_log2);
    qbuf ^= 1;
    float* lg = LOGITS ? logits + ((int64_t(b) * Hkv + g) * cap + i0 * TILE + warp * WT + gid) * G + 2 * t
                       : nullptr;
    int n = WT;  // records of the part being attended
    auto put = [&](int h, int nt, const float (&x)[4]) {
      const int h0 = nt * 8 + 2 * t, nv = n - 16 * h;
      float* r = lg + 16 * h * G + nt * 8;
      if (h0 + 1 < G) {
        if (gid < nv) *reinterpret_cast<float2*>(r) = make_float2(x[0], x[1]);
        if (gid + 8 < nv) *reinterpret_cast<float2*>(r + 8 * G) = make_float2(x[2], x[3]);
      } else if (h0 < G) {
        if (gid < nv) r[0] = x[0];
        if (gid + 8 < nv) r[8 * G] = x[2];
      }
    };
    auto arrive = [&]() {  // the next stage's records, once they have landed
      if (!__all_sync(0xffffffffu, mbar_try_wait(&full[warp][n_out % STAGES], (n_out / STAGES) & 1)) && ok)
        ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][n_out % STAGES], (n_out / STAGES) & 1));
      return ring + (n_out % STAGES) * STAGE_BYTES;
    };
    auto release = [&]() {
      ++n_out;
      __syncwarp();  // every lane has read the stage before it is filled again
      if (ok) fill();
    };
#pragma unroll 1
    for (int i = 0; i < mine.whole; ++i) {
      q4_step<NT, WT / 16, true, LOGITS>(st, arrive(), ~0u, put);
      if (LOGITS) lg += TILE * G;
      release();
    }
    if (mine.part > 0) {
      n = mine.part;
      q4_step<NT, WT / 16, false, LOGITS>(st, arrive(), (1u << n) - 1, put);
      release();
    }
    // ---- join the warps and write the partial
    q4_put<NT>(st, join.m[warp], join.l[warp], join.o[warp]);
    __syncthreads();
    const int64_t slot = int64_t(blockIdx.x) + int64_t(b) * Hkv + g;
    for (int h = warp; h < G; h += NW) {
      float4 acc;
      const float2 ml = joined<NT, NW>(join, h, lane, acc);
      *reinterpret_cast<float4*>(part_o + (slot * G + h) * 128 + 4 * lane) = acc;
      if (lane == 0) part[slot * G + h] = ml;
    }
  }
  // after a wait that ran out: every copy that was issued lands before exit
  if (!ok && lane == 0)
    for (unsigned s = 0; s < STAGES; ++s)
      drain_phase(&full[warp][s], n_in > s ? (n_in - 1 - s) / STAGES + 1 : 0);
}

// The partials of one head, `base + i * G` for i = first, first + step, ... < n,
// joined by one warp, MU at a time: {m, l}, four dims per lane in acc.
constexpr int MU = 16;
__device__ __forceinline__ float2 join_partials(const float2* __restrict__ part,
                                                const float* __restrict__ part_o, int64_t base, int G,
                                                int first, int step, int n, float4& acc) {
  const int lane = lane_id();
  float M = -INFINITY, L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 < n; i0 += MU * step) {
    float2 p[MU];
    float4 v[MU];
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      p[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u * step < n) {
        const int64_t at = base + int64_t(i0 + u * step) * G;
        p[u] = __ldcg(part + at);
        v[u] = __ldcg(reinterpret_cast<const float4*>(part_o + at * 128) + lane);
      }
    }
    float m = M;
#pragma unroll
    for (int u = 0; u < MU; ++u) m = fmaxf(m, p[u].x);
    const float keep = M == -INFINITY ? 0.f : fast_exp2(M - m);
    M = m;
    L *= keep;
    acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      const float w = p[u].x == -INFINITY ? 0.f : fast_exp2(p[u].x - M);
      L += p[u].y * w;
      acc.x += v[u].x * w;
      acc.y += v[u].y * w;
      acc.z += v[u].z * w;
      acc.w += v[u].w * w;
    }
  }
  return make_float2(M, L);
}

// grid (Hkv * G / HC, B): the partials of HC heads of one KV head -> o, lse.  A
// warp joins a head alone where it has few partials, the CTA's warps together
// where it has many.
template <int HC, int W>
__global__ void __launch_bounds__(W * 32)
    decode_attn_q4_merge(const float2* __restrict__ part, const float* __restrict__ part_o,
                         const int2* __restrict__ where, const __grid_constant__ Q4Lens lens,
                         int64_t cap, int Hkv, int G, __nv_bfloat16* __restrict__ o,
                         float* __restrict__ lse, float* __restrict__ lse2,
                         uint32_t* __restrict__ zero, int64_t n_zero) {
  __shared__ float2 s_ml[W];
  __shared__ __align__(16) float s_o[W][128];
  const int per = G / HC, g = blockIdx.x / per, h0 = (blockIdx.x % per) * HC, b = blockIdx.y;
  const int lane = lane_id(), warp = warp_id();
  const int64_t pair = int64_t(b) * Hkv + g;
  auto store = [&](int h, float2 ml, const float4& acc) {
    const float inv = ml.y == 0.f ? 0.f : __fdividef(1.f, ml.y);  // no context, or every logit -inf
    const int64_t head = pair * G + h;
    *reinterpret_cast<uint2*>(o + head * 128 + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0) {
      const float l2 = ml.y == 0.f ? -INFINITY : ml.x + __log2f(ml.y);
      if (lse != nullptr) lse[head] = l2 * kLn2;
      if (lse2 != nullptr) lse2[head] = l2;
    }
  };
  grid_wait();
  grid_trigger();
  if (zero != nullptr)  // the selection's counters, for the kernels that follow
    for (int64_t i = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * W * 32 + threadIdx.x;
         i < n_zero; i += int64_t(gridDim.x) * gridDim.y * W * 32)
      zero[i] = 0;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (seq_length(lens, b, cap) == 0) {
    for (int h = warp; h < HC; h += W) store(h0 + h, make_float2(-INFINITY, 0.f), acc);
    return;
  }
  const int2 w = __ldcg(where + pair);
  const int64_t base = int64_t(w.x) * G + h0;
  if (w.y <= MU) {
    for (int h = warp; h < HC; h += W)
      store(h0 + h, join_partials(part, part_o, base + h, G, 0, 1, w.y, acc), acc);
    return;
  }
  for (int h = 0; h < HC; ++h) {
    s_ml[warp] = join_partials(part, part_o, base + h, G, warp, W, w.y, acc);
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
    __syncthreads();
    if (warp == h % W) {
      float M = -INFINITY, L = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < W; ++i) M = fmaxf(M, s_ml[i].x);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float f = s_ml[i].x == -INFINITY ? 0.f : fast_exp2(s_ml[i].x - M);
        const float4 v = *reinterpret_cast<const float4*>(&s_o[i][4 * lane]);
        L += s_ml[i].y * f;
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
      store(h0 + h, make_float2(M, L), acc);
    }
    if (h + 1 < HC) __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// sparse_q4
// ---------------------------------------------------------------------------
constexpr int SK = 32;                     // records per stage
constexpr int SST = 2;                     // stages per warp
constexpr int SSTAGE_BYTES = SK * Q4_REC;  // 4608

template <int NT, int W>
constexpr int sparse_smem_bytes() {
  constexpr int ring = W * SST * SSTAGE_BYTES, join = int(sizeof(JoinBuf<NT, W>));
  return (ring > join ? ring : join) + 16;  // the join reuses the drained ring
}

struct Q4Layers {
  const void* q[kQ4MaxLayers];
  void* o[kQ4MaxLayers];
};

// grid (CS * pairs, layers): a pair is G query heads and the list that they
// share with the split - 1 pairs beside it
template <int G, int CS>
__global__ void __launch_bounds__(NW * 32, G > 8 ? 2 : 3)
    sparse_q4(const __grid_constant__ Q4Layers layers, const uint8_t* __restrict__ cache,
              const int32_t* __restrict__ idx, float* __restrict__ lse, int64_t cap, int kw,
              int split, float scale_log2) {
  constexpr int NT = G > 8 ? G / 8 : 1, W = NW;
  grid_wait();
  // this CTA's joined state, read by the cluster's other CTAs
  __shared__ float2 c_ml[NT * 8];
  __shared__ __align__(16) float c_o[NT * 8][128];
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* dsmem = dsmem_raw + ((16u - (smem_u32(dsmem_raw) & 15u)) & 15u);
  JoinBuf<NT, W>& join = *reinterpret_cast<JoinBuf<NT, W>*>(dsmem);
  const int warp = warp_id(), lane = lane_id();
  uint8_t* ring = dsmem + warp * SST * SSTAGE_BYTES;
  const int64_t pair = blockIdx.x / CS;
  const int crank = int(blockIdx.x % CS);
  const auto* q = reinterpret_cast<const __nv_bfloat16*>(layers.q[blockIdx.y]);
  auto* O = reinterpret_cast<__nv_bfloat16*>(layers.o[blockIdx.y]);
  // this warp's entries [lo, hi) of the list, SK per step
  const int per = (kw + CS * W - 1) / (CS * W);
  const int lo = min(kw, (crank * W + warp) * per), hi = min(kw, lo + per);
  const int32_t* list = idx + pair / split * kw;
  const uint8_t* rows = cache + pair / split * cap * Q4_REC;
  auto entry = [&](int step) {
    const int e = lo + step * SK + lane;
    return e < hi ? __ldg(list + e) : -1;
  };
  // copies the records of one step's entries into stage s (one copy group,
  // which may be empty) and returns which of them are valid: SK * 9 pieces of
  // 16 bytes, piece p = part p % 9 of record p / 9
  auto fill = [&](int j, int s) -> uint32_t {
    if (j != -1 && unsigned(j) >= unsigned(cap)) {
      set_dev_status(DEV_BAD_INDEX);
      j = -1;
    }
    const uint32_t keep = __ballot_sync(0xffffffffu, j >= 0);
    if (keep != 0) {
#pragma unroll
      for (int k = 0; k < 9; ++k) {
        const int p = lane + 32 * k, r = (p * 911) >> 13;  // p / 9 for p < 288
        const int jr = __shfl_sync(0xffffffffu, j, r);
        if (jr >= 0)
          cp_async16(ring + s * SSTAGE_BYTES + 16 * p, rows + int64_t(jr) * Q4_REC + 16 * (p - 9 * r));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return keep;
  };
  // records are copied SST steps ahead of their use, the list is read two
  // steps further ahead
  const int steps = (hi - lo + SK - 1) / SK;
  int j[SST];
#pragma unroll
  for (int s = 0; s < SST; ++s) j[s] = entry(s);
  int j1 = entry(SST), j2 = entry(SST + 1);
  uint32_t keep[SST];
#pragma unroll
  for (int s = 0; s < SST; ++s) keep[s] = fill(j[s], s);
  Q4State<NT> st;
  q4_init<NT>(st, q + pair * G * 128, G, scale_log2);
  const auto none = [](int, int, const float (&)[4]) {};
  int s = 0;
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(SST - 1) : "memory");
    __syncwarp();  // every lane's pieces have landed
    const uint32_t k0 = keep[0];
    if (k0 == 0xFFFFFFFFu)
      q4_step<NT, SK / 16, true, false>(st, ring + s * SSTAGE_BYTES, k0, none);
    else if (k0 >> 16)
      q4_step<NT, SK / 16, false, false>(st, ring + s * SSTAGE_BYTES, k0, none);
    else if (k0 != 0)  // a short last step: half the work
      q4_step<NT, 1, false, false>(st, ring + s * SSTAGE_BYTES, k0, none);
    __syncwarp();  // every lane has read the stage
#pragma unroll
    for (int u = 0; u + 1 < SST; ++u) keep[u] = keep[u + 1];
    keep[SST - 1] = fill(j1, s);
    j1 = j2;
    j2 = entry(i + SST + 2);
    s = s + 1 == SST ? 0 : s + 1;
  }
  __syncthreads();  // every warp is done with its ring (copies past the list's end are empty groups)
  q4_put<NT>(st, join.m[warp], join.l[warp], join.o[warp]);
  __syncthreads();
  auto store = [&](int h, float2 ml, const float4& acc) {
    const float inv = ml.y == 0.f ? 0.f : __fdividef(1.f, ml.y);  // an empty list: o = 0, lse = -inf
    const int64_t head = pair * G + h;
    *reinterpret_cast<uint2*>(O + head * 128 + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lse != nullptr && lane == 0)
      lse[head] = ml.y == 0.f ? -INFINITY : (ml.x + __log2f(ml.y)) * kLn2;
  };
  for (int h = warp; h < G; h += W) {
    float4 acc;
    const float2 ml = joined<NT, W>(join, h, lane, acc);
    if (CS == 1) {
      store(h, ml, acc);
    } else {
      *reinterpret_cast<float4*>(&c_o[h][4 * lane]) = acc;
      if (lane == 0) c_ml[h] = ml;
    }
  }
  if constexpr (CS > 1) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    // heads are spread over the cluster's CTAs
    for (int h = crank + CS * warp; h < G; h += CS * W) {
      float2 ml[CS];
      float4 v[CS];
#pragma unroll
      for (int c = 0; c < CS; ++c) {
        ml[c] = *cluster.map_shared_rank(&c_ml[h], c);
        v[c] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&c_o[h][0], c) + 4 * lane);
      }
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int c = 0; c < CS; ++c) M = fmaxf(M, ml[c].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < CS; ++c) {
        const float w = ml[c].x == -INFINITY ? 0.f : fast_exp2(ml[c].x - M);
        L += ml[c].y * w;
        acc.x += v[c].x * w;
        acc.y += v[c].y * w;
        acc.z += v[c].z * w;
        acc.w += v[c].w * w;
      }
      store(h, make_float2(M, L), acc);
    }
    cluster.sync();  // shared memory stays until it has been read
  }
}

// workspace: partials' {m, l}, their outputs, and per (sequence, KV head) the
// place and number of its partials
struct AttnWs {
  size_t o, where, bytes;
};
AttnWs attn_ws(int B, int Hkv, int G) {
  const size_t slots = size_t(kQ4AttnCtas) + size_t(B) * Hkv;
  auto r = [](size_t x) { return (x + 255) / 256 * 256; };
  AttnWs w;
  w.o = r(slots * G * sizeof(float2));
  w.where = w.o + slots * G * 512;
  w.bytes = w.where + r(size_t(B) * Hkv * sizeof(int2));
  return w;
}

template <int HC, int W>
cudaError_t launch_merge(const Q4AttnArgs& a, const float2* part, const float* part_o,
                         const int2* where, cudaStream_t st) {
  // the merge's CTAs may start while the last tiles are attended; they wait
  // for the whole grid before they read a partial
  const int G = a.Hq / a.Hkv;
  return launch_dependent(decode_attn_q4_merge<HC, W>, dim3(unsigned(a.Hq / HC), unsigned(a.B)),
                          dim3(W * 32), 0, st, 1, part, part_o, where, a.lens, a.cap, a.Hkv, G,
                          reinterpret_cast<__nv_bfloat16*>(a.o), a.lse, a.lse2, a.zero, a.n_zero);
}

template <int G, bool LOGITS>
cudaError_t launch_attn_g(const Q4AttnArgs& a, cudaStream_t st) {
  constexpr int NT = G > 8 ? G / 8 : 1;
  const int64_t most = int64_t(a.B) * a.Hkv * ((a.cap + TILE - 1) / TILE);
  constexpr int kMost = G > 8 ? kQ4AttnCtas * 2 / 3 : kQ4AttnCtas;  // one wave (launch bounds)
  const int ctas = int(most < kMost ? most : kMost);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.ws);
  const AttnWs w = attn_ws(a.B, a.Hkv, G);
  float2* part = reinterpret_cast<float2*>(ws);
  float* part_o = reinterpret_cast<float*>(ws + w.o);
  int2* where = reinterpret_cast<int2*>(ws + w.where);
  const auto kernel = decode_attn_q4<G, LOGITS>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), attn_smem_bytes<NT>());
  if (e != cudaSuccess) return e;
  kernel<<<ctas, NW * 32, attn_smem_bytes<NT>(), st>>>(
      reinterpret_cast<const __nv_bfloat16*>(a.q), a.cache, a.lens, a.B, a.cap, a.Hkv,
      a.scale * kLog2e, a.logits, part, part_o, where);
  // Many heads have few partials each on average: a warp per head.  Few heads
  // may have hundreds (one context of 1M tokens, one KV head: 43 us with 16
  // warps per head, 50 with 4), but 512 such CTAs take several waves (16 x 1000
  // tokens, 32 heads: 20.8 us, 16.6 with 4).
  const int64_t heads = int64_t(a.B) * a.Hq;
  if (G >= 4 && heads >= 4 * 148)
    e = launch_merge<G >= 4 ? 4 : 1, 4>(a, part, part_o, where, st);
  else if (heads > 148)
    e = launch_merge<1, 4>(a, part, part_o, where, st);
  else
    e = launch_merge<1, 16>(a, part, part_o, where, st);
  if (e != cudaSuccess) return e;
  count_launch(2);
  return cudaGetLastError();
}

template <int G, int CS>
cudaError_t launch_sparse_cs(const Q4SparseArgs& a, cudaStream_t st) {
  constexpr int NT = G > 8 ? G / 8 : 1, W = NW;
  const int split = a.Hq / a.Hkv / G;
  const auto kernel = sparse_q4<G, CS>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), sparse_smem_bytes<NT, W>());
  if (e != cudaSuccess) return e;
  Q4Layers layers{};
  for (int l = 0; l < a.layers; ++l) {
    layers.q[l] = a.q[l];
    layers.o[l] = a.o[l];
  }
  const dim3 grid(unsigned(int64_t(a.B) * a.Hkv * split * CS), unsigned(a.layers));
  e = launch_dependent(kernel, grid, dim3(W * 32), sparse_smem_bytes<NT, W>(), st, CS, layers, a.cache,
                       a.idx, a.lse, a.cap, a.kw, split, a.scale * kLog2e);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

// How many CTAs share a list.  More of them shorten the chain of steps of a
// warp, until the launch no longer fits the GPU at once (its second wave costs
// as much as the first) or a warp's part falls below one step of 32 entries.
// Measured, us: lists of 1152, G = 8: 32 lists 13.4 / 10.3 / 8.7 / 8.5 for 1 /
// 2 / 4 / 8 CTAs, 64 lists 13.4 / 10.3 / 9.8 / 16.5, 256 lists 18.5 / 23.6 /
// 30.9 / 47.8; 32 lists of 2176 22.6 / 14.9 / 10.4 / 9.8; lists of 128: 4.2 /
// 5.2 / 5.2 / 6.1.
template <int G>
cudaError_t launch_sparse_g(const Q4SparseArgs& a, cudaStream_t st) {
  const int64_t pairs = int64_t(a.B) * a.Hq / G * a.layers;
  const int64_t wave = G > 8 ? 2 * 148 : 3 * 148;  // CTAs (launch bounds)
  if constexpr (G <= 8) {  // 16 heads go together only where lists are many
    if (pairs * 8 <= 2 * 148 && a.kw >= 8 * NW * SK) return launch_sparse_cs<G, 8>(a, st);
    if (pairs * 4 <= wave && a.kw >= 4 * NW * SK) return launch_sparse_cs<G, 4>(a, st);
  }
  if (pairs * 2 <= wave && a.kw >= 2 * NW * SK) return launch_sparse_cs<G, 2>(a, st);
  return launch_sparse_cs<G, 1>(a, st);
}

}  // namespace

size_t attn_q4_workspace_bytes(int B, int Hq, int Hkv) { return attn_ws(B, Hkv, Hq / Hkv).bytes; }

cudaError_t launch_attn_q4(const Q4AttnArgs& a, cudaStream_t st) {
  switch (a.Hq / a.Hkv) {
#define HS2_Q4_CASE(G)                                                     \
  case G:                                                                  \
    return a.logits != nullptr ? launch_attn_g<G, true>(a, st) : launch_attn_g<G, false>(a, st)
    HS2_Q4_CASE(1);
    HS2_Q4_CASE(2);
    HS2_Q4_CASE(4);
    HS2_Q4_CASE(8);
    HS2_Q4_CASE(16);
#undef HS2_Q4_CASE
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_sparse_q4(const Q4SparseArgs& a, cudaStream_t st) {
  switch (a.Hq / a.Hkv) {
    case 1: return launch_sparse_g<1>(a, st);
    case 2: return launch_sparse_g<2>(a, st);
    case 4: return launch_sparse_g<4>(a, st);
    case 8: return launch_sparse_g<8>(a, st);
    case 16:
      // Few lists: their heads in two pairs, twice the warps (one list of 2304
      // 8.8 against 10.8 us, 16 lists 10.5 against 12.9, 96 lists 23.6 against
      // 24.1).  Many: all heads together, each record unpacked once (128 lists
      // 25.4 against 33.0 us).
      if (int64_t(a.B) * a.Hkv * a.layers * 4 <= 3 * 148) return launch_sparse_g<8>(a, st);
      return launch_sparse_g<16>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace hs2
