// cache.cu -- quantising new K/V rows as they are written into a decode
// cache, and reading cache rows back as bf16.
//
// Two formats.  The e4m3 cache is the one hs2_block_decode reads (one fp32
// scale per token and KV head, the rule of hs2_bridge_kv_fp8).  The 4-bit
// cache (q4.cuh) keeps a token's K and V of one head as one 144-byte record.
//
// Both are pure streams: per (token, head) 512 bytes of bf16 on one side and
// 260 (e4m3) or 144 (4-bit) bytes on the other, so HBM bounds them.  A warp
// takes TOK consecutive tokens of one head: lanes 0-15 hold the K row and
// lanes 16-31 the V row, eight dims (16 bytes) each, with the TOK rows' loads
// issued before any is used.  Consecutive tokens of a head are adjacent in the
// 4-bit cache, so a warp's records fill whole sectors together.
//
// Measured, written and read back (4 KV heads): a prompt of 128K tokens in
// 4-bit records 125 us = 5.5 TB/s, 0.85 of the measured copy rate; 64K tokens
// in e4m3 72 us = 5.6 TB/s, 0.87.  The quantiser issues 114 instructions
// per (token, head) and warp and keeps the issue slots 80% busy: scale, codes
// and addresses without a division took it there from 213 us.
#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace hs2 {

HS2_STATUS_ACCESSOR(status_cache)

namespace {

constexpr int TOK = 4;       // tokens per warp, a power of two (8: 134 us where 4 takes 129)
constexpr int CW_WARPS = 4;  // warps per CTA

// s / cap for s < 2^31, cap > 1: mul = floor(2^(31 + l) / cap) + 1 with l =
// ceil(log2 cap) is 2^(31 + l) / cap (1 + e), 0 < e <= 2^-31, so s * mul /
// 2^(31 + l) exceeds s / cap by less than 1 / cap and has the same whole part.
// cap > 2^(l - 1) keeps mul below 2^32.
struct SlotDiv {
  uint32_t mul, shift, cap;  // shift = l - 1 behind a 32-bit multiply-high
};
SlotDiv slot_div(int64_t cap) {
  uint32_t l = 1;
  while ((int64_t(1) << l) < cap) ++l;
  return SlotDiv{cap == 1 ? 0u : uint32_t((uint64_t(1) << (31 + l)) / uint64_t(cap) + 1), l - 1,
                 uint32_t(cap)};
}

// The cache slot of token i, or -1 for none (a slot outside [0, n_slots) is
// reported and skipped like -1).
__device__ __forceinline__ int64_t token_slot(const int32_t* __restrict__ slot, int64_t first,
                                              int64_t i, int64_t n, int64_t n_slots) {
  if (i >= n) return -1;
  if (slot == nullptr) return first + i;
  const int s = __ldg(slot + i);
  if (s >= 0 && s < n_slots) return s;
  if (s != -1) set_dev_status(DEV_BAD_INDEX);
  return -1;
}

// Byte offset of slot s's record (s >= 0; -1 stays -1).
__device__ __forceinline__ int64_t record_of(int64_t s, const SlotDiv& d, int h, int Hkv) {
  if (s < 0) return -1;
  const uint32_t b = d.cap == 1 ? uint32_t(s) : __umulhi(uint32_t(s), d.mul) >> d.shift;
  return ((int64_t(b) * Hkv + h) * d.cap + (uint32_t(s) - b * d.cap)) * Q4_REC;
}

// largest |x| of a lane's eight bf16 values, as bf16 bits (a NaN ranks above
// an infinity, both above every finite value)
__device__ __forceinline__ uint32_t amax_bits(const uint4& v) {
  const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                               max_u16x2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m >> 16, m & 0xFFFFu);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}

// A lane's word of a record's 64-byte code half: natural word m = 4 g + t
// (dims 32 g + 8 t ..) -> where the format keeps it.  K: word 4 t + g.  V: half
// words 4 x + g for x = 2 t, 2 t + 1; lanes of groups g and g ^ 1 trade halves
// so that each ends with one whole word.
__device__ __forceinline__ uint32_t v_trade(uint32_t w, int g) {
  const uint32_t give = (g & 1) ? (w & 0xFFFFu) : (w >> 16);
  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
  return (g & 1) ? (got | (w & 0xFFFF0000u)) : ((w & 0xFFFFu) | (got << 16));
}
__device__ __forceinline__ int stored_word(bool v, int g, int t) {
  return v ? 2 * (2 * t + (g & 1)) + (g >> 1) : 4 * t + g;
}

__global__ void __launch_bounds__(CW_WARPS * 32)
    cache_write_q4(const __nv_bfloat16* __restrict__ K, const __nv_bfloat16* __restrict__ V,
                   int64_t ldk, int64_t ldv, const int32_t* __restrict__ slot, int64_t first,
                   int64_t n, uint8_t* __restrict__ cache, SlotDiv div, int64_t n_slots, int Hkv) {
  const int h = blockIdx.y, lane = lane_id();
  const bool is_v = lane >= 16;
  const int m = lane & 15, g = m >> 2, t = m & 3;
  const int64_t i0 = (int64_t(blockIdx.x) * CW_WARPS + warp_id()) * TOK;
  if (i0 >= n) return;
  const __nv_bfloat16* src = (is_v ? V : K) + h * 128 + m * 8;
  const int64_t ld = is_v ? ldv : ldk;
  // lane u % TOK finds where token u goes
  const int64_t mine = record_of(token_slot(slot, first, i0 + lane % TOK, n, n_slots), div, h, Hkv);
  const uint32_t live = __ballot_sync(0xffffffffu, mine >= 0);
  uint4 v[TOK];
  src += i0 * ld;
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    v[u] = live >> u & 1 ? ldg_stream(src) : make_uint4(0, 0, 0, 0);
    src += ld;
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    uint32_t a = amax_bits(v[u]);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const Q4Scale sc = q4_scale(a);
    float x[8];
    unpack8(v[u], x);
    uint32_t w = q4_codes8(x, sc);
    const uint32_t wv = v_trade(w, g);
    if (is_v) w = wv;
    // the pair of groups (g, g ^ 1): the even one stores both scales
    const uint32_t s2 = __shfl_xor_sync(0xffffffffu, sc.bits, 4);
    uint8_t* rec = cache + __shfl_sync(0xffffffffu, mine, u);
    if (!(live >> u & 1)) continue;
    reinterpret_cast<uint32_t*>(rec + (is_v ? Q4_V : Q4_K))[stored_word(is_v, g, t)] = w;
    if (t == 0 && (g & 1) == 0)
      reinterpret_cast<uint32_t*>(rec + (is_v ? Q4_VS : Q4_KS))[g >> 1] = sc.bits | (s2 << 16);
  }
}

__global__ void __launch_bounds__(CW_WARPS * 32)
    cache_read_q4(const uint8_t* __restrict__ cache, const int32_t* __restrict__ slot,
                  int64_t first, int64_t n, __nv_bfloat16* __restrict__ K,
                  __nv_bfloat16* __restrict__ V, int64_t ldk, int64_t ldv, SlotDiv div,
                  int64_t n_slots, int Hkv) {
  const int h = blockIdx.y, lane = lane_id();
  const bool is_v = lane >= 16;
  const int m = lane & 15, g = m >> 2, t = m & 3;
  const int64_t i0 = (int64_t(blockIdx.x) * CW_WARPS + warp_id()) * TOK;
  if (i0 >= n) return;
  const int64_t ld = is_v ? ldv : ldk;
  __nv_bfloat16* dst = (is_v ? V : K) + h * 128 + m * 8 + i0 * ld;
  const int64_t mine = record_of(token_slot(slot, first, i0 + lane % TOK, n, n_slots), div, h, Hkv);
  const uint32_t live = __ballot_sync(0xffffffffu, mine >= 0);
  uint32_t w[TOK], s[TOK];
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const uint8_t* rec = cache + __shfl_sync(0xffffffffu, mine, u);
    w[u] = s[u] = 0;
    if (live >> u & 1) {
      w[u] = __ldg(reinterpret_cast<const uint32_t*>(rec + (is_v ? Q4_V : Q4_K)) +
                   stored_word(is_v, g, t));
      s[u] = __ldg(reinterpret_cast<const uint16_t*>(rec + (is_v ? Q4_VS : Q4_KS)) + g);
    }
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const uint32_t wv = v_trade(w[u], g);  // its own inverse
    if (live >> u & 1) stg_stream(dst, q4_values8(is_v ? wv : w[u], s[u]));
    dst += ld;
  }
}

// x / s rounded to nearest, for r = the correctly rounded 1 / s: one step of
// Markstein's correction (P. Markstein, IBM Journal of Research and Development
// 34, 1990: q' = q + r (x - s q) is the correctly rounded quotient), whose
// remainder is exact as long as it is not subnormal.  A row pair whose largest
// |x| lies below 2^-60 takes the plain division; above, s >= 2^-69, and an x
// whose remainder could be subnormal (|x| < 2^-101) has a quotient below 2^-32,
// which every rounding sends to the code 0.
constexpr uint32_t kPlainBelow = (127 - 60) << 7;
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return copysignf(__fmaf_rn(__fmaf_rn(-s, q, x), r, q), x);  // -0 stays -0
}

// e4m3 of one fp32 quotient pair: nearest, ties to the even code, saturated
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__global__ void __launch_bounds__(CW_WARPS * 32)
    cache_write_fp8(const __nv_bfloat16* __restrict__ K, const __nv_bfloat16* __restrict__ V,
                    int64_t ldk, int64_t ldv, const int32_t* __restrict__ slot, int64_t first,
                    int64_t n, uint8_t* __restrict__ Kc, uint8_t* __restrict__ Vc,
                    float* __restrict__ scale, int64_t n_slots, int Hkv) {
  const int h = blockIdx.y, lane = lane_id();
  const bool is_v = lane >= 16;
  const int m = lane & 15;
  const int64_t i0 = (int64_t(blockIdx.x) * CW_WARPS + warp_id()) * TOK;
  if (i0 >= n) return;
  const __nv_bfloat16* src = (is_v ? V : K) + h * 128 + m * 8;
  const int64_t ld = is_v ? ldv : ldk;
  const int mine = int(token_slot(slot, first, i0 + lane % TOK, n, n_slots));
  const uint32_t live = __ballot_sync(0xffffffffu, mine >= 0);
  uint4 v[TOK];
  src += i0 * ld;
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    v[u] = live >> u & 1 ? ldg_stream(src) : make_uint4(0, 0, 0, 0);
    src += ld;
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    // one scale for the row pair: the largest |x| over K and V
    const uint32_t a = __reduce_max_sync(0xffffffffu, amax_bits(v[u]));
    const int64_t row = int64_t(__shfl_sync(0xffffffffu, mine, u)) * Hkv + h;
    if (!(live >> u & 1)) continue;
    const bool finite = a < 0x7F80u;
    const float amax = __uint_as_float(a << 16);
    const float s = a == 0 ? 1.f : finite ? amax / 448.f : __uint_as_float(0x7FC00000u);
    float x[8];
    unpack8(v[u], x);
    uint32_t c[2] = {0, 0};
    if (a >= kPlainBelow && finite) {
      const float r = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i >> 1] |= e4m3x2(quotient(x[2 * i], s, r), quotient(x[2 * i + 1], s, r)) << (16 * (i & 1));
    } else if (finite) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i >> 1] |= e4m3x2(x[2 * i] / s, x[2 * i + 1] / s) << (16 * (i & 1));
    }
    *reinterpret_cast<uint2*>((is_v ? Vc : Kc) + row * 128 + m * 8) = make_uint2(c[0], c[1]);
    if (lane == 0) scale[row] = s;
  }
}

// two e4m3 codes -> two fp32 values (exact)
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h)
      : "r"(two));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__global__ void __launch_bounds__(CW_WARPS * 32)
    cache_read_fp8(const uint8_t* __restrict__ Kc, const uint8_t* __restrict__ Vc,
                   const float* __restrict__ ks, const float* __restrict__ vs,
                   const int32_t* __restrict__ slot, int64_t first, int64_t n,
                   __nv_bfloat16* __restrict__ K, __nv_bfloat16* __restrict__ V, int64_t ldk,
                   int64_t ldv, int64_t n_slots, int Hkv) {
  const int h = blockIdx.y, lane = lane_id();
  const bool is_v = lane >= 16;
  const int m = lane & 15;
  const int64_t i0 = (int64_t(blockIdx.x) * CW_WARPS + warp_id()) * TOK;
  if (i0 >= n) return;
  const int64_t ld = is_v ? ldv : ldk;
  __nv_bfloat16* dst = (is_v ? V : K) + h * 128 + m * 8 + i0 * ld;
  const int mine = int(token_slot(slot, first, i0 + lane % TOK, n, n_slots));
  const uint32_t live = __ballot_sync(0xffffffffu, mine >= 0);
  uint2 c[TOK];
  float s[TOK];
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const int64_t row = int64_t(__shfl_sync(0xffffffffu, mine, u)) * Hkv + h;
    c[u] = make_uint2(0, 0);
    s[u] = 0.f;
    if (live >> u & 1) {
      c[u] = __ldg(reinterpret_cast<const uint2*>((is_v ? Vc : Kc) + row * 128 + m * 8));
      s[u] = __ldg((is_v ? vs : ks) + row);
    }
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const uint32_t w[2] = {c[u].x, c[u].y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e4m3x2_f32(w[i >> 1] >> (16 * (i & 1)));
      o[i] = pack_bf16x2(f.x * s[u], f.y * s[u]);
    }
    if (live >> u & 1) stg_stream(dst, make_uint4(o[0], o[1], o[2], o[3]));
    dst += ld;
  }
}

dim3 cache_grid(const CacheRowsArgs& a) {
  const int64_t per = int64_t(CW_WARPS) * TOK;
  return dim3(unsigned((a.n + per - 1) / per), unsigned(a.Hkv));
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsArgs& a, cudaStream_t st) {
  const auto* K = reinterpret_cast<const __nv_bfloat16*>(a.K);
  const auto* V = reinterpret_cast<const __nv_bfloat16*>(a.V);
  if (a.cache != nullptr)
    cache_write_q4<<<cache_grid(a), CW_WARPS * 32, 0, st>>>(
        K, V, a.ldk, a.ldv, a.slot, a.first, a.n, a.cache, slot_div(a.cap), a.n_slots, a.Hkv);
  else
    cache_write_fp8<<<cache_grid(a), CW_WARPS * 32, 0, st>>>(
        K, V, a.ldk, a.ldv, a.slot, a.first, a.n, a.Kc, a.Vc, const_cast<float*>(a.ks), a.n_slots,
        a.Hkv);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t st) {
  auto* K = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(a.K));
  auto* V = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(a.V));
  if (a.cache != nullptr)
    cache_read_q4<<<cache_grid(a), CW_WARPS * 32, 0, st>>>(a.cache, a.slot, a.first, a.n, K, V,
                                                           a.ldk, a.ldv, slot_div(a.cap), a.n_slots,
                                                           a.Hkv);
  else
    cache_read_fp8<<<cache_grid(a), CW_WARPS * 32, 0, st>>>(a.Kc, a.Vc, a.ks, a.vs, a.slot,
                                                            a.first, a.n, K, V, a.ldk, a.ldv,
                                                            a.n_slots, a.Hkv);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs2
