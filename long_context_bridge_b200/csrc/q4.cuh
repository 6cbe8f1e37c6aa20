// q4.cuh -- the 4-bit KV cache: its record, and the warp step that attends a
// tile of records.
//
// The cache is [batch][n_kv_heads][capacity] records of 144 bytes; a record is
// one token's K and V of one KV head:
//     0 ..  63   K codes, 4 bits each
//    64 .. 127   V codes
//   128 .. 135   K scales, bf16, one per group of 32 dims
//   136 .. 143   V scales
//   value = (nibble - 8) * scale;  scale = max(bf16(amax / 7), 2^-120),
//   nibble - 8 = x / scale rounded to nearest even, within [-7, 7]; a group
//   that holds an infinity or a NaN gets the scale NaN and the codes 0.
// A head's tokens are contiguous, so its context is one dense stream (untiled
// bulk copies, whole DRAM bursts), and 144 bytes = 36 words put consecutive
// rows four banks apart: the fragment loads below need no swizzle.
//
// Dims are interleaved so that every mma.sync fragment word is a mask of a
// loaded word.  K: dim 32 g + 8 t + n (n < 8) is nibble 8 (4 t + g) + n, so
// lane t's 16 bytes are its 8 dims of each group g.  V: dim 32 g + 4 x + j
// (j < 4) is nibble 4 (4 x + g) + j, so the lane of output row x finds its
// four dims of each group in one half word.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace hs2 {

constexpr int Q4_REC = 144, Q4_K = 0, Q4_V = 64, Q4_KS = 128, Q4_VS = 136;

// ---------------------------------------------------------------------------
// quantising (cache.cu)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void stg_stream(void* p, const uint4& v) {
  __stcs(reinterpret_cast<uint4*>(p), v);
}

// the larger of each 16-bit half
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

struct Q4Scale {
  float inv;      // 1 / scale, within 2^-22 of it
  uint32_t bits;  // the scale's bf16 bits
  bool finite;
};

// Scale of a group whose largest |x| has the bf16 bits a.  amax * (1 / 7) is
// within 2^-22 of amax / 7, which lies at least 2^-12 away (relative) from
// every tie between two bf16 values (14 * the distance, in units of its ulp, is
// a non-zero whole number), so both round to the same scale.
__device__ __forceinline__ Q4Scale q4_scale(uint32_t a) {
  Q4Scale s;
  s.finite = a < 0x7F80u;
  const float q = fmaxf(__uint_as_float(a << 16) * (1.f / 7.f), __uint_as_float(7u << 23));  // 2^-120
  const __nv_bfloat16 b = __float2bfloat16_rn(q);
  s.bits = s.finite ? uint32_t(*reinterpret_cast<const uint16_t*>(&b)) : 0x7FC0u;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.inv) : "f"(__uint_as_float(s.bits << 16)));
  return s;
}

// Eight codes as one word, element n in nibble n.  x * inv is within 2^-19 of
// x / s (|x / s| < 7.04).  x and s have 8 significant bits each, so a quotient
// is a tie k + 1/2 exactly or at least 1 / 510 away from it: forming x * inv +
// 6144 (ulp 2^-11) puts every tie back on itself and moves no other quotient
// across one.  Adding 12582920 - 6144 then rounds to an integer (ulp 1, ties to
// even) and leaves code + 8 in the low bits.
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], const Q4Scale& s) {
  constexpr uint32_t kBase = 0x4B400000u;  // bits of 12582912
  uint32_t w = 0u - (kBase + (kBase << 4) + (kBase << 8));  // further shifts leave the word
  const uint64_t inv = f2(s.inv, s.inv), snap = f2(6144.f, 6144.f),
                 round = f2(12582920.f - 6144.f, 12582920.f - 6144.f);
#pragma unroll
  for (int n = 0; n < 8; n += 2) {
    float q0, q1;
    f2_split(f2_add(f2_fma(f2(x[n], x[n + 1]), inv, snap), round), q0, q1);
    w += (__float_as_uint(q0) << (4 * n)) + (__float_as_uint(q1) << (4 * n + 4));
  }
  return s.finite ? w : 0x88888888u;
}

// Eight values (nibble - 8) * scale rounded to bf16, in order.  bf16 bits
// 0x4300 | u = 128 + u; nibbles j and j + 4 are handled as a pair.
__device__ __forceinline__ uint4 q4_values8(uint32_t w, uint32_t scale_bits) {
  const __nv_bfloat162 k136 = __float2bfloat162_rn(-136.f);
  const uint32_t s2 = scale_bits * 0x00010001u;
  uint32_t p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&u), k136),
                                     *reinterpret_cast<const __nv_bfloat162*>(&s2));
    p[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// ---------------------------------------------------------------------------
// attending
// ---------------------------------------------------------------------------
// D = A B + C
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                              float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  mma_f16_16816(c, a0, a1, a2, a3, b0, b1, c[0], c[1], c[2], c[3]);
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// transpose of an 8 x 8 matrix of 16-bit values held as an mma fragment
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes)
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The state of one warp that attends records with the G query heads of one KV
// head (NT = ceil(G / 8) tiles of eight).  Lane (gid, t) = (lane / 4, lane %
// 4) owns heads 8 nt + 2 t and + 1 of the logits (keys gid and gid + 8) and of
// the output (dims by gid).
//
// S^T = K q^T in f16: a code u = nibble is taken as the f16 bits 0x000u (u *
// 2^-24, a subnormal, exact) or 0x00u0 (u * 2^-20); the query's elements that
// meet the latter carry 2^-4.  The -8 of the code enters as the accumulator's
// start, -8 * sum of the group's q.  q is scaled by a power of two per head so
// that its largest element lies in [2^14, 2^15): bf16's 8 bits then stay exact
// in f16 down to 2^-28 of it.  A group's sum leaves the MMA in fp32 and meets
// its K scale there, so the logits see no rounding below fp32.
//
// The softmax is base 2 against a reference `ref`: p = 2^(x - ref), with ref =
// the running maximum - 10 and moved only when some x passes it by 14, so p
// is at most 2^14 and the accumulators are rarely rescaled.  x is rounded to fp32
// before ref is taken from it and subtracted, ref is rounded up and ref + 14
// down: that holds for every finite x, also where fp32's spacing exceeds 14.
// (With the product left exact in a fused multiply-add, half a spacing came on
// top of the exponent, and from x = 2^27 on P left f16.  The multiplication of
// its own is four instructions per 16 keys of about 310: 64 x 8K 56.6 us against
// 55.6, 2 x 1M 226 against 224.)
//
// O^T += V^T P^T: P times each group's V scale relative to the group's `r2` (the
// power of two at or below the group's largest V scale met so far) is rounded to
// f16 (2^-11 relative; below 2^-24 of the running maximum of P times the largest
// scale an absolute 2^-35 of that) where the softmax has it, [key][head], and
// transposed by movmatrix into the B fragment; V's codes are exact in f16.  A
// reference per group keeps a group of small V beside one of large V (one for all
// four lost it at 2^36); the division by it is exact in bf16, four instructions
// per 16 keys in place of the four that divided P (64 x 8K 57.7 against 56.9 us,
// 2 x 1M equal).
template <int NT>
struct Q4State {
  uint32_t qf[NT][4][2][2];  // [group][MMA][register]
  float q8[NT][4][4];        // -8 * sum of the group's q * 2^-24, heads 2t, 2t+1, twice
  float f[NT][2];            // logit x (base 2) = f * scaled sum, rounded (f > 0)
  float ref[NT][2], l[NT][2];
  float top[NT][2];          // ref + 14: a logit above it moves ref
  float o[NT][8][4];
  uint32_t r_top[2];         // per group the largest bf16 below 2 r2 (two groups a word)
  uint32_t r_inv[2];         // 1 / r2 as bf16
  uint32_t magic;            // 0x64006400 (see q4_step)
};

__device__ __forceinline__ float q4_pow2_bits(uint32_t bits) { return __uint_as_float(bits << 16); }
// bf16 bits of 1 / 2^(e - 127) for those of a power of two with biased exponent e in [1, 254]
__device__ __forceinline__ uint32_t q4_inv_pow2(uint32_t bits) {
  const uint32_t e = bits >> 7;
  return e < 254 ? (254 - e) << 7 : 0x0040u;
}
// the lane's V scales of a key relative to the groups' references (exact)
__device__ __forceinline__ uint32_t q4_scaled(uint32_t two, uint32_t inv) {
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&two),
                                   *reinterpret_cast<const __nv_bfloat162*>(&inv));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// q: the G rows of 128 bf16 of this KV head's query heads (shared or global memory)
template <int NT>
__device__ __forceinline__ void q4_init(Q4State<NT>& st, const __nv_bfloat16* q, int G,
                                        float scale_log2) {
  const int lane = lane_id(), gid = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int hh = nt * 8 + gid;
    uint32_t w[4][4];  // [group][pair] dims 32 g + 8 t + 2 pair, + 1
    uint32_t a = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint4 v = hh < G ? *reinterpret_cast<const uint4*>(q + hh * 128 + 32 * g + 8 * t)
                             : make_uint4(0, 0, 0, 0);
      w[g][0] = v.x;
      w[g][1] = v.y;
      w[g][2] = v.z;
      w[g][3] = v.w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a = max(a, max(w[g][i] & 0x7FFFu, (w[g][i] >> 16) & 0x7FFFu));
    }
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    // in a vector register and unknown to the compiler (a < 2^15, but it comes
    // from a shuffle): with two constants, or one in a uniform register, (x &
    // mask) | magic takes two instructions, and the integer pipe bounds q4_step
    st.magic = 0x64006400u | (a >> 15);
    // biased exponent of the head's largest |q|; 2^up brings it to [2^14, 2^15)
    const int e = int(a >> 7);
    const int up = e == 255 || a == 0 ? 0 : min(141 - e, 126);
    const float mul = __uint_as_float(uint32_t(127 + up) << 23);
    const float back = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float x[8], s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(w[g][i]) * mul;
        x[2 * i + 1] = bf16hi(w[g][i]) * mul;
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) s += x[n];
      // MMA m takes nibbles (2m, 2m + 4) and (2m + 1, 2m + 5)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        st.qf[nt][g][m][0] = pack_h2(x[2 * m], x[2 * m + 4]);
        st.qf[nt][g][m][1] = pack_h2(x[2 * m + 1] * 0.0625f, x[2 * m + 5] * 0.0625f);
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s *= -8.f / 16777216.f;
      // an accumulator's four starts, from two lanes that hold the same sum: four
      // registers of their own, or every MMA would first copy two of them
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st.q8[nt][g][i] = __shfl_sync(0xffffffffu, s, 4 * (2 * t + (i & 1)) + (i >> 1));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // finite for scale * |q| below 2^117, in this order for every scale
      st.f[nt][i] = (scale_log2 * __shfl_sync(0xffffffffu, back, 4 * (2 * t + i))) * 16777216.f;
      st.ref[nt][i] = st.top[nt][i] = -INFINITY;
      st.l[nt][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) st.o[nt][i][0] = st.o[nt][i][1] = st.o[nt][i][2] = st.o[nt][i][3] = 0.f;
  }
  constexpr uint32_t kLeast = (127 - 120) << 7;  // the least scale that is written
  st.r_top[0] = st.r_top[1] = (kLeast | 0x7Fu) * 0x00010001u;
  st.r_inv[0] = st.r_inv[1] = q4_inv_pow2(kLeast) * 0x00010001u;
}

// Moves the softmax references up to (maximum - 10) and each group's r2 up to its
// largest finite V scale's power of two; rescales what was accumulated.  x: the base-2
// logits of 16 H keys; vs: V scales of the lane's 2 H keys.
template <int NT, int H>
__device__ __forceinline__ void q4_raise(Q4State<NT>& st, const float (&x)[H][NT][4],
                                         const uint2 (&vs)[H][2]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(x[0][nt][i], x[0][nt][i + 2]);
#pragma unroll
      for (int h = 1; h < H; ++h) mx = fmaxf(mx, fmaxf(x[h][nt][i], x[h][nt][i + 2]));
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float old = st.ref[nt][i], up = fmaxf(old, __fadd_ru(mx, -10.f));
      const float al = old == up ? 1.f : fast_exp2(old - up);
      st.ref[nt][i] = up;
      st.top[nt][i] = __fadd_rd(up, 14.f);
      st.l[nt][i] *= al;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        st.o[nt][d][i] *= al;
        st.o[nt][d][i + 2] *= al;
      }
    }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int sh = 16 * (g & 1);
    uint32_t r = 0;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t b = (g < 2 ? vs[h][u].x : vs[h][u].y) >> sh & 0xFFFFu;
        r = max(r, b < 0x7F80u ? b : 0u);
      }
    r = __reduce_max_sync(0xffffffffu, r) & 0x7F80u;
    const uint32_t old = st.r_top[g >> 1] >> sh & 0x7F80u;
    if (r > old) {
      const float al = q4_pow2_bits(old) * q4_pow2_bits(q4_inv_pow2(r));
      st.r_top[g >> 1] = (st.r_top[g >> 1] & ~(0xFFFFu << sh)) | (r | 0x7Fu) << sh;
      st.r_inv[g >> 1] = (st.r_inv[g >> 1] & ~(0xFFFFu << sh)) | q4_inv_pow2(r) << sh;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int d = 2 * g; d < 2 * g + 2; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[nt][d][i] *= al;
    }
  }
}

// Attends those of the 16 H records at `rec` (shared memory) whose bit of
// `keep` is set; FULL: all of them (one instance without masks).  What a masked
// record holds does not matter.  on_logits(h, nt, x): the lane's base-2 logits
// of keys 16 h + gid (heads 2t, 2t + 1) and 16 h + gid + 8 (the same heads).
template <int NT, int H, bool FULL, bool LOGITS, class F>
__device__ __forceinline__ void q4_step(Q4State<NT>& st, const uint8_t* rec, uint32_t keep,
                                        F&& on_logits) {
  const int lane = lane_id(), gid = lane >> 2, t = lane & 3;
  float s[H][NT][4];
  uint2 vs[H][2];  // V scales of keys gid, gid + 8
  // ---- S^T: per group of dims an fp32 sum, times the key's K scale
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const uint8_t* ra = rec + (16 * h + gid) * Q4_REC;
    const uint8_t* rb = ra + 8 * Q4_REC;
    const uint4 ka = *reinterpret_cast<const uint4*>(ra + Q4_K + 16 * t);
    const uint4 kb = *reinterpret_cast<const uint4*>(rb + Q4_K + 16 * t);
    const uint4 sa = *reinterpret_cast<const uint4*>(ra + Q4_KS);  // K scales, V scales
    const uint4 sb = *reinterpret_cast<const uint4*>(rb + Q4_KS);
    vs[h][0] = make_uint2(sa.z, sa.w);
    vs[h][1] = make_uint2(sb.z, sb.w);
    if (!FULL) {
      if (!(keep >> (16 * h + gid) & 1)) vs[h][0] = make_uint2(0, 0);
      if (!(keep >> (16 * h + gid + 8) & 1)) vs[h][1] = make_uint2(0, 0);
    }
    const uint32_t kw0[4] = {ka.x, ka.y, ka.z, ka.w}, kw1[4] = {kb.x, kb.y, kb.z, kb.w};
    const float ks0[4] = {bf16lo(sa.x), bf16hi(sa.x), bf16lo(sa.y), bf16hi(sa.y)};
    const float ks1[4] = {bf16lo(sb.x), bf16hi(sb.x), bf16lo(sb.y), bf16hi(sb.y)};
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t w0 = kw0[g], w1 = kw1[g], v0 = w0 >> 8, v1 = w1 >> 8;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float c[4];
        mma_f16_16816(c, w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u,
                      st.qf[nt][g][0][0], st.qf[nt][g][0][1], st.q8[nt][g][0], st.q8[nt][g][1],
                      st.q8[nt][g][2], st.q8[nt][g][3]);
        mma_f16_16816(c, v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x00F000F0u,
                      st.qf[nt][g][1][0], st.qf[nt][g][1][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float k = i < 2 ? ks0[g] : ks1[g];
          s[h][nt][i] = g == 0 ? c[i] * k : fmaf(c[i], k, s[h][nt][i]);
        }
      }
    }
  }
  // ---- does a reference have to move?
  bool raise = false;
  uint32_t vmax[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[h][nt][i] = __fmul_rn(s[h][nt][i], st.f[nt][i & 1]);  // from here on the logit
        if (!FULL && !(keep >> (16 * h + gid + 8 * (i >> 1)) & 1)) s[h][nt][i] = -INFINITY;
        raise |= s[h][nt][i] > st.top[nt][i & 1];
      }
      if (LOGITS) on_logits(h, nt, s[h][nt]);
    }
    vmax[0] = max_u16x2(vmax[0], max_u16x2(vs[h][0].x, vs[h][1].x));
    vmax[1] = max_u16x2(vmax[1], max_u16x2(vs[h][0].y, vs[h][1].y));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) raise |= max_u16x2(vmax[i], st.r_top[i]) != st.r_top[i];
  if (__any_sync(0xffffffffu, raise)) q4_raise<NT, H>(st, s, vs);
  float sub[NT][2];  // no key yet: ref = -inf, every logit = -inf, p = 0
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) sub[nt][i] = !FULL && st.ref[nt][i] == -INFINITY ? 0.f : -st.ref[nt][i];
  const __half2 k1032 = __float2half2_rn(-1032.f), k16th = __float2half2_rn(0.0625f),
                k72 = __float2half2_rn(-72.f);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    // ---- P' of each group, as B fragments [keys][head]
    const uint32_t v01 = q4_scaled(vs[h][0].x, st.r_inv[0]), v23 = q4_scaled(vs[h][0].y, st.r_inv[1]);
    const uint32_t w01 = q4_scaled(vs[h][1].x, st.r_inv[0]), w23 = q4_scaled(vs[h][1].y, st.r_inv[1]);
    const float va[4] = {bf16lo(v01), bf16hi(v01), bf16lo(v23), bf16hi(v23)};
    const float vb[4] = {bf16lo(w01), bf16hi(w01), bf16lo(w23), bf16hi(w23)};
    uint32_t pb[NT][4][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = fast_exp2(s[h][nt][i] + sub[nt][i & 1]);
        st.l[nt][i & 1] += p[i];
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        pb[nt][g][0] = movmatrix_trans(pack_h2(p[0] * va[g], p[1] * va[g]));
        pb[nt][g][1] = movmatrix_trans(pack_h2(p[2] * vb[g], p[3] * vb[g]));
      }
    }
    // ---- O^T: per group two 16-dim tiles; nibble j of a half word = tile j / 2,
    // row gid + 8 (j % 2).  The usual expansion of small integers through f16's
    // exponent: bits 0x6400 | u = 1024 + u, 0x6400 | u << 4 = 1024 + 16 u.  vw: V words of keys 2t, 2t + 1, 2t + 8, 2t + 9
    uint2 vw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      vw[u] = *reinterpret_cast<const uint2*>(
          rec + (16 * h + 2 * t + (u & 1) + 8 * (u >> 1)) * Q4_REC + Q4_V + 8 * gid);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
      const uint32_t h01 = g < 2 ? __byte_perm(vw[0].x, vw[1].x, sel) : __byte_perm(vw[0].y, vw[1].y, sel);
      const uint32_t h89 = g < 2 ? __byte_perm(vw[2].x, vw[3].x, sel) : __byte_perm(vw[2].y, vw[3].y, sel);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t y0 = m ? h01 >> 8 : h01, y1 = m ? h89 >> 8 : h89;
        uint32_t a[4] = {(y0 & 0x000F000Fu) | st.magic, (y0 & 0x00F000F0u) | st.magic,
                         (y1 & 0x000F000Fu) | st.magic, (y1 & 0x00F000F0u) | st.magic};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __half2 hv = *reinterpret_cast<const __half2*>(&a[i]);
          hv = (i & 1) ? __hfma2(hv, k16th, k72) : __hadd2(hv, k1032);
          a[i] = *reinterpret_cast<const uint32_t*>(&hv);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16_16816(st.o[nt][2 * g + m], a[0], a[1], a[2], a[3], pb[nt][g][0], pb[nt][g][1]);
      }
    }
  }
}

// One warp's state for the join: per head h < 8 NT the base-2 log-sum-exp sM
// (-inf: no key), its weight sL (1, or 0 without a key) and the normalised
// output sO, which stays within the range of V.
template <int NT>
__device__ __forceinline__ void q4_put(const Q4State<NT>& st, float* sM, float* sL,
                                       float (*sO)[128]) {
  const int lane = lane_id(), gid = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = st.l[nt][i];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      const int h = nt * 8 + 2 * t + i;
      if (gid == 0) {
        sM[h] = l == 0.f ? -INFINITY : st.ref[nt][i] + __log2f(l);
        sL[h] = l == 0.f ? 0.f : 1.f;
      }
      const float n = l == 0.f ? 0.f : __fdividef(1.f, l);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        // dims 32 g + 4 gid + {0, 1, 2, 3} = tiles 2g, 2g + 1, rows gid, gid + 8
        const float r2 = q4_pow2_bits(st.r_top[g >> 1] >> (16 * (g & 1)) & 0x7F80u);
        *reinterpret_cast<float4*>(&sO[h][32 * g + 4 * gid]) =
            make_float4(st.o[nt][2 * g][i] * n * r2, st.o[nt][2 * g][i + 2] * n * r2,
                        st.o[nt][2 * g + 1][i] * n * r2, st.o[nt][2 * g + 1][i + 2] * n * r2);
      }
    }
}

}  // namespace hs2
