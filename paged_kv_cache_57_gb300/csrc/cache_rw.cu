// cache_rw.cu -- rows into the pools, and blocks back out of them (lazy_attn_cache_write,
// lazy_attn_cache_read).
//
// Write: one row is one token's K or V of one KV head. Eight dims per lane (one 16-byte
// load where the strides allow), D/8 neighbouring lanes per row, four tokens per lane where
// there are many; rows in the order (token, K or V, head), so that the slices of a fused qkv
// product are read in the order they lie. Nothing is staged: a row's codes are whole bytes
// of its own.
//  - copy: the pool has the rows' type;
//  - e4m3: code = x / scale, correctly rounded (ties to even), saturated at +-448;
//  - int4: per group of 64 dims z = min, s = bf16((max - min) / 15), code =
//    rint((x - z) / s).
// Quotients are formed by an approximate reciprocal and exact remainders in fp32, and where
// that does not tell a border between two codes (or two scales) in 64 bits, so the codes are
// those of the definition. That arithmetic is what bounds the kernel (74% of the issue slots
// taken, e4m3 77%): 173 instructions for eight int4 codes of 32 lanes, 149 for e4m3. Writing 8192
// tokens of 8 heads takes 13.4 us (int4, 43 MB), 16384 tokens 22.6 us (e4m3, 101 MB), the
// rows coming from L2; 8192 as they are 11.5 us (bf16, 5.8 TB/s). Both worked on borders as they
// came, a fifth and two fifths slower, before ties fell out of a corrected quotient (int4) and
// the odd bit out of two roundings (e4m3).
// Read: one warp per (block, head, K or V) record, eight dims per lane (4 bytes of int4 codes, 8
// of e4m3, 16-byte loads of a copied record), written as `dtype` in 16-byte stores; bound by
// bandwidth (16384 int4 blocks of 8 heads 206 us, 6.7 TB/s; bf16 6.9).
#include "int4.cuh"
#include "kernels.h"

namespace lazy {

namespace {

constexpr int kThreads = 256;

enum { kCopy16 = 0, kCopy32 = 1, kE4m3 = 2, kInt4 = 3 };

__device__ __forceinline__ void bf16x8_to_f32(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// x / s rounded to odd (the last bit set where it is inexact), so that a second rounding, to
// e4m3, is that of the exact quotient: scales like amax / 448 put one bf16 value in some
// hundred on a tie or next to it. A product, corrected by its remainder to the nearest fp32
// value; that one's remainder, rounded towards zero on top of it, gives the truncated
// quotient, and whether it is 0 the odd bit. Remainders are exact for 2^-36 <= s <= 2^100 and
// the quotients that matter (the caller scales x and s to that); rounded down they keep the
// sign of a -0. The bit is all that the integer pipe does, which bounds the kernel.
__device__ __forceinline__ float div_to_odd(float x, float s, float inv, float q0) {
  const float q = fmaf(__fmaf_rd(-q0, s, x), inv, q0), rest = __fmaf_rd(-q, s, x);
  const float a = __fmaf_rz(rest, inv, q);
  return rest != 0.f ? __uint_as_float(__float_as_uint(a) | 1u) : a;
}

__device__ __forceinline__ uint2 quantise_e4m3x8(const float (&x)[8], float pre, float s, float inv) {
  float q[8], big = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = x[i] * pre, q0 = v * inv;
    big = fmaf(q0, 0.f, big);
    q[i] = div_to_odd(v, s, inv, q0);
  }
  if (!(big == 0.f)) {  // a product past fp32's range, an infinity or a NaN: passes as it is
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = x[i] * pre * inv;
      if (!(fabsf(q0) < INFINITY)) q[i] = q0;
    }
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = pack_e4m3x2(q[2 * i], q[2 * i + 1]);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// NaN where either is.
__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The code c (as a float, cf) of a quotient next to a border, corrected by
// |(x - lo) - s c| - s / 2, which fp32 holds without an error (x - lo as a sum of two, the
// product of 8 and 5 bits, a difference of near values). A tie goes to the even code.
__device__ __forceinline__ uint32_t int4_code_border(float x, float lo, float s, uint32_t c, float cf) {
  const float d = x - lo, b = d - x, rest = (x - (d - b)) + (-lo - b);
  const float r = fmaf(-s, cf, d), off = (fabsf(r) - 0.5f * s) + (r < 0.f ? -rest : rest);
  const uint32_t to = r < 0.f ? c - 1u : c + 1u;
  return off > 0.f || (off == 0.f && (c & 1u)) ? to : c;
}

// quantise_int4x8 behind its minima in 64 bits: groups that are not finite, of one value, of
// a range that overflows or whose parts leave fp32's normal numbers, or with a scale next to
// a tie.
__device__ __noinline__ uint2 int4_word_exact(uint4 v, float lo, float hi) {
  if (!(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY)) return make_uint2(0u, 0x7fc07fc0u);  // reads back as NaN
  if (hi == lo) return make_uint2(0u, pack_bf16x2(0.f, lo));
  const uint32_t meta = pack_bf16x2(static_cast<float>((static_cast<double>(hi) - static_cast<double>(lo)) / 15.0), lo);
  const float s = meta_scale(meta);
  if (s == 0.f) return make_uint2(0u, meta);  // nearer than bf16 tells
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t word = 0u;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const double x = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    word = word << 4 | static_cast<uint32_t>(fmin(rint((x - static_cast<double>(lo)) / static_cast<double>(s)), 15.0));
  }
  return make_uint2(word, meta);
}

// The lane's eight codes as one word, and its group's (scale, zero) word, from eight bf16
// values. The group's eight lanes are neighbours; all 32 lanes call it.
__device__ __forceinline__ uint32_t quantise_int4x8(const uint4& v, uint32_t& meta) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // (min, -max) in one word: a step across lanes is one shuffle and one minimum
  const uint32_t mn = bmin2(bmin2(w[0], w[1]), bmin2(w[2], w[3])), mx = bmax2(bmax2(w[0], w[1]), bmax2(w[2], w[3])) ^ 0x80008000u;
  uint32_t m = bmin2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = bmin2(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float lo = bf16_lo(m), hi = -bf16_hi(m);
  // range / 15 by a product, off by 2^-22: rounds to bf16 as the quotient does unless its
  // low 16 bits are next to a tie's
  const float range = hi - lo, s0 = range * (1.f / 15.f);
  const uint32_t sb = __float_as_uint(s0);
  constexpr uint32_t kLeastScale = (127u - 99u) << 23, kInf = 255u << 23;
  if (((sb + 8u) & 0xffffu) - 0x8000u <= 16u || sb - kLeastScale >= kInf - kLeastScale) {
    const uint2 r = int4_word_exact(v, lo, hi);
    meta = r.y;
    return r.x;
  }
  meta = pack_bf16x2(s0, lo);
  const float s = meta_scale(meta);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  // q, the quotient of d = x - lo corrected by its remainder (exact: 24 + 8 bits less what
  // cancels), is (x - lo) / s rounded to fp32 wherever that decides a code: ties come out as
  // such, and q + 1.5 x 2^23 has the code, rounded to nearest even, in its last bits. It
  // takes a d without a rounding and quotients that are ties or 2^-21 (half a step of q) away
  // from one. Both hold for |x| and |lo| of 2^-16 of the range or more (or lo = 0): their last
  // bits, and d, are multiples of a power of two above 2^-24 range, so 2 d - (2 k + 1) s is 0
  // or above 2^-23 range, over 2 s < 2.02 range / 15 more than 2^-20.1.
  constexpr float kMagic = 12582912.f;
  auto quotient = [&](float x) {
    const float d = x - lo, q = d * inv;
    return fmaf(fmaf(-q, s, d), inv, q);
  };
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = __float_as_uint(quotient((i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1])) + kMagic);
  const uint32_t least = bmin2(bmin2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), bmin2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  const float tiny = range * 0x1p-16f;
  if (fminf(bf16_lo(least), bf16_hi(least)) < tiny || (fabsf(lo) < tiny && lo != 0.f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]), cf = __uint_as_float(c[i]) - kMagic;
      if (!(fabsf(quotient(x) - cf) < 0.5f - 0x1p-18f)) c[i] = int4_code_border(x, lo, s, c[i], cf);
    }
  }
  uint32_t word = c[7], off = __float_as_uint(kMagic);
#pragma unroll
  for (int i = 6; i >= 0; --i) {
    word = word * 16u + c[i];
    off = off * 16u + __float_as_uint(kMagic);
  }
  return word - off;
}

// U consecutive tokens per lane, same dims of the same head.
template <int KIND, int D, bool VEC, int U>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int LPR = D / 8;  // lanes per row
  constexpr int ESZ = KIND == kCopy32 ? 4 : 2;
  const int u = threadIdx.x % LPR;
  const uint32_t per_token = 2u * (uint32_t)a.Hkv;
  const uint32_t r = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;  // (U tokens, K or V, head)
  const uint32_t tq = (__umulhi(r, a.div_mul) + r) >> a.div_shift;       // r / per_token
  uint32_t h = r - tq * per_token;
  const bool is_v = h >= (uint32_t)a.Hkv;
  if (is_v) h -= a.Hkv;
  const int64_t step = (is_v ? a.v_token_stride : a.k_token_stride) * ESZ;
  const int64_t t0 = (int64_t)tq * U;
  const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.v : a.k) + t0 * step +
                       ((is_v ? a.v_head_stride : a.k_head_stride) * h + 8 * u) * ESZ;
  // All lanes of a warp take part (the groups' shuffles); tokens past the end do nothing. A
  // skipped token's row is read (not behind its slot's load) and dropped.
  uint4 x[U][ESZ / 2];
  int slot[U];
  wait_for_launch_before();
#pragma unroll
  for (int n = 0; n < U; ++n) {
    slot[n] = -1;
#pragma unroll
    for (int i = 0; i < ESZ / 2; ++i) x[n][i] = make_uint4(0, 0, 0, 0);
    if (t0 + n < a.num_tokens) {
      slot[n] = a.slots[t0 + n];
      const uint8_t* row = src + n * step;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < ESZ / 2; ++i) x[n][i] = reinterpret_cast<const uint4*>(row)[i];
      } else if constexpr (ESZ == 4) {
        uint32_t* w = reinterpret_cast<uint32_t*>(x[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const uint32_t*>(row)[i];
      } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(x[n]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = reinterpret_cast<const uint16_t*>(row)[2 * i] |
                 (uint32_t)reinterpret_cast<const uint16_t*>(row)[2 * i + 1] << 16;
      }
    }
  }
  uint8_t* pool = is_v ? a.v_pool : a.k_pool;
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const int blk = slot[n] >> 4, tok = slot[n] & (kBlock - 1);
    const bool live = slot[n] >= 0 && blk < a.num_pool_blocks;
    if (slot[n] >= 0 && !live && u == 0) raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
    const size_t rec = (uint64_t)(uint32_t)(live ? blk : 0) * (uint32_t)a.Hkv + h;
    if constexpr (KIND == kCopy16 || KIND == kCopy32) {
      if (live) {
        uint4* dst = reinterpret_cast<uint4*>(pool + ((rec * kBlock + tok) * D + 8 * u) * ESZ);
#pragma unroll
        for (int i = 0; i < ESZ / 2; ++i) dst[i] = x[n][i];
      }
    } else if constexpr (KIND == kE4m3) {
      float f[8];
      bf16x8_to_f32(x[n][0], f);
      const uint2 c = is_v ? quantise_e4m3x8(f, a.v_pre, a.v_scale, a.v_inv) : quantise_e4m3x8(f, a.k_pre, a.k_scale, a.k_inv);
      if (live) *reinterpret_cast<uint2*>(pool + (rec * kBlock + tok) * D + 8 * u) = c;
    } else {
      using G = Int4Geom<D>;
      uint32_t meta;
      const uint32_t w = quantise_int4x8(x[n][0], meta);
      if (live) {
        uint8_t* base = pool + rec * G::REC;
        const int group = u >> 3;
        *reinterpret_cast<uint32_t*>(base + (is_v ? int4_v_row(tok) : tok) * G::ROW + 4 * (G::NG * (u & 7) + group)) = w;
        if ((u & 7) == 0) *reinterpret_cast<uint32_t*>(base + G::META + 4 * (tok * G::NG + group)) = meta;
      }
    }
  }
}

// ------------------------------------------------------------------ read

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;  // rows a warp takes at a time
  const int lane = threadIdx.x & 31, u = lane % LPR;
  const uint32_t recs = (uint32_t)a.num_blocks * 2u * (uint32_t)a.Hkv;
  wait_for_launch_before();
  for (uint32_t rec = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); rec < recs; rec += gridDim.x * (kThreads / 32)) {
    const uint32_t i = rec / (2u * a.Hkv), rem = rec - i * (2u * a.Hkv);
    const bool is_v = rem >= (uint32_t)a.Hkv;
    const uint32_t h = is_v ? rem - a.Hkv : rem;
    const int blk = a.block_ids[i];
    if (blk < 0) continue;  // padding: its rows stay as they are
    if (blk >= a.num_pool_blocks) {
      if (lane == 0) raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
      continue;
    }
    const size_t src_rec = (size_t)blk * a.Hkv + h, dst_rec = (size_t)i * a.Hkv + h;
    const uint8_t* pool = is_v ? a.v_pool : a.k_pool;
    uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_out : a.k_out);
    if constexpr (KIND == kCopy16 || KIND == kCopy32) {
      constexpr int BYTES = kBlock * D * (KIND == kCopy32 ? 4 : 2);
      constexpr int PER = BYTES / 16 / 32;
      const uint4* src = reinterpret_cast<const uint4*>(pool + src_rec * BYTES) + lane;
      uint4 x[PER];
#pragma unroll
      for (int c = 0; c < PER; ++c) x[c] = src[32 * c];
#pragma unroll
      for (int c = 0; c < PER; ++c) reinterpret_cast<uint4*>(out + dst_rec * BYTES)[lane + 32 * c] = x[c];
    } else {
      uint32_t w[kBlock / RPW][2];
#pragma unroll
      for (int n = 0; n < kBlock / RPW; ++n) {
        const int row = n * RPW + lane / LPR;
        if constexpr (KIND == kE4m3) {
          const uint2 c = *reinterpret_cast<const uint2*>(pool + (src_rec * kBlock + row) * D + 8 * u);
          w[n][0] = c.x, w[n][1] = c.y;
        } else {
          using G = Int4Geom<D>;
          const uint8_t* base = pool + src_rec * G::REC;
          const int tok = is_v ? int4_v_token(row) : row;
          w[n][0] = *reinterpret_cast<const uint32_t*>(base + row * G::ROW + 4 * u);
          w[n][1] = *reinterpret_cast<const uint32_t*>(base + G::META + 4 * (tok * G::NG + u % G::NG));
        }
      }
#pragma unroll
      for (int n = 0; n < kBlock / RPW; ++n) {
        const int row = n * RPW + lane / LPR;
        float f[8];
        int tok = row, dim = 8 * u;
        if constexpr (KIND == kE4m3) {
          const float s = is_v ? a.v_scale : a.k_scale;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t lo, hi;
            e4m3x4_to_f16x4(w[n][e], lo, hi);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            f[4 * e] = x.x * s, f[4 * e + 1] = x.y * s, f[4 * e + 2] = y.x * s, f[4 * e + 3] = y.y * s;
          }
        } else {
          using G = Int4Geom<D>;
          tok = is_v ? int4_v_token(row) : row;
          dim = 64 * (u % G::NG) + 8 * (u / G::NG);
          const float s = meta_scale(w[n][1]), z = meta_zero(w[n][1]);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = fmaf(s, static_cast<float>((w[n][0] >> (4 * e)) & 15u), z);
        }
        *reinterpret_cast<uint4*>(out + ((dst_rec * kBlock + tok) * D + dim) * 2) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      }
    }
  }
}

template <int KIND, int D, int U>
cudaError_t write_u(CacheWriteArgs a, bool vec, cudaStream_t st) {
  const int64_t rows = ((int64_t)a.num_tokens + U - 1) / U * 2 * a.Hkv, per = kThreads / (D / 8);
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  // r / d = (umulhi(r, mul) + r) >> shift for r < 2^31: shift = ceil(log2 d), mul =
  // floor(2^32 (2^shift - d) / d) + 1
  const uint64_t d = 2 * (uint64_t)a.Hkv;
  a.div_shift = 0;
  while ((1ull << a.div_shift) < d) ++a.div_shift;
  a.div_mul = (uint32_t)(((1ull << 32) * ((1ull << a.div_shift) - d)) / d + 1);
  return launch_behind(vec ? cache_write_kernel<KIND, D, true, U> : cache_write_kernel<KIND, D, false, U>, grid, kThreads, 0, st, a);
}

// Four tokens per lane share its addresses and keep four loads in flight (8192 tokens of 8
// heads: 16.0 us against 17.5 with one, when a code took a third more); one where four would leave threads of the device
// idle.
template <int KIND, int D>
cudaError_t write_t(const CacheWriteArgs& a, bool vec, int sms, cudaStream_t st) {
  const int64_t threads = (int64_t)a.num_tokens * 2 * a.Hkv * (D / 8);
  return threads >= (int64_t)sms * 2048 * 4 ? write_u<KIND, D, 4>(a, vec, st) : write_u<KIND, D, 1>(a, vec, st);
}

template <int KIND, int D>
cudaError_t read_t(const CacheReadArgs& a, int sms, cudaStream_t st) {
  const int64_t recs = (int64_t)a.num_blocks * 2 * a.Hkv, per = kThreads / 32;
  const int64_t want = (recs + per - 1) / per, most = (int64_t)sms * 64;
  return launch_behind(cache_read_kernel<KIND, D>, (unsigned)(want < most ? want : most), kThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, int kv_dtype, bool vec, int sms, cudaStream_t st) {
  switch (kv_dtype) {
    case LAZY_F32: return a.D == 128 ? write_t<kCopy32, 128>(a, vec, sms, st) : write_t<kCopy32, 64>(a, vec, sms, st);
    case LAZY_BF16: return a.D == 128 ? write_t<kCopy16, 128>(a, vec, sms, st) : write_t<kCopy16, 64>(a, vec, sms, st);
    case LAZY_FP8_E4M3: return a.D == 128 ? write_t<kE4m3, 128>(a, vec, sms, st) : write_t<kE4m3, 64>(a, vec, sms, st);
    default: return a.D == 128 ? write_t<kInt4, 128>(a, vec, sms, st) : write_t<kInt4, 64>(a, vec, sms, st);
  }
}

cudaError_t launch_cache_read(const CacheReadArgs& a, int kv_dtype, int sms, cudaStream_t st) {
  switch (kv_dtype) {
    case LAZY_F32: return a.D == 128 ? read_t<kCopy32, 128>(a, sms, st) : read_t<kCopy32, 64>(a, sms, st);
    case LAZY_BF16: return a.D == 128 ? read_t<kCopy16, 128>(a, sms, st) : read_t<kCopy16, 64>(a, sms, st);
    case LAZY_FP8_E4M3: return a.D == 128 ? read_t<kE4m3, 128>(a, sms, st) : read_t<kE4m3, 64>(a, sms, st);
    default: return a.D == 128 ? read_t<kInt4, 128>(a, sms, st) : read_t<kInt4, 64>(a, sms, st);
  }
}

}  // namespace lazy
