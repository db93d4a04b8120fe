// cache_rw.cu -- rows into the pools, and blocks back out of them (lazy_attn_cache_write,
// lazy_attn_cache_read).
//
// Write: one row is one token's K or V of one KV head. Eight dims per lane (one 16-byte
// load where the strides allow), D/8 neighbouring lanes per row; rows in the order
// (token, K or V, head), so that the slices of a fused qkv product are read in the order
// they lie. Nothing is staged: a row's codes are whole bytes of its own.
//  - copy: the pool has the rows' type;
//  - e4m3: code = x / scale, correctly rounded (ties to even), saturated at +-448;
//  - int4: per group of 64 dims z = min, s = bf16((max - min) / 15), code =
//    rint((x - z) / s). x / s is formed in fp32 and only a value within 2^-12 of a border
//    between two codes is divided in fp64, so the codes are those of the definition.
// Read: one warp per (block, head, K or V) record, eight dims per lane, written as `dtype`.
//
// Both are bound by bandwidth; they compute a few operations per element.
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

// x / s with the result's last bit set when it is inexact (rounded to odd), so that the
// second rounding, to e4m3, is that of the exact quotient. Infinities and NaN pass.
__device__ __noinline__ float div_to_odd(float x, float s) {
  const float q = __fdiv_rz(x, s);
  if (!isfinite(q)) return q;
  return fmaf(-q, s, x) != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// Two codes of x / s. The product with 1 / s is off by less than 2^-22: only a pair whose
// codes would differ within +-2^-20 of it takes the exact division.
__device__ __forceinline__ uint32_t quantise_e4m3x2(float x, float y, float s, float inv) {
  const float a = x * inv, b = y * inv;
  const uint32_t lo = pack_e4m3x2(a * (1.f - 0x1p-20f), b * (1.f - 0x1p-20f));
  const uint32_t hi = pack_e4m3x2(a * (1.f + 0x1p-20f), b * (1.f + 0x1p-20f));
  return lo == hi ? lo : pack_e4m3x2(div_to_odd(x, s), div_to_odd(y, s));
}

// The lane's eight codes as one word, and its group's (scale, zero) word. The group's
// eight lanes are neighbours; all 32 lanes call it.
__device__ __forceinline__ uint32_t quantise_int4x8(const float (&x)[8], uint32_t& meta) {
  float lo = x[0], hi = x[0], bad = x[0] * 0.f;  // NaN once an element is infinite or NaN
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad = fmaf(x[i], 0.f, bad);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    bad += __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (bad != 0.f) {  // not finite: the group reads back as NaN
    meta = 0x7fc07fc0u;
    return 0u;
  }
  float range = hi - lo;
  range = range < INFINITY ? __fdiv_rn(range, 15.f) : __fdiv_rn(hi, 15.f) - __fdiv_rn(lo, 15.f);
  meta = pack_bf16x2(range, lo);
  const float s = meta_scale(meta);
  if (s == 0.f) return 0u;  // all equal (or nearer than bf16 tells): the zero is the value
  const float inv = __frcp_rn(s);
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = (x[i] - lo) * inv;
    float c = rintf(q);
    // fp32's q is within 15 x 2^-22 of the quotient, unless s is so small that 1 / s overflows
    if (!(fabsf(q - c) < 0.5f - 0x1p-12f) || s < 0x1p-100f)
      c = static_cast<float>(rint((static_cast<double>(x[i]) - static_cast<double>(lo)) / static_cast<double>(s)));
    w |= static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f)) << (4 * i);
  }
  return w;
}

template <int KIND, int D, bool VEC>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int LPR = D / 8;  // lanes per row
  constexpr int ESZ = KIND == kCopy32 ? 4 : 2;
  const int u = threadIdx.x % LPR;
  const uint32_t rows = (uint32_t)a.num_tokens * 2u * (uint32_t)a.Hkv;
  const uint32_t stride = gridDim.x * (kThreads / LPR);
  // All lanes of a warp take part in every step (the groups' shuffles); rows past the end do nothing.
  for (uint32_t r0 = blockIdx.x * (kThreads / LPR); r0 < rows; r0 += stride) {
    const uint32_t r = r0 + threadIdx.x / LPR;
    const uint32_t t = r / (2u * a.Hkv), rem = r - t * (2u * a.Hkv);
    const bool is_v = rem >= (uint32_t)a.Hkv;
    const uint32_t h = is_v ? rem - a.Hkv : rem;
    const int slot = r < rows ? __ldg(&a.slots[t]) : -1;
    const int blk = slot >> 4, tok = slot & (kBlock - 1);
    const bool live = slot >= 0 && blk < a.num_pool_blocks;
    if (slot >= 0 && !live && u == 0) raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
    uint4 x[ESZ / 2];
#pragma unroll
    for (int i = 0; i < ESZ / 2; ++i) x[i] = make_uint4(0, 0, 0, 0);
    if (live) {
      const int64_t off = is_v ? (int64_t)t * a.v_token_stride + (int64_t)h * a.v_head_stride
                               : (int64_t)t * a.k_token_stride + (int64_t)h * a.k_head_stride;
      const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.v : a.k) + (off + 8 * u) * ESZ;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < ESZ / 2; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
      } else if constexpr (ESZ == 4) {
        uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + i);
      } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = __ldg(reinterpret_cast<const uint16_t*>(src) + 2 * i) |
                 (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(src) + 2 * i + 1) << 16;
      }
    }
    uint8_t* pool = is_v ? a.v_pool : a.k_pool;
    const size_t rec = live ? (size_t)blk * a.Hkv + h : 0;
    if constexpr (KIND == kCopy16 || KIND == kCopy32) {
      if (live) {
        uint4* dst = reinterpret_cast<uint4*>(pool + ((rec * kBlock + tok) * D + 8 * u) * ESZ);
#pragma unroll
        for (int i = 0; i < ESZ / 2; ++i) dst[i] = x[i];
      }
    } else if constexpr (KIND == kE4m3) {
      const float s = is_v ? a.v_scale : a.k_scale, inv = is_v ? a.v_inv : a.k_inv;
      float f[8];
      bf16x8_to_f32(x[0], f);
      uint2 c;
      c.x = quantise_e4m3x2(f[0], f[1], s, inv) | quantise_e4m3x2(f[2], f[3], s, inv) << 16;
      c.y = quantise_e4m3x2(f[4], f[5], s, inv) | quantise_e4m3x2(f[6], f[7], s, inv) << 16;
      if (live) *reinterpret_cast<uint2*>(pool + (rec * kBlock + tok) * D + 8 * u) = c;
    } else {
      using G = Int4Geom<D>;
      float f[8];
      bf16x8_to_f32(x[0], f);
      uint32_t meta;
      const uint32_t w = quantise_int4x8(f, meta);
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
  for (uint32_t rec = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); rec < recs; rec += gridDim.x * (kThreads / 32)) {
    const uint32_t i = rec / (2u * a.Hkv), rem = rec - i * (2u * a.Hkv);
    const bool is_v = rem >= (uint32_t)a.Hkv;
    const uint32_t h = is_v ? rem - a.Hkv : rem;
    const int blk = __ldg(&a.block_ids[i]);
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
#pragma unroll
      for (int c = lane; c < BYTES / 16; c += 32)
        reinterpret_cast<uint4*>(out + dst_rec * BYTES)[c] = __ldg(reinterpret_cast<const uint4*>(pool + src_rec * BYTES) + c);
    } else {
      uint32_t w[kBlock / RPW][2];
#pragma unroll
      for (int n = 0; n < kBlock / RPW; ++n) {
        const int row = n * RPW + lane / LPR;
        if constexpr (KIND == kE4m3) {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(pool + (src_rec * kBlock + row) * D + 8 * u));
          w[n][0] = c.x, w[n][1] = c.y;
        } else {
          using G = Int4Geom<D>;
          const uint8_t* base = pool + src_rec * G::REC;
          const int tok = is_v ? int4_v_token(row) : row;
          w[n][0] = __ldg(reinterpret_cast<const uint32_t*>(base + row * G::ROW + 4 * u));
          w[n][1] = __ldg(reinterpret_cast<const uint32_t*>(base + G::META + 4 * (tok * G::NG + u % G::NG)));
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

template <int KIND, int D>
cudaError_t write_t(const CacheWriteArgs& a, bool vec, int sms, cudaStream_t st) {
  const int64_t rows = (int64_t)a.num_tokens * 2 * a.Hkv, per = kThreads / (D / 8);
  const int64_t want = (rows + per - 1) / per, most = (int64_t)sms * 64;
  const unsigned grid = (unsigned)(want < most ? want : most);
  if (vec) cache_write_kernel<KIND, D, true><<<grid, kThreads, 0, st>>>(a);
  else cache_write_kernel<KIND, D, false><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int KIND, int D>
cudaError_t read_t(const CacheReadArgs& a, int sms, cudaStream_t st) {
  const int64_t recs = (int64_t)a.num_blocks * 2 * a.Hkv, per = kThreads / 32;
  const int64_t want = (recs + per - 1) / per, most = (int64_t)sms * 64;
  cache_read_kernel<KIND, D><<<(unsigned)(want < most ? want : most), kThreads, 0, st>>>(a);
  return cudaGetLastError();
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
