// cache_fp8_block.cu -- rows into pools of e4m3 codes with a scale per block and head, and blocks
// back out of them (lazy_attn_cache_write, lazy_attn_cache_read; format in fp8_block.cuh).
//
// Write: a block's scale is 2^e with the least e that holds the greatest of the written rows, and
// at least the old e where the block goes on (row 0 is not written). So rows are written a block at a time: a
// warp takes the tokens of a call that go into one block, for one KV head of K or V (a "run"). It finds
// them around the run's first token in `slots`, loads their rows in the order of the record's chunks (a
// lane's rows give its own chunks whole), takes the maximum across the warp, and writes the
// chunks that hold one of the rows. The other rows' codes are touched only where the scale
// grows: a power of two, so that a code of 4 bits changes only where it falls below e4m3's least step.
// A step's 64 tokens of 8 heads take 2.8 us in a graph (latency: slots, rows, record), 16384 tokens of
// documents 22.5 us, 4.5 TB/s: 67% of the measured copy, issue slots 60%, 44% of the warps resident. A run's loads,
// maximum, conversions and stores follow one another in its warp; which of them it waits for most was not separated.
//
// Read: 1024 blocks of 8 heads 17.0 us, 5.9 TB/s: memory.
#include "fp8_block.cuh"
#include "kernels.h"

namespace lazy {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kExpMin = -100, kExpMax = 119;  // 448 * 2^119 is bf16's last binade

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Whether a record's scale is one that a write leaves: 2^e of the range. (A pool that nothing wrote holds anything.)
__device__ __forceinline__ bool is_scale(uint32_t bits) {
  return (bits & 0x7fffffu) == 0u && bits >> 23 >= (uint32_t)(kExpMin + 127) && bits >> 23 <= (uint32_t)(kExpMax + 127);
}

// The least e with m <= 448 * 2^e = 1.75 * 2^(e + 8), for bf16 bits m of a finite value >= 0.
__device__ __forceinline__ int exponent_for(uint32_t m) {
  const int e = (int)(m >> 7) - 127 - 8 + ((m & 127u) > 96u ? 1 : 0);
  return min(max(e, kExpMin), kExpMax);
}

// Eight consecutive bf16 values.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint8_t* p) {
  if constexpr (VEC) return *reinterpret_cast<const uint4*>(p);
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t abs_max(uint32_t m, const uint4& x) {
  return __vmaxu2(__vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu)), x.w & 0x7fff7fffu);
}

// The two bf16 values of a word, those that are not finite dropped (drop = 0) or NaN.
__device__ __forceinline__ uint32_t bad_as(uint32_t w, uint32_t to) {
  if ((w & 0x7f80u) == 0x7f80u) w = (w & 0xffff0000u) | (to & 0xffffu);
  if ((w & 0x7f800000u) == 0x7f800000u) w = (w & 0xffffu) | (to & 0xffff0000u);
  return w;
}
__device__ __forceinline__ uint4 bad_as(const uint4& x, uint32_t to) {
  return make_uint4(bad_as(x.x, to), bad_as(x.y, to), bad_as(x.z, to), bad_as(x.w, to));
}

// Two codes times 2^d, rounded (nearest even; NaN kept), d <= 0.
__device__ __forceinline__ uint32_t rescale2(uint32_t pair16, float by) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair16));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_e4m3x2(f.x * by, f.y * by);
}
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float by) { return rescale2(w & 0xffffu, by) | rescale2(w >> 16, by) << 16; }
__device__ __forceinline__ uint4 rescale16(const uint4& x, float by) {
  return make_uint4(rescale4(x.x, by), rescale4(x.y, by), rescale4(x.z, by), rescale4(x.w, by));
}

// Codes of the values of a and b: of a's four words in K's order (eight neighbouring dims)...
__device__ __forceinline__ uint2 codes8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = pack_e4m3x2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// ... and of both in V's, token a's beside token b's.
__device__ __forceinline__ uint4 codes16(const uint4& a, const uint4& b, float inv) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = pack_e4m3x2(bf16_lo(x[i]) * inv, bf16_lo(y[i]) * inv) | pack_e4m3x2(bf16_hi(x[i]) * inv, bf16_hi(y[i]) * inv) << 16;
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// A warp's run: `rowtok`[r] is the token whose row goes to row r of the record, or -1. Row n of
// the lane's rows x[n] and, of K, its two halves of 16 dims.
template <int D, bool IS_V, bool VEC>
__device__ __forceinline__ void write_run(const uint8_t* src, int64_t step, const int* rowtok, uint32_t rowmask, uint8_t* rec,
                                          int lane) {
  using G = Fp8Geom<D>;
  constexpr int NG = G::NG;
  constexpr int ROWS = IS_V ? 4 : 2;        // rows of the lane: V 2t, 2t + 1, 2t + 8, 2t + 9; K g, g + 8
  constexpr int PER = G::CHUNKS * 2 / ROWS;  // loads of eight dims of each
  const int g = lane >> 2, t = lane & 3;
  auto row_of = [&](int n) { return IS_V ? 2 * t + (n & 1) + 8 * (n >> 1) : g + 8 * n; };
  uint4 x[ROWS][PER];
  uint32_t m = 0u;
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const int tok = rowtok[row_of(n)];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // V: dims 8 (g + 8 i); K: 16 (t + 4 (i / 2)) + 8 (i % 2)
      const int dim = IS_V ? 8 * g + 64 * i : 64 * (i / 2) + 16 * t + 8 * (i % 2);
      x[n][i] = make_uint4(0, 0, 0, 0);
      if (tok >= 0) x[n][i] = load8<VEC>(src + tok * step + 2 * dim);
      m = abs_max(m, x[n][i]);
    }
  }
  const uint32_t was = rowmask & 1u ? 0u : *reinterpret_cast<const uint32_t*>(rec + G::SCALE);
  const bool anew = !is_scale(was);
  const int e_old = anew ? kExpMin : (int)(was >> 23) - 127;
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if (m >= 0x7f80u) {  // infinities and NaN do not count, and are written as NaN
    m = 0u;
#pragma unroll
    for (int n = 0; n < ROWS; ++n)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        m = abs_max(m, bad_as(x[n][i], 0u));
        x[n][i] = bad_as(x[n][i], 0x7fc07fc0u);
      }
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  }
  const int e = max(exponent_for(m), e_old);
  const bool grown = !anew && e > e_old;
  const float inv = pow2f(-e), by = pow2f(e_old - e < -120 ? -120 : e_old - e);
  uint4* dst = reinterpret_cast<uint4*>(rec) + lane;
#pragma unroll
  for (int j = 0; j < G::CHUNKS; ++j) {
    if constexpr (IS_V) {
      const int jlo = j % NG, n = 2 * (j / NG);
      const bool in0 = rowmask >> row_of(n) & 1u, in1 = rowmask >> row_of(n + 1) & 1u;
      if (!(anew || grown || in0 || in1)) continue;
      uint4 c = codes16(x[n][jlo], x[n + 1][jlo], inv);
      if (!anew && !(in0 && in1)) {
        uint4 old = dst[32 * j];
        if (grown) old = rescale16(old, by);
        const uint32_t keep = (in0 ? 0u : 0x00ff00ffu) | (in1 ? 0u : 0xff00ff00u);
        c = make_uint4((c.x & ~keep) | (old.x & keep), (c.y & ~keep) | (old.y & keep), (c.z & ~keep) | (old.z & keep),
                       (c.w & ~keep) | (old.w & keep));
      }
      dst[32 * j] = c;
    } else {
      const int n = j % 2, i = 2 * (j / 2);
      const bool in = rowmask >> row_of(n) & 1u;
      if (in || anew) {
        const uint2 lo = codes8(x[n][i], inv), hi = codes8(x[n][i + 1], inv);
        dst[32 * j] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else if (grown) {
        dst[32 * j] = rescale16(dst[32 * j], by);
      }
    }
  }
  if (lane == 0 && (anew || grown)) *reinterpret_cast<float*>(rec + G::SCALE) = pow2f(e);
}

// A warp per (W tokens, K or V, KV head): the runs that begin among the tokens.
template <int D, bool VEC, int W>
__global__ void __launch_bounds__(kThreads, 4) cache_write_fp8_block_kernel(const CacheWriteArgs a) {
  __shared__ int rowtok_all[kWarps][kBlock];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* rowtok = rowtok_all[warp];
  const uint32_t per_window = 2u * (uint32_t)a.Hkv;
  const uint32_t r = blockIdx.x * kWarps + warp, win = r / per_window;  // (window, K or V, head)
  uint32_t h = r - win * per_window;
  const bool is_v = h >= (uint32_t)a.Hkv;
  if (is_v) h -= a.Hkv;
  const int64_t base = (int64_t)win * W;
  if (base >= a.num_tokens) return;
  const int64_t step = 2 * (is_v ? a.v_token_stride : a.k_token_stride);
  const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.v : a.k) + 2 * (is_v ? a.v_head_stride : a.k_head_stride) * h;
  uint8_t* pool = is_v ? a.v_pool : a.k_pool;
  wait_for_launch_before();
  // the slots of 32 tokens before the window, of the window's and of what may follow
  auto slot_at = [&](int64_t t) { return t >= 0 && t < a.num_tokens ? a.slots[t] : -1; };
  const int before = slot_at(base - 32 + lane), at = slot_at(base + lane), after = W > 1 ? slot_at(base + 32 + lane) : -1;
#pragma unroll 1
  for (int i = 0; i < W; ++i) {
    const int first = __shfl_sync(0xffffffffu, at, i);
    if (first < 0) continue;
    const int blk = first >> 4;
    if (blk >= a.num_pool_blocks) {
      if (lane == 0) raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
      continue;
    }
    // (slots of padding are negative, and so is a sixteenth of them)
    const bool earlier = (lane > i && before >> 4 == blk) || (lane < i && at >> 4 == blk);
    if (__any_sync(0xffffffffu, earlier)) continue;  // the run began there
    if (lane < kBlock) rowtok[lane] = -1;
    __syncwarp();
    if (lane >= i && at >> 4 == blk) rowtok[at & 15] = (int)base + lane;
    if (lane < i && after >> 4 == blk) rowtok[after & 15] = (int)base + 32 + lane;
    __syncwarp();
    const uint32_t rowmask = __ballot_sync(0xffffffffu, lane < kBlock && rowtok[lane & 15] >= 0);
    uint8_t* rec = pool + ((size_t)(uint32_t)blk * (uint32_t)a.Hkv + h) * Fp8Geom<D>::REC;
    if (is_v) write_run<D, true, VEC>(src, step, rowtok, rowmask, rec, lane);
    else write_run<D, false, VEC>(src, step, rowtok, rowmask, rec, lane);
    __syncwarp();  // before the next run's rows take the list
  }
}

// Two e4m3 codes times a power of two as bf16 (exact below bf16's greatest value).
__device__ __forceinline__ uint32_t bf16_of(uint32_t pair16, float s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair16));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x * s, f.y * s);
}

// A warp per (block, K or V, KV head): 16-byte stores that fill whole lines. Of V a lane has eight dims
// of two tokens; of K it takes half a chunk, eight dims.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_fp8_block_kernel(const CacheReadArgs a) {
  using G = Fp8Geom<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t recs = (uint32_t)a.num_blocks * 2u * (uint32_t)a.Hkv;
  wait_for_launch_before();
  for (uint32_t r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < recs; r += gridDim.x * kWarps) {
    const uint32_t i = r / (2u * a.Hkv), rem = r - i * (2u * a.Hkv);
    const bool is_v = rem >= (uint32_t)a.Hkv;
    const uint32_t h = is_v ? rem - a.Hkv : rem;
    const int blk = a.block_ids[i];
    if (blk < 0) continue;  // padding: its rows stay as they are
    if (blk >= a.num_pool_blocks) {
      if (lane == 0) raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
      continue;
    }
    const uint8_t* rec = (is_v ? a.v_pool : a.k_pool) + ((size_t)(uint32_t)blk * (uint32_t)a.Hkv + h) * G::REC;
    uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_out : a.k_out) + ((size_t)i * a.Hkv + h) * kBlock * D * 2;
    const float s = *reinterpret_cast<const float*>(rec + G::SCALE);
    if (is_v) {
      uint4 c[G::CHUNKS];
#pragma unroll
      for (int j = 0; j < G::CHUNKS; ++j) c[j] = reinterpret_cast<const uint4*>(rec)[32 * j + lane];
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int j = 0; j < G::CHUNKS; ++j) {
        const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
        uint32_t o[2][4];  // the tokens' words
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // codes (dim 2k: both tokens, dim 2k + 1: both tokens) to (token: both dims)
          const uint32_t x = __byte_perm(w[k], 0u, 0x4420), y = __byte_perm(w[k], 0u, 0x4431);
          o[0][k] = bf16_of(x, s);
          o[1][k] = bf16_of(y, s);
        }
        const int dim = 8 * (g + 8 * (j % G::NG)), tok = 2 * (t + 4 * (j / G::NG));
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(out + ((tok + k) * D + dim) * 2) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
      }
    } else {
      uint2 c[2 * G::CHUNKS];
#pragma unroll
      for (int j = 0; j < 2 * G::CHUNKS; ++j) c[j] = reinterpret_cast<const uint2*>(rec)[32 * j + lane];
#pragma unroll
      for (int j = 0; j < 2 * G::CHUNKS; ++j) {
        const int chunk = 16 * j + (lane >> 1), g = chunk % 32 / 4, t = chunk % 4;
        const int tok = g + 8 * (chunk / 32 % 2), dim = 16 * (t + 4 * (chunk / 64)) + 8 * (lane & 1);
        *reinterpret_cast<uint4*>(out + (tok * D + dim) * 2) =
            make_uint4(bf16_of(c[j].x & 0xffffu, s), bf16_of(c[j].x >> 16, s), bf16_of(c[j].y & 0xffffu, s), bf16_of(c[j].y >> 16, s));
      }
    }
  }
}

template <int D, int W>
cudaError_t write_w(const CacheWriteArgs& a, bool vec, cudaStream_t st) {
  const int64_t warps = ((int64_t)a.num_tokens + W - 1) / W * 2 * a.Hkv;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  return launch_behind(vec ? cache_write_fp8_block_kernel<D, true, W> : cache_write_fp8_block_kernel<D, false, W>, grid, kThreads, 0, st, a);
}

// A window of one token finds every run at once, but in a document fifteen warps of sixteen find that
// theirs began before; windows of a block's length waste none, and take the runs among them in turn. 64
// tokens of 64 sequences took 2.8 us with windows of one token and 24.6 with 16, 16384 tokens of documents 54.5 and
// 22.5 (8 heads); 4378 of 2 heads 4.2 and 4.7. Windows of one up to what is resident four times over.
template <int D>
cudaError_t write_d(const CacheWriteArgs& a, bool vec, int sms, cudaStream_t st) {
  return (int64_t)a.num_tokens * 2 * a.Hkv <= (int64_t)sms * 128 ? write_w<D, 1>(a, vec, st) : write_w<D, kBlock>(a, vec, st);
}

template <int D>
cudaError_t read_d(const CacheReadArgs& a, int sms, cudaStream_t st) {
  const int64_t recs = (int64_t)a.num_blocks * 2 * a.Hkv;
  const int64_t want = (recs + kWarps - 1) / kWarps, most = (int64_t)sms * 64;
  return launch_behind(cache_read_fp8_block_kernel<D>, (unsigned)(want < most ? want : most), kThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_cache_write_fp8_block(const CacheWriteArgs& a, bool vec, int sms, cudaStream_t st) {
  return a.D == 128 ? write_d<128>(a, vec, sms, st) : write_d<64>(a, vec, sms, st);
}

cudaError_t launch_cache_read_fp8_block(const CacheReadArgs& a, int sms, cudaStream_t st) {
  return a.D == 128 ? read_d<128>(a, sms, st) : read_d<64>(a, sms, st);
}

}  // namespace lazy
