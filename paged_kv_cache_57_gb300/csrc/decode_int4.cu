// decode_int4.cu -- the decodes over int4 pools: per sequence (lazy_attn_decode) and over
// shared document runs (lazy_attn_decode_shared). The arithmetic of a tile is in
// int4.cuh; the query rows of a KV head are its heads (per sequence), or members x heads
// (shared).
#include <climits>

#include "decode_block.cuh"
#include "int4.cuh"
#include "kernels.h"

namespace lazy {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 2;  // blocks a warp takes at a time
constexpr int kMembers = LAZY_PLAN_MAX_MEMBERS;
constexpr int kItemInts = LAZY_PLAN_ITEM_INTS;

template <int D, int NT>
struct Int4Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int QS = D + 4;   // fp32 query rows
  static constexpr int RED = D + 4;  // merge rows: o[D], m, l
};

// One warp: a query row of D bf16 values times `scale` to fp32 in shared memory, over the
// power of two that brings its largest value to 1..2; returns that power.
template <int D>
__device__ __forceinline__ float int4_load_row(const __nv_bfloat16* q, float* dst, float scale, int lane) {
  constexpr int PER = D / 32;
  float v[PER], mx = 0.f;
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    v[c] = __bfloat162float(q[lane + 32 * c]) * scale;
    mx = fmaxf(mx, fabsf(v[c]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 27u), 227u);  // 2^(+-100)
  const float inv = __uint_as_float((254u - ex) << 23);
#pragma unroll
  for (int c = 0; c < PER; ++c) dst[lane + 32 * c] = v[c] * inv;
  return __uint_as_float(ex << 23);
}

// A warp's (or a team's first) partial of its rows to shared memory: o[D], m, l per row.
template <int D, int NT>
__device__ __forceinline__ void int4_store_partial(const Int4State<D, NT>& st, float* red, int stride, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float* row = red + (8 * nt + 2 * t + c) * stride;
#pragma unroll
      for (int j = 0; j < Int4Geom<D>::NG; ++j) {
        float v[8];
        int4_out8(st, j, nt, c, v);
        float4* dst = reinterpret_cast<float4*>(row + 64 * j + 8 * g);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      if (g == 0) {
        row[D] = st.m[nt][c];
        row[D + 1] = st.l[nt][c];
      }
    }
}

}  // namespace

// ------------------------------------------------------------------ per sequence
// One CTA per (sequence, KV head and tile of 8 NT query heads, split), four warps with a
// quarter of the split's blocks each, read from global memory as the fragments want them.
template <int D, int NT, bool LAZY>
__global__ void __launch_bounds__(kThreads) decode_int4_kernel(const DecodeArgs a, int head_tiles) {
  using C = Int4Cfg<D, NT>;
  using G = Int4Geom<D>;
  constexpr int HALF = D / 2;
  __shared__ __align__(16) float qs[C::ROWS * C::QS];
  __shared__ float row_scale[C::ROWS];
  __shared__ float2 cs[kWarps][HALF];
  __shared__ __align__(16) float red[kWarps * C::ROWS * C::RED];
  const int split = blockIdx.x, kvh = blockIdx.y / head_tiles, ht = blockIdx.y % head_tiles, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = min(C::ROWS, a.G - ht * C::ROWS);
  const size_t q0 = (size_t)s * a.Hq + (size_t)kvh * a.G + ht * C::ROWS;  // the first row's head
  int seq_len = a.seq_lens[s];
  if (seq_len < 0 || seq_len > kBlock * a.max_blocks) {
    if (threadIdx.x == 0) raise_status(a.status, LAZY_DEV_BAD_LEN);
    seq_len = seq_len < 0 ? 0 : kBlock * a.max_blocks;
  }
  const int nb = (seq_len + kBlock - 1) / kBlock;
  const int b0 = split * a.bps;
  const int n = max(0, min(nb, b0 + a.bps) - b0);
  if (n == 0 && a.splits > 1) return;  // the combine does not look here
  const int m_pos = a.q_pos[s];
  const uint32_t* wrow = a.words + (size_t)s * a.max_blocks;
  for (int r = warp; r < C::ROWS; r += kWarps) {
    if (r < heads) {
      const float sc = int4_load_row<D>(static_cast<const __nv_bfloat16*>(a.q) + (q0 + r) * D, qs + r * C::QS, a.scale_log2, lane);
      if (lane == 0) row_scale[r] = sc;
    } else {
      for (int c = lane; c < D; c += 32) qs[r * C::QS + c] = 0.f;
      if (lane == 0) row_scale[r] = 1.f;
    }
  }
  __syncthreads();

  const int per_warp = (n + kWarps - 1) / kWarps;
  const int kb0 = warp * per_warp;
  const int nk = max(0, min(n, kb0 + per_warp) - kb0);
  const size_t head_off = (size_t)kvh * G::REC, blk_bytes = (size_t)a.Hkv * G::REC;
  const uint8_t* kp = static_cast<const uint8_t*>(a.k_pool) + head_off;
  const uint8_t* vp = static_cast<const uint8_t*>(a.v_pool) + head_off;
  Int4Query<D, NT> q;
  Int4State<D, NT> st;
  int4_init(st);
  LaneBlock cur{a.num_pool_blocks, 0, 0};
  int delta = INT_MIN;
  bool built = false;
  for (int k = 0, step = 0; k < nk; k += step) {
    const int at = k & 31;
    if (at == 0) {
      const int i = k + lane, b = b0 + kb0 + i;
      const uint32_t w = i < nk ? __ldg(&wrow[b]) : 0u;
      const uint32_t wn = (i < nk && b + 1 < nb) ? __ldg(&wrow[b + 1]) : 0u;
      cur = describe_block(i < nk, b, nb, seq_len, w, wn, a.id_bits, a.num_pool_blocks, a.status);
    }
    const int p = __shfl_sync(0xffffffffu, cur.p, at);
    const int p2 = __shfl_sync(0xffffffffu, cur.p, (at + 1) & 31);
    const bool two = at < 31 && k + 1 < nk && (p2 == p || !LAZY);  // a tile lies in one document
    step = two ? 2 : 1;
    const int dnew = LAZY ? m_pos - p : m_pos;
    if (!built || dnew != delta) {
      delta = dnew;
      built = true;
      __syncwarp();
      for (int f = lane; f < HALF; f += 32) cs[warp][f] = rope_cs(__ldg(&a.rope[f]), delta, a.status);
      __syncwarp();
      int4_build_query<D, NT>(
          q, lane, [&](int r, int d) { return qs[r * C::QS + d]; }, [&](int, int f) { return cs[warp][f]; },
          [&](int r) { return row_scale[r]; });
    }
    GlobalRecord kr[kTile], vr[kTile];
    int nv[kTile];
#pragma unroll
    for (int b = 0; b < kTile; ++b) {
      const int ph = __shfl_sync(0xffffffffu, cur.phys, (at + b) & 31);
      nv[b] = __shfl_sync(0xffffffffu, cur.nv, (at + b) & 31);
      if (b > 0 && !two) nv[b] = 0;
      const size_t off = (size_t)(nv[b] > 0 ? ph : 0) * blk_bytes;  // no keys: any record of the pool
      kr[b].p = kp + off;
      vr[b].p = vp + off;
    }
    int4_attend<D, NT, kTile>(kr, vr, nv, q, st, lane);
  }
  int4_finish(st);
  int4_store_partial(st, red + warp * C::ROWS * C::RED, C::RED, lane);
  __syncthreads();
  for (int idx = threadIdx.x; idx < heads * D; idx += kThreads) {
    const int row = idx / D, col = idx % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[(w * C::ROWS + row) * C::RED + D]);
    float acc = 0.f, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* src = red + (w * C::ROWS + row) * C::RED;
      const float f = src[D] == -INFINITY ? 0.f : exp2f(src[D] - M);
      acc += f * src[col];
      L += f * src[D + 1];
    }
    if (a.splits == 1) {
      static_cast<__nv_bfloat16*>(a.out)[(q0 + row) * D + col] = __float2bfloat16_rn(L > 0.f || L != L ? acc / L : 0.f);
    } else {
      const size_t pidx = (q0 + row) * a.splits + split;
      a.ws_o[pidx * D + col] = acc;
      if (col == 0) {
        a.ws_ml[2 * pidx] = M;
        a.ws_ml[2 * pidx + 1] = L;
      }
    }
  }
}

// ------------------------------------------------------------------ shared runs
// One CTA per (work item, KV head). The item's rows (members x heads, at most 64) are
// tiles of 16; the warps form 4 / RT teams of RT warps, a team with a contiguous part of
// the item's blocks and a warp with one of its tiles, as in decode_shared.cu.
template <int D, bool LAZY>
__global__ void __launch_bounds__(kThreads) decode_shared_int4_kernel(const SharedDecodeArgs a, const uint8_t* k_pool,
                                                                      const uint8_t* v_pool) {
  constexpr int NT = 2;
  using C = Int4Cfg<D, NT>;
  using G = Int4Geom<D>;
  constexpr int HALF = D / 2, MAX_ROWS = 64;
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;                             // [64][QS], then the merge area [teams][rows][RED]
  float2* cs_tab = reinterpret_cast<float2*>(smem + MAX_ROWS * C::QS);  // [members][HALF]
  __shared__ int rec[kItemInts], m_delta[kMembers], m_ok[kMembers];
  __shared__ float row_scale[MAX_ROWS];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv, item = blockIdx.x / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kItemInts / 4)
    reinterpret_cast<int4*>(rec)[threadIdx.x] =
        __ldg(reinterpret_cast<const int4*>(a.items) + (size_t)item * (kItemInts / 4) + threadIdx.x);
  __syncthreads();
  const int src = rec[0], b0 = rec[1], nblk = rec[2], last_nv = rec[3], nmem = rec[4];
  const bool item_ok = src >= 0 && src < a.B && b0 >= 0 && nblk >= 1 && nblk <= a.max_blocks - b0 &&
                       last_nv >= 1 && last_nv <= kBlock && nmem >= 1 && nmem <= kMembers && nmem * a.G <= MAX_ROWS;
  if (!item_ok) {  // uniform over the CTA: nothing is loaded or written
    if (threadIdx.x == 0) raise_status(a.status, LAZY_DEV_LAYOUT);
    return;
  }
  auto mem_seq = [&](int m) { return rec[8 + 4 * m]; };
  auto mem_slot = [&](int m) { return rec[8 + 4 * m + 2]; };
  if (threadIdx.x < nmem) {
    const int m = threadIdx.x, seq = mem_seq(m), bm = rec[8 + 4 * m + 1], slot = mem_slot(m);
    bool good = seq >= 0 && seq < a.B && bm >= 0 && bm <= a.max_blocks - nblk && slot >= 0 && slot < a.num_slots;
    int delta = 0;
    if (good) {
      const BlockInfo mi = decode_word(__ldg(&a.words[(size_t)seq * a.max_blocks + bm]), bm, a.id_bits);
      good = mi.phys == decode_word(__ldg(&a.words[(size_t)src * a.max_blocks + b0]), b0, a.id_bits).phys;
      const int qp = __ldg(&a.q_pos[seq]);
      delta = LAZY ? qp - mi.p : qp;
    }
    if (!good) raise_status(a.status, LAZY_DEV_LAYOUT);
    m_ok[m] = good;
    m_delta[m] = delta;
  }
  __syncthreads();
  const int rows = nmem * a.G;
  const int RT = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4), TEAMS = kWarps / RT;
  const int team = warp / RT, rt = warp % RT;
  for (int r = warp; r < 16 * RT; r += kWarps) {
    const int m = r / a.G;
    if (r < rows && m_ok[m]) {
      const size_t qh = (size_t)mem_seq(m) * a.Hq + (size_t)kvh * a.G + (r - m * a.G);
      const float sc = int4_load_row<D>(static_cast<const __nv_bfloat16*>(a.q) + qh * D, qs + r * C::QS, a.scale_log2, lane);
      if (lane == 0) row_scale[r] = sc;
    } else {
      for (int c = lane; c < D; c += 32) qs[r * C::QS + c] = 0.f;
      if (lane == 0) row_scale[r] = 1.f;
    }
  }
  for (int idx = threadIdx.x; idx < nmem * HALF; idx += kThreads)
    cs_tab[idx] = rope_cs(__ldg(&a.rope[idx % HALF]), m_delta[idx / HALF], a.status);
  __syncthreads();
  Int4Query<D, NT> q;
  int4_build_query<D, NT>(
      q, lane, [&](int r, int d) { return qs[(16 * rt + r) * C::QS + d]; },
      [&](int r, int f) { return cs_tab[(16 * rt + r < rows ? (16 * rt + r) / a.G : 0) * HALF + f]; },
      [&](int r) { return row_scale[16 * rt + r]; });
  Int4State<D, NT> st;
  int4_init(st);
  const int per_team = (nblk + TEAMS - 1) / TEAMS;
  const int kb0 = team * per_team;
  const int nk = max(0, min(nblk, kb0 + per_team) - kb0);
  const uint32_t* wrow = a.words + (size_t)src * a.max_blocks + b0 + kb0;
  const uint32_t id_mask = (1u << a.id_bits) - 1u;
  const size_t head_off = (size_t)kvh * G::REC, blk_bytes = (size_t)a.Hkv * G::REC;
  int c_phys = 0, c_nv = 0;
  for (int k = 0; k < nk; k += kTile) {
    if ((k & 31) == 0) {
      const int i = k + lane;
      c_phys = c_nv = 0;
      if (i < nk) {
        const int ph = (int)(__ldg(&wrow[i]) & id_mask);
        if (kb0 + i < LAZY_PLAN_ITEM_BLOCK_IDS && rec[8 + 4 * kMembers + kb0 + i] != ph) {
          raise_status(a.status, LAZY_DEV_LAYOUT);
        } else if (ph < a.num_pool_blocks) {
          c_phys = ph;
          c_nv = kb0 + i == nblk - 1 ? last_nv : kBlock;
        } else {
          raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
        }
      }
    }
    GlobalRecord kr[kTile], vr[kTile];
    int nv[kTile];
#pragma unroll
    for (int b = 0; b < kTile; ++b) {
      const int ph = __shfl_sync(0xffffffffu, c_phys, (k + b) & 31);
      nv[b] = __shfl_sync(0xffffffffu, c_nv, (k + b) & 31);
      const size_t off = (size_t)ph * blk_bytes + head_off;
      kr[b].p = k_pool + off;
      vr[b].p = v_pool + off;
    }
    int4_attend<D, NT, kTile>(kr, vr, nv, q, st, lane);
  }
  int4_finish(st);
  __syncthreads();  // every warp has read its queries: the merge takes their place
  const int trows = 16 * RT;
  int4_store_partial(st, smem + (team * trows + 16 * rt) * C::RED, C::RED, lane);
  __syncthreads();
  constexpr int PER = D / 32;
  for (int r = warp; r < rows; r += kWarps) {
    const int m = r / a.G, h = r - m * a.G;
    if (mem_slot(m) < 0 || mem_slot(m) >= a.num_slots) continue;
    float M = -INFINITY, acc[PER], L = 0.f;
    if (m_ok[m])  // a member that failed its checks leaves an empty partial
      for (int tm = 0; tm < TEAMS; ++tm) M = fmaxf(M, smem[(tm * trows + r) * C::RED + D]);
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = 0.f;
    if (m_ok[m])
      for (int tm = 0; tm < TEAMS; ++tm) {
        const float* row = smem + (tm * trows + r) * C::RED;
        const float w = row[D] == -INFINITY ? 0.f : fast_ex2(row[D] - M);
        L += w * row[D + 1];
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] += w * row[lane + 32 * c];
      }
    const size_t pidx = (size_t)mem_slot(m) * a.Hq + (size_t)kvh * a.G + h;
#pragma unroll
    for (int c = 0; c < PER; ++c) a.ws_o[pidx * D + lane + 32 * c] = acc[c];
    if (lane == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * pidx) = make_float2(M, L);
  }
}

// ------------------------------------------------------------------ launchers

template <int D, int NT>
static cudaError_t launch_decode_t(const DecodeArgs& a, bool lazy, cudaStream_t st) {
  const int ht = (a.G + 8 * NT - 1) / (8 * NT);
  const dim3 grid(a.splits, a.Hkv * ht, a.B);
  if (lazy) decode_int4_kernel<D, NT, true><<<grid, kThreads, 0, st>>>(a, ht);
  else decode_int4_kernel<D, NT, false><<<grid, kThreads, 0, st>>>(a, ht);
  return cudaGetLastError();
}

cudaError_t launch_decode_int4(const DecodeArgs& a, bool lazy, cudaStream_t st) {
  if (a.D == 128) return a.G <= 8 ? launch_decode_t<128, 1>(a, lazy, st) : launch_decode_t<128, 2>(a, lazy, st);
  return a.G <= 8 ? launch_decode_t<64, 1>(a, lazy, st) : launch_decode_t<64, 2>(a, lazy, st);
}

template <int D, bool LAZY>
static cudaError_t launch_shared_t(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, cudaStream_t st) {
  constexpr int SMEM = 64 * (D + 4) * 4 + kMembers * (D / 2) * 8;
  cudaError_t e = set_smem_once<decode_shared_int4_kernel<D, LAZY>>(SMEM);
  if (e != cudaSuccess) return e;
  decode_shared_int4_kernel<D, LAZY><<<(unsigned)((long long)a.num_items * a.Hkv), kThreads, SMEM, st>>>(
      a, static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool));
  return cudaGetLastError();
}

cudaError_t launch_decode_shared_int4(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, bool lazy,
                                      cudaStream_t st) {
  if (a.num_items == 0) return cudaSuccess;
  if (a.D == 128)
    return lazy ? launch_shared_t<128, true>(a, k_pool, v_pool, st) : launch_shared_t<128, false>(a, k_pool, v_pool, st);
  return lazy ? launch_shared_t<64, true>(a, k_pool, v_pool, st) : launch_shared_t<64, false>(a, k_pool, v_pool, st);
}

}  // namespace lazy
