// decode_units.cu -- the plan of the per-sequence decodes over packed pools, and the join of the
// parts that they leave (decode_units.cuh).
#include <algorithm>
#include <climits>

#include "decode_units.cuh"

namespace lazy {

// out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c over the parts of a unit of several pieces
// or in several ranges; with ranges 0 for a sequence without blocks (with pieces its unit's CTA
// writes that). A CTA looks after PAIRS (sequence, query head) pairs: a warp finds a pair's parts
// and merges up to kCombineBatch of them by itself; more are shared by the CTA's warps. Launched
// as a programmatic dependent of the decode kernel: it waits for that grid before it reads
// anything.
//
// Up to kCombineAlone pairs, as many CTAs as are resident at once, get a CTA each: whole
// calls of 32 heads took 21 us at 1 x 16384 tokens and at 4 x 4096, with PAIRS = 8 30 and 29.
// Most of a large batch's pairs have nothing to merge, and CTAs that find that out come in
// waves: at 64 x 4160 tokens PAIRS = 8 took 73.5 us, a CTA per pair 80.
constexpr int kCombineWarps = 8, kCombineBatch = 8, kCombineAlone = 3 * 152;

namespace {

template <int D>
struct Merged {
  static constexpr int PER = D / 32;
  float M, L, acc[PER];
  // Parts first, first + step, ... of a row's n, a lane the columns lane + 32 i. Part i is CTA c0 + i stride's.
  __device__ __forceinline__ Merged(const UnitDecodeArgs& a, int row, int c0, int n, int stride, int first, int step) {
    const int lane = threadIdx.x & 31;
    M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    for (int cb = first; cb < n; cb += step * kCombineBatch) {
      float2 ml[kCombineBatch];
      float v[kCombineBatch][PER];
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {
        const int c = cb + b * step;
        ml[b] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[b][i] = 0.f;
        if (c < n) {
          const size_t p = (2 * ((size_t)c0 + (size_t)c * stride) + (c == 0 ? 1 : 0)) * a.plan.rows + row;
          ml[b] = *reinterpret_cast<const float2*>(a.ws_ml + 2 * p);
#pragma unroll
          for (int i = 0; i < PER; ++i) v[b][i] = a.ws_o[p * D + lane + 32 * i];
        }
      }
      float Mn = M;
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) Mn = fmaxf(Mn, ml[b].x);
      const float Mr = Mn == -INFINITY ? 0.f : Mn;
      const float r = fast_ex2(M - Mr);
      L *= r;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= r;
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {
        const float w = fast_ex2(ml[b].x - Mr);  // an empty part (m = -inf) weighs 0
        L = fmaf(w, ml[b].y, L);
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = fmaf(w, v[b][i], acc[i]);
      }
      M = Mn;
    }
  }
};

}  // namespace

template <int D, int PAIRS>
__global__ void __launch_bounds__(32 * kCombineWarps) combine_units_kernel(const UnitDecodeArgs a) {
  constexpr int PER = D / 32;
  __shared__ float red[kCombineWarps][D + 2];
  __shared__ int2 parts[PAIRS];  // what the CTA's warps share: first part's CTA and parts; 0 or 1: nothing to merge
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t pair0 = (int64_t)blockIdx.x * PAIRS, pairs = (int64_t)a.B * a.Hq;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  auto row_of = [&](int64_t pair) { return (int)(pair % a.Hq) % a.G % a.plan.rows; };
  wait_for_launch_before();
  const bool ranges = a.plan.range_ctas > 0 && a.prefix[a.B + 1] != 0;
  const int stride = ranges ? 1 : a.B * a.plan.units;
  if (warp < PAIRS) {
    const int64_t pair = pair0 + warp;
    int2 mine = make_int2(0, 0);
    if (pair < pairs) {
      const int s = (int)(pair / a.Hq), h = (int)(pair - (int64_t)s * a.Hq), kvh = h / a.G;
      const int u = kvh * (a.plan.units / a.Hkv) + (h - kvh * a.G) / a.plan.rows;
      if (ranges) {
        const int64_t p0 = a.prefix[s], len = a.prefix[s + 1] - p0, lo = p0 * a.plan.units + u * len;
        const int64_t chunk = chunk_of(a, a.prefix[a.B] * a.plan.units);
        if (len == 0) {
#pragma unroll
          for (int i = 0; i < PER; ++i) out[pair * D + lane + 32 * i] = __float2bfloat16_rn(0.f);
        } else {
          const int64_t c0 = lo / chunk;
          mine = make_int2((int)c0, (int)((lo + len - 1) / chunk - c0) + 1);  // in one range: written there
        }
      } else {
        int seq_len;
        const int nb = blocks_of(a, s, seq_len), len = piece_of(a.plan, nb);
        mine = make_int2(s * a.plan.units + u, nb > len ? (nb + len - 1) / len : 1);  // of one piece: written there
      }
      if (PAIRS > 1 && mine.y > 1 && mine.y <= kCombineBatch) {
        const Merged<D> m(a, row_of(pair), mine.x, mine.y, stride, 0, 1);
#pragma unroll
        for (int i = 0; i < PER; ++i) out[pair * D + lane + 32 * i] = __float2bfloat16_rn(m.L == 0.f ? 0.f : m.acc[i] / m.L);
        mine.y = 0;
      }
    }
    if (lane == 0) parts[warp] = mine;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < PAIRS; ++i) {
    const int2 p = parts[i];
    if (p.y <= 1) continue;
    const Merged<D> m(a, row_of(pair0 + i), p.x, p.y, stride, warp, kCombineWarps);
#pragma unroll
    for (int j = 0; j < PER; ++j) red[warp][lane + 32 * j] = m.acc[j];
    if (lane == 0) {
      red[warp][D] = m.M;
      red[warp][D + 1] = m.L;
    }
    __syncthreads();
    for (int col = threadIdx.x; col < D; col += 32 * kCombineWarps) {
      float Ma = -INFINITY, x = 0.f, La = 0.f;
#pragma unroll
      for (int w = 0; w < kCombineWarps; ++w) Ma = fmaxf(Ma, red[w][D]);
      if (Ma == -INFINITY) Ma = 0.f;
#pragma unroll
      for (int w = 0; w < kCombineWarps; ++w) {
        const float f = fast_ex2(red[w][D] - Ma);
        x += f * red[w][col];
        La += f * red[w][D + 1];
      }
      out[(pair0 + i) * D + col] = __float2bfloat16_rn(La == 0.f ? 0.f : x / La);
    }
    __syncthreads();
  }
}

UnitPlan plan_units(int B, int rows, int units, int max_blocks, int num_splits, int64_t resident, int least_log2, int most) {
  UnitPlan p{};
  p.rows = rows;
  p.units = units;
  const int mb = max_blocks > 0 ? max_blocks : 1;
  const int64_t all = (int64_t)(B > 0 ? B : 1) * units;
  p.least_log2 = num_splits > 0 ? 0 : least_log2;
  p.splits = num_splits > 0 ? std::min(num_splits, mb)
                            : (int)std::max<int64_t>(1, std::min<int64_t>(resident / all, mb >> least_log2));
  if (num_splits > 0) p.splits = (int)std::max<int64_t>(p.splits, ((int64_t)mb + most - 1) / most);  // (else kMaxPiece or a range)
  p.ctas = all * p.splits;
  p.parts = p.splits > 1 ? p.ctas : 0;
  if (num_splits <= 0 && mb > kMaxPiece * p.splits) {
    p.range_ctas = std::max(std::min<int64_t>((all * mb + kMinChunk - 1) / kMinChunk, resident), (all * mb + most - 1) / most);
    p.ctas = B > kMaxLook ? p.range_ctas : std::max(p.ctas, p.range_ctas);
    p.parts = std::max(p.parts, p.range_ctas);
  }
  return p;
}

int64_t longest_part(const UnitPlan& p, int B, int max_blocks) {
  if (p.range_ctas == 0) return ((int64_t)max_blocks + p.splits - 1) / p.splits;
  const int64_t chunk = ((int64_t)B * p.units * max_blocks + p.range_ctas - 1) / p.range_ctas;
  return std::max<int64_t>(kMaxPiece, std::min<int64_t>(max_blocks, chunk));
}

size_t unit_workspace_bytes(const UnitPlan& p, int B, int D) {
  if (p.parts == 0) return 0;
  return (size_t)2 * p.parts * p.rows * (D + 2) * sizeof(float) + ((size_t)B + 2) * sizeof(int64_t);
}

cudaError_t launch_combine_units(const UnitDecodeArgs& a, cudaStream_t st) {
  const long long pairs = (long long)a.B * a.Hq;
  const bool one = pairs <= kCombineAlone;
  const long long grid = one ? pairs : (pairs + kCombineWarps - 1) / kCombineWarps;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  auto kern = a.D == 128 ? (one ? combine_units_kernel<128, 1> : combine_units_kernel<128, kCombineWarps>)
                         : (one ? combine_units_kernel<64, 1> : combine_units_kernel<64, kCombineWarps>);
  return launch_behind(kern, (unsigned)grid, 32 * kCombineWarps, 0, st, a);
}

}  // namespace lazy
