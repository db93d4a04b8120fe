// fp8_block.cuh -- the pool format of e4m3 codes with a scale per block of tokens and head
// (LAZY_FP8_E4M3_BLOCK, laid out in lazy_attn.h), and the step of the decodes over it: one
// 16-token block against the query heads of a KV head.
//
// A block's values are codes times one power of two, so for a query q
//   <q, k> = 2^ek <q, c_k>,   sum_t w_t v_t = sum_t (w_t 2^ev) c_t:
// the products take the codes, and the scale is one factor of a block's scores and weights.
//
// Keys (or V's dims) are the A operand's 16 rows of mma.sync m16n8k16 and the query heads its 8
// columns: a product takes 256 codes, twice what heads as rows would. S^T = C q^T comes out with
// keys as rows; the weights become the B operand of O^T = C_v^T P^T by an 8 x 8 transpose.
//
// The records lie in the order in which lanes need them: chunk 32 j + lane of a record is 16
// bytes of lane's own fragments, whose neighbouring codes (dims of K, tokens of V) are the
// pairs of f16 that an operand register holds. So a warp reads 512 bytes in a row without a bank
// conflict, and a conversion of two codes (exact: every e4m3 value is an f16 value) gives a
// register of an operand: no transposes, masks or shuffles of codes.
#pragma once

#include "decode_block.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace lazy {

template <int D>
struct Fp8Geom {
  static constexpr int CODES = kBlock * D;  // bytes
  static constexpr int SCALE = CODES;       // offset of the scale
  static constexpr int REC = CODES + 32;    // one (block, KV head)
  static constexpr int CHUNKS = D / 32;     // 16-byte chunks of a lane
  static constexpr int NG = D / 64;
};

// Chunk j of lane (g, t) = (lane / 4, lane % 4). K: token g + 8 (j % 2), dims
// 16 (t + 4 (j / 2)) .. + 15. V: dims 8 (g + 8 (j % NG)) .. + 7 of the tokens 2 (t + 4 (j / NG))
// and that + 1, side by side.

// A team's ring of stages. A stage is one block's K and V records, which one lane copies with two bulk copies; `full`
// counts their bytes, `empty` the team's warps that are done with them. `info` goes with a stage: valid
// slots, and what else its reader wants to know of it.
constexpr int kFp8Slots = 16;  // stages of a CTA's rings at most
struct Fp8Bars {
  uint64_t full[kFp8Slots], empty[kFp8Slots];
  int info[kFp8Slots];
};

// A wait gave up: copies of the loads first .. last - 1 (counted through the ring of R) still land, or not within
// 10 ms each, before the CTA ends. (By value: a ring whose address is taken lies in memory.)
static __device__ __noinline__ void fp8_drain(uint64_t* full, uint32_t first_load, uint32_t last_load, uint32_t R, unsigned int* status) {
  for (uint32_t n = first_load; n < last_load; ++n) warp_wait(&full[n % R], n / R & 1, status, 10000000ull);
}

template <int D>
struct Fp8Ring {
  using G = Fp8Geom<D>;
  static constexpr int STAGE = 2 * G::REC;
  const uint8_t *k, *v;  // the pools at the KV head
  uint32_t blk_bytes;
  uint8_t* base;         // the team's first stage
  Fp8Bars* bars;         // of the CTA
  int first;             // index of the team's first stage among them

  // Block ph (inside the pool) to stage `slot`, by one lane.
  __device__ __forceinline__ void fill(int slot, int ph, int info) const {
    uint64_t* bar = &bars->full[first + slot];
    bars->info[first + slot] = info;  // seen by those who see the barrier's phase
    mbar_arrive_expect_tx(bar, STAGE);
    const uint32_t dst = smem_u32(base) + slot * STAGE, b = smem_u32(bar);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(k + (uint64_t)(uint32_t)ph * blk_bytes), "n"(G::REC), "r"(b)
                 : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst + G::REC),
                 "l"(v + (uint64_t)(uint32_t)ph * blk_bytes), "n"(G::REC), "r"(b)
                 : "memory");
  }
  __device__ __forceinline__ bool wait_full(int slot, uint32_t parity, unsigned int* status) const {
    return warp_wait(&bars->full[first + slot], parity, status);
  }
  __device__ __forceinline__ bool wait_empty(int slot, uint32_t parity, unsigned int* status) const {
    return warp_wait(&bars->empty[first + slot], parity, status);
  }
  __device__ __forceinline__ void drain(uint32_t first_load, uint32_t last_load, uint32_t R, unsigned int* status) const {
    fp8_drain(&bars->full[first], first_load, last_load, R, status);
  }
  __device__ __forceinline__ void release(int slot) const { mbar_arrive(&bars->empty[first + slot]); }
};

// Query rows of a warp: NT tiles of 8, or (HL = 1, NT = 1) one tile of 4 in the products' even
// columns, which halves the softmax's work per lane. A lane (g, t) sees the rows HL t .. HL t +
// HL - 1 of a tile.
template <int NT, int HL>
struct Fp8Rows {
  static_assert(HL == 2 || (HL == 1 && NT == 1), "one row a lane: one tile of 4 rows");
  static constexpr int TILE = 4 * HL;
  static constexpr int ALL = NT * TILE;
};

// Query fragments: product 4 jh + i of a tile takes, in lane (g, t), column g's dims
// 16 (t + 4 jh) + 4 i + 0, 1 (b0) and + 2, 3 (b1). A block's scores, in log2 units, are the products'
// sums times f and K's scale; f is the row's power of two, for the rows that the lane sees.
// Four tiles' fragments (64 registers, d = 128) lie in shared memory, a lane its own.
template <int D, int NT, int HL>
struct Fp8Query {
  static constexpr bool kShared = NT == 4;
  static constexpr int BYTES = kShared ? 32 * NT * (D / 16) * 8 : 0;  // of a warp
  uint32_t b[kShared ? 1 : NT][kShared ? 1 : D / 16][2];
  uint32_t* s;  // the lane's first word of the warp's area
  float f[NT][HL];

  // Product k's fragments of all tiles.
  __device__ __forceinline__ void get(int k, uint32_t (&x)[NT][2]) const {
    if constexpr (kShared) {
#pragma unroll
      for (int nt = 0; nt + 1 < NT; nt += 2) {  // 16 bytes: two tiles' fragments
        const uint4 v = *reinterpret_cast<const uint4*>(s + 128 * (k * (NT / 2) + nt / 2));
        x[nt][0] = v.x, x[nt][1] = v.y, x[nt + 1][0] = v.z, x[nt + 1][1] = v.w;
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][0] = b[nt][k][0], x[nt][1] = b[nt][k][1];
    }
  }
  __device__ __forceinline__ void set(int nt, int k, int h, uint32_t v) {
    if constexpr (kShared) s[128 * (k * (NT / 2) + nt / 2) + 2 * (nt % 2) + h] = v;
    else b[nt][k][h] = v;
  }
};

// A lane reads the query rows (bf16) of the columns g of its tiles, row 8 nt + g (or g / 2); row(nt) points
// at one (where there is none, at another). A row is scaled by mul: softmax scale and log2 e, over the row's power of
// two, so that the largest value is in 1..2; 0 for a row that is not there. Here a lane's own dims of its rows,
// loaded ahead of their use.
template <int D, int NT>
struct Fp8RawRows {
  uint4 x[NT][D / 32];
  template <typename RowFn>
  __device__ __forceinline__ Fp8RawRows(RowFn row, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        x[nt][i] = *reinterpret_cast<const uint4*>(row(nt) + 64 * (i / 2) + 16 * (lane & 3) + 8 * (i % 2));
  }
};

// Fills mul and q.f from the rows' values (all lanes).
template <int D, int NT, int HL>
__device__ __forceinline__ void fp8_scale_rows(Fp8Query<D, NT, HL>& q, float (&mul)[NT], const Fp8RawRows<D, NT>& raw,
                                               const bool (&live)[NT], float scale, int lane) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t mx = 0u;  // |bf16| compares as its bits
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 x = raw.x[nt][i];
      mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu)), x.w & 0x7fff7fffu);
    }
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float m = fmaxf(bf16_lo(mx), bf16_hi(mx)) * scale;
    const uint32_t ex = min(max(__float_as_uint(m) >> 23, 27u), 227u);  // 2^(+-100)
    mul[nt] = live[nt] ? scale * __uint_as_float((254u - ex) << 23) : 0.f;
#pragma unroll
    for (int c = 0; c < HL; ++c)  // a lane of column 2t + c
      q.f[nt][c] = __shfl_sync(0xffffffffu, __uint_as_float(ex << 23), 8 * (lane & 3) + 4 * c);
  }
}

// Rotates the rows by their angles: cs(nt) points at the (cos, sin) of the lane's row (shared
// memory, 16-byte aligned); put(nt, k, h, x) takes word h of tile nt's fragment for product k. The rounding to f16 is
// off by 2^-11 of an operand.
template <int D, int NT, int HL, typename RowFn, typename CsFn, typename PutFn>
__device__ __forceinline__ void fp8_build_query(const float (&mul)[NT], RowFn row, int lane, CsFn cs, PutFn put) {
  constexpr int HALF = D / 2;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2* ang = cs(nt);
    const __nv_bfloat16* src = row(nt);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      asm volatile("" ::: "memory");  // eight dims' loads at a time: registers
      const int base = 64 * (i / 2) + 16 * t + 8 * (i % 2);
      const float sgn = base < HALF ? -1.f : 1.f;
      const uint4 x4 = *reinterpret_cast<const uint4*>(src + base);
      const uint4 y4 = *reinterpret_cast<const uint4*>(src + (base ^ HALF));
      const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float4 c = *reinterpret_cast<const float4*>(ang + (base & (HALF - 1)) + 2 * h);
        const uint32_t b = pack_f16x2(fmaf(bf16_lo(x[h]), c.x, bf16_lo(y[h]) * (sgn * c.y)) * mul[nt],
                                      fmaf(bf16_hi(x[h]), c.z, bf16_hi(y[h]) * (sgn * c.w)) * mul[nt]);
        put(nt, 2 * i + h / 2, h % 2, HL == 1 && (g & 1) ? 0u : b);
      }
    }
  }
}

// Running state: per row nm, which puts a score s (log2 units) at a weight of 2^(s + nm) -- 2^kFp8Lift for the greatest
// score when nm was set, at most 2^kFp8Most until it is set anew; +inf before the first key -- and the
// weight sum l (partial over the lanes of equal t until fp8_finish), and O^T: o[i][nt] is product i's
// columns 2t, 2t + 1 for the dim 8 g + i in [0], [1] and for 64 + 8 g + i (d = 64: 8 g + 4 + i) in
// [2], [3]. Weights and V's scale over the power of two 1 / inv meet as f16: `inv` follows the scales as they
// grow, the largest is 1 then, at most kFp8ScaleTop before the reference moves. What f16 has below
// is for the long tails: a weight keeps its 11 bits from 2^-18 of the largest, and is off by 2^-29
// of that (times the largest V scale) below.
constexpr float kFp8Lift = 4.f, kFp8Most = 12.f, kFp8ScaleTop = 8.f;
template <int D, int NT, int HL>
struct Fp8State {
  float o[D / 16][NT][4];
  float nm[NT][HL], l[NT][HL];
  float inv, lim;  // the same in all lanes; a scale above lim moves the reference
};

template <int D, int NT, int HL>
__device__ __forceinline__ void fp8_init(Fp8State<D, NT, HL>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i][nt][0] = st.o[i][nt][1] = st.o[i][nt][2] = st.o[i][nt][3] = 0.f;
#pragma unroll
    for (int c = 0; c < HL; ++c) {
      st.nm[nt][c] = INFINITY;
      st.l[nt][c] = 0.f;
    }
  }
  st.inv = 1.f;
  st.lim = -1.f;
}

// The products truncate their running sums (by up to 2^-23 a block, always towards zero). In lazy_attn_decode a warp's sums
// leave the accumulators every kFp8Keep blocks (2^-14 at most by then) for local memory, where they are added with rounding,
// and their references with them; registers hold no second set. The kernel for parts that long is one of its own: with the way
// out in the others' code one sequence of 16384 tokens took 14.2 us for 13.6, and shared items 120 for 112 (32 x 16384 tokens), which
// keep theirs: of the lengths that the planner takes (384 blocks at most) 2^-14. No warp sums more than kFp8MaxRun = 16384 blocks:
// pieces, ranges and items are cut there. 16 sequences of 262144 tokens: 32 heads on 8 1242 us for 1230 without the way
// out, 64 on 4 662 for 623 (its registers spill); 48 with 32 on one 714 for 705.
constexpr int kFp8Keep = 512;
template <int D, int NT, int HL>
struct Fp8Kept {
  static constexpr int SUMS = D / 16 * NT * 2 * HL;  // (HL = 1: of the columns that count)
  volatile float o[SUMS], nm[NT * HL], inv;          // volatile: stays in memory
  bool any;

  // f(sum, place, row's tile, row).
  template <typename Fn>
  static __device__ __forceinline__ void each(Fp8State<D, NT, HL>& st, Fn f) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < HL; ++c) f(st.o[i][nt][2 * h + c], ((i * NT + nt) * 2 + h) * HL + c, nt, c);
  }
  // What the kept sums weigh by the state's references, per row.
  __device__ __forceinline__ void weights(const Fp8State<D, NT, HL>& st, float (&w)[NT][HL]) const {
    const float r = st.inv / inv;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < HL; ++c) w[nt][c] = fast_ex2(st.nm[nt][c] - nm[nt * HL + c]) * r;
  }
  __device__ __forceinline__ void keep(Fp8State<D, NT, HL>& st) {
    if (st.lim < 0.f) return;  // no block yet (the same in all lanes)
    if (any) {
      float w[NT][HL];
      weights(st, w);
      each(st, [&](float& x, int n, int nt, int c) { o[n] = fmaf(o[n], w[nt][c], x), x = 0.f; });
    } else {
      each(st, [&](float& x, int n, int, int) { o[n] = x, x = 0.f; });
    }
    any = true;
    inv = st.inv;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < HL; ++c) nm[nt * HL + c] = st.nm[nt][c];
  }
  // And back, at the end.
  __device__ __forceinline__ void give_back(Fp8State<D, NT, HL>& st) const {
    if (!any) return;
    float w[NT][HL];
    weights(st, w);
    each(st, [&](float& x, int n, int nt, int c) { x = fmaf(o[n], w[nt][c], x); });
  }
};

// A block in its stage: the first nv slots are keys (1 .. 16, the same in all lanes); what the others hold does not
// matter.
template <int D, int NT, int HL>
__device__ __forceinline__ void fp8_attend(const uint8_t* stage, int nv, const Fp8Query<D, NT, HL>& q, Fp8State<D, NT, HL>& st,
                                           int lane) {
  using G = Fp8Geom<D>;
  const int g = lane >> 2, t = lane & 3;
  const bool partial = nv < kBlock;
  const float ks = *reinterpret_cast<const float*>(stage + G::SCALE), vs = *reinterpret_cast<const float*>(stage + G::REC + G::SCALE);

  // Scores of keys g and g + 8 over f: p[tile][2 key + row]. The tiles' products take turns, so that
  // none waits for the one before it (one tile: even and odd ones).
  constexpr int CH = NT == 1 ? 2 : 1;
  float p[NT][4];
  {
    float odd[4];
#pragma unroll
    for (int jh = 0; jh < G::NG; ++jh) {
      uint32_t x[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 v = reinterpret_cast<const uint4*>(stage)[lane + 64 * jh + 32 * r];
        x[r][0] = v.x, x[r][1] = v.y, x[r][2] = v.z, x[r][3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t k[NT][2], a[4];
        q.get(4 * jh + i, k);
        e4m3x4_to_f16x4(x[0][i], a[0], a[2]);
        e4m3x4_to_f16x4(x[1][i], a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float(&sum)[4] = CH == 2 && i % 2 ? odd : p[nt];
          if (jh == 0 && i < CH) mma_16816_f16_first(sum, a, k[nt][0], k[nt][1]);
          else mma_16816_f16(sum, a, k[nt][0], k[nt][1]);
        }
      }
    }
    if (CH == 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[0][e] += odd[e];
  }
  uint64_t f[NT];  // pairs: the lane's rows (HL = 1: its row, for both keys)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) f[nt] = f2_mul(f2(q.f[nt][0], q.f[nt][HL - 1]), f2(ks, ks));
  // a pair of sums: row 2t, 2t + 1 of key r (HL = 1: keys g and g + 8 of the row)
  auto pair = [&](int nt, int r) { return HL == 1 ? f2(p[nt][0], p[nt][2]) : f2(p[nt][2 * r], p[nt][2 * r + 1]); };
  auto set_pair = [&](int nt, int r, uint64_t v) {
    const float2 x = f2_split(v);
    p[nt][HL == 1 ? 0 : 2 * r] = x.x;
    p[nt][HL == 1 ? 2 : 2 * r + 1] = x.y;
  };
  auto mask = [&](float to) {  // the scores of slots that are no keys
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (g + 8 * (e / 2) >= nv)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) p[nt][e] = to;
  };
  const bool first = st.lim < 0.f;  // the same in all lanes (a scale of 0, of a pool that nothing wrote, counts too)
  if (first) {
    if (partial) mask(-INFINITY);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < HL; ++c) {
        float x = fmaxf(p[nt][c], p[nt][2 + c]) * fmaxf(q.f[nt][c] * ks, 0x1p-126f);  // (-inf times 0 would be NaN)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        st.nm[nt][c] = kFp8Lift - x;
      }
  }
  // Exponents s + nm.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < HL; ++r) set_pair(nt, r, f2_fma(pair(nt, r), f[nt], f2(st.nm[nt][0], st.nm[nt][HL - 1])));
  if (partial) {
    asm volatile("" ::: "memory");  // a branch, not selects on every block
    mask(-INFINITY);
  }

  // References are refreshed together, when some weight or scale would outgrow its own (a vote; the
  // cross-lane maxima only then).
  float high = p[0][0];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if constexpr (HL == 1) high = fmaxf(high, p[nt][2]);
    else high = fmaxf(fmax3(high, p[nt][0], p[nt][1]), fmaxf(p[nt][2], p[nt][3]));
  }
  if (__any_sync(0xffffffffu, high > kFp8Most || vs > st.lim)) {
    if (vs > st.lim) {
      // 2^-e for a scale 2^e. Kept a normal number.
      const uint32_t ex = min(max(__float_as_uint(vs) >> 23, 4u), 250u);
      const float inv = __uint_as_float((254u - ex) << 23), r = inv / st.inv;
      st.inv = inv;
      st.lim = kFp8ScaleTop / inv;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[i][nt][e] *= r;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < HL; ++c) {
        float x = fmaxf(p[nt][c], p[nt][2 + c]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (x > kFp8Most) {
          const float down = kFp8Lift - x, alpha = fast_ex2(down);
          st.nm[nt][c] += down;
          st.l[nt][c] *= alpha;
          p[nt][c] += down, p[nt][2 + c] += down;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            st.o[i][nt][c] *= alpha;
            st.o[i][nt][2 + c] *= alpha;
          }
        }
      }
  }

  // Weights, their sum in fp32, and weights times V's scale over its reference, a power of two, rounded to f16 once
  // (off by 2^-11, next to the codes' 4 bits). The k-order of O^T += C_v^T P^T is tokens
  // 2t, 2t + 1 (b0), 2t + 8, 2t + 9 (b1).
  uint32_t pb[NT][2];
  const float v_scale = vs * st.inv;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 4; e += HL == 1 ? 2 : 1) p[nt][e] = fast_ex2(p[nt][e]);
    if constexpr (HL == 1) {
      st.l[nt][0] += p[nt][0] + p[nt][2];
    } else {
      const float2 sum = f2_split(f2_add(f2(st.l[nt][0], st.l[nt][HL - 1]), f2_add(pair(nt, 0), pair(nt, 1))));
      st.l[nt][0] = sum.x, st.l[nt][HL - 1] = sum.y;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 w = HL == 1 ? make_float2(p[nt][2 * r] * v_scale, 0.f) : f2_split(f2_mul(pair(nt, r), f2(v_scale, v_scale)));
      pb[nt][r] = transpose_8x8(pack_f16x2(w.x, w.y));
    }
  }

  // Products 2 w and 2 w + 1 take the words w of the lane's chunks (d = 64: w and w + 2).
  uint4 v4[2][G::NG];  // [tokens 2t, 2t + 1 or 2t + 8, 2t + 9][dims]
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int j = 0; j < G::NG; ++j) v4[r][j] = reinterpret_cast<const uint4*>(stage + G::REC)[lane + 32 * (G::NG * r + j)];
  if (partial) {  // codes of slots without a key may be NaN
    asm volatile("" ::: "memory");
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int tok = 2 * t + 8 * r;
      const uint32_t keep = (tok < nv ? 0x00ff00ffu : 0u) | (tok + 1 < nv ? 0xff00ff00u : 0u);
#pragma unroll
      for (int j = 0; j < G::NG; ++j) v4[r][j].x &= keep, v4[r][j].y &= keep, v4[r][j].z &= keep, v4[r][j].w &= keep;
    }
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    uint32_t a[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t lo[4] = {v4[r][0].x, v4[r][0].y, v4[r][0].z, v4[r][0].w};
      const uint32_t hi[4] = {v4[r][G::NG - 1].x, v4[r][G::NG - 1].y, v4[r][G::NG - 1].z, v4[r][G::NG - 1].w};
      e4m3x4_to_f16x4(lo[w], a[0][2 * r], a[1][2 * r]);
      e4m3x4_to_f16x4(hi[G::NG == 2 ? w : w + 2], a[0][2 * r + 1], a[1][2 * r + 1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16816_f16(st.o[2 * w + e][nt], a[e], pb[nt][0], pb[nt][1]);
  }
}

// Sums the lanes' parts of l: after it every lane holds the rows' full sums.
template <int D, int NT, int HL>
__device__ __forceinline__ void fp8_finish(Fp8State<D, NT, HL>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < HL; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) st.l[nt][c] += __shfl_xor_sync(0xffffffffu, st.l[nt][c], o);
}

// A warp's partial of its rows to shared memory: o[D], m, l per row.
template <int D, int NT, int HL>
__device__ __forceinline__ void fp8_store_partial(const Fp8State<D, NT, HL>& st, float* red, int stride, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float r = 1.f / st.inv;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < HL; ++c) {
      float* row = red + (8 * nt + HL * t + c) * stride;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
          *reinterpret_cast<float4*>(row + 8 * g + (D / 2 == 64 ? 64 : 4) * h + i) =
              make_float4(st.o[i][nt][2 * h + c] * r, st.o[i + 1][nt][2 * h + c] * r, st.o[i + 2][nt][2 * h + c] * r,
                          st.o[i + 3][nt][2 * h + c] * r);
      if (g == 0) {
        row[D] = -st.nm[nt][c];
        row[D + 1] = st.l[nt][c];
      }
    }
}

}  // namespace lazy
