// int4.cuh -- the 4-bit pool format (LAZY_INT4, laid out in lazy_attn.h) and the step of
// the int4 decodes: one tile of 16-token blocks against the query heads of a KV head.
//
// A group of 64 dims of one token holds whole numbers c in 0..15 with a scale s and a
// zero z: the values are s c + z. So for a query q and the groups j of a key,
//   <q, k>  = sum_j  s_j <q_j, c_j> + z_j sum(q_j),
//   sum_t w_t v_t = sum_t (w_t s_t) c_t + sum_t w_t z_t   (per group),
// and the matrix products take the codes themselves: scales and zeros touch scores and
// weights (one per key and group), never elements.
//
// Codes enter mma.sync m16n8k16 as f16 without a conversion: a nibble in the low bits of
// an f16 is the subnormal c 2^-24, a byte of two nibbles (c + 16 c') 2^-24, both exact, and
// the products are summed in fp32. The operands are low nibbles c and whole bytes
// c + 16 c': (w & 0x000f000f), (w & 0x00ff00ff) and the same of w's odd bytes, four
// operations for eight codes (nibbles alone need five: a mask each and a shift). For the
// queries c q + c' q' = c (q - q'/16) + (c + 16 c') q'/16; of the outputs the second is
// (bytes - nibbles) / 16, in fp32. 2^24 is taken off the sums.
//
// Keys (or V's dims) are the A operand's 16 rows and the query heads its 8 columns: a
// product takes 256 codes, twice what heads as rows would. S^T = C q^T comes out with keys
// as rows; the weights become the B operand of O^T = C_v^T P^T by an 8 x 8 transpose
// (movmatrix).
//
// A tile of 32 keys and 8 rows is about 590 instructions of a warp: 128 unpack codes, 32 are
// products and 24 transposes, the rest scales, zeros and softmax in fp32. Masks and shifts issue
// every second cycle and keep the integer pipe 44 to 56% busy, more than any other. e4m3 codes (a
// byte 0..15 is c 2^-9, three such operations for eight codes) looked better: mma.sync takes them here as conversions and two f16 products (113 us against 104 on
// 64 x 4160 tokens, when the rest of the step was slower than it is now).
//
// tcgen05 needs the codes as f16 in shared memory and did not pay: with the values s c + z
// unpacked once per 64-key tile for up to 64 rows of an item (f16 over a power of two per
// token), items of more than 16 rows took 129 us against 135 on 32 x 16384 Zipf-drawn tokens
// with 8 heads per KV head and 68 against 62 on 64 x 4160 with 4; two CTAs an SM spent 2700
// cycles a tile, half of it in the softmax of one warp's keys and half unpacking.
#pragma once

#include "decode_block.cuh"

namespace lazy {

template <int D>
struct Int4Geom {
  static constexpr int NG = D / 64;             // groups of a row
  static constexpr int ROW = D / 2;             // code bytes of a row
  static constexpr int META = kBlock * ROW;     // offset of the (scale, zero) words
  static constexpr int REC = META + kBlock * NG * 4;  // one (block, KV head)
};

// V row that holds token t of a block, and back (the format's order).
__host__ __device__ __forceinline__ int int4_v_row(int t) { return (t & 8) + 4 * (t & 1) + ((t & 7) >> 1); }
__host__ __device__ __forceinline__ int int4_v_token(int r) { return (r & 8) + 2 * (r & 3) + ((r >> 2) & 1); }

__device__ __forceinline__ float meta_scale(uint32_t m) { return __uint_as_float(m << 16); }
__device__ __forceinline__ float meta_zero(uint32_t m) { return __uint_as_float(m & 0xffff0000u); }

// A record in shared memory.
struct SharedRecord {
  const uint8_t* p;
  __device__ __forceinline__ uint4 v4(int off) const { return *reinterpret_cast<const uint4*>(p + off); }
  __device__ __forceinline__ uint2 v2(int off) const { return *reinterpret_cast<const uint2*>(p + off); }
  __device__ __forceinline__ uint32_t v1(int off) const { return *reinterpret_cast<const uint32_t*>(p + off); }
};

// A warp's copies of two blocks' records into a ring stage ([block][K, V]), 16 bytes a lane:
// the rows of codes, then the four records' scales and zeros at once. (A bulk copy per
// record took about 20 instructions each, one lane at a time, against 25 for all of these:
// a step of 32 keys is bound by the instructions it issues.)
template <int D>
struct Int4Loader {
  using G = Int4Geom<D>;
  static constexpr int STAGE = 4 * G::REC;
  static constexpr int MLANES = kBlock * G::NG * 4 / 16;  // lanes for a record's scales and zeros
  const uint8_t *k, *v, *meta;  // the pools at the KV head, plus the lane's offset
  uint32_t blk_bytes, meta_dst;

  __device__ __forceinline__ Int4Loader(const void* k_pool, const void* v_pool, int hkv, int kvh, int lane) {
    blk_bytes = (uint32_t)hkv * G::REC;
    const size_t head = (size_t)kvh * G::REC;
    k = static_cast<const uint8_t*>(k_pool) + head + 16 * lane;
    v = static_cast<const uint8_t*>(v_pool) + head + 16 * lane;
    const int rec = (lane / MLANES) & 3, off = G::META + 16 * (lane % MLANES);
    meta = static_cast<const uint8_t*>((rec & 1) ? v_pool : k_pool) + head + off;
    meta_dst = rec * G::REC + off;
  }

  // Blocks ph0 and ph1 (both inside the pool) to the stage at shared address `dst`.
  __device__ __forceinline__ void operator()(uint32_t dst, int ph0, int ph1, int lane) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const size_t off = (size_t)(uint32_t)(b ? ph1 : ph0) * blk_bytes;
#pragma unroll
      for (int c = 0; c < G::META; c += 512) {
        cp_async16(dst + 16 * lane + 2 * b * G::REC + c, k + off + c);
        cp_async16(dst + 16 * lane + (2 * b + 1) * G::REC + c, v + off + c);
      }
    }
    if (4 * MLANES == 32 || lane < 4 * MLANES)
      cp_async16(dst + meta_dst, meta + (size_t)(uint32_t)(lane < 2 * MLANES ? ph0 : ph1) * blk_bytes);
  }
};

// Query rows of a warp: NT tiles of 8, or (HL = 1, NT = 1) one tile of 4 in the products'
// even columns, which halves the softmax's work per lane. A lane (g, t) = (lane / 4,
// lane % 4) sees the rows HL t .. HL t + HL - 1 of a tile.
template <int NT, int HL>
struct Int4Rows {
  static_assert(HL == 2 || (HL == 1 && NT == 1), "one row a lane: one tile of 4 rows");
  static constexpr int TILE = 4 * HL;
  static constexpr int ALL = NT * TILE;
};

// Query fragments for the k-order of the codes: lane (g, t) holds column g's dims of words
// D/32 t .. D/32 t + D/32 - 1 of a K row. k-step 2i + h: word i, its bytes h and h + 2; b0
// is q - q'/16 and b1 q'/16 for the dims (q, q') of each. A score, in log2 units, is f times
// the products' sums with the keys' scales and zeros: f is 2^24 and the row's power of two,
// `sum` the row's sums per group over f. Both are for the rows that the lane sees.
template <int D, int NT, int HL>
struct Int4Query {
  uint32_t b[NT][D / 16][2];
  float f[NT][HL];
  float sum[NT][HL][Int4Geom<D>::NG];
};

// The rows of the queries (bf16) that a lane reads, row 8 nt + g (or g / 2), with the factor
// that scales them (softmax scale, log2 e, and over the row's power of two `pow2`, so that
// the largest value is in 1..2; 0 for a row that is not there, whose pointer is another's).
template <int NT>
struct Int4QueryRows {
  const __nv_bfloat16* q[NT];
  float mul[NT], pow2[NT];
};

// First dim of a lane's word i.
template <int D>
__device__ __forceinline__ int int4_word_dim(int t, int i) {
  constexpr int NG = Int4Geom<D>::NG, W = D / 32;
  return 64 * (i % NG) + 8 * ((W * t + i) / NG);
}

// A lane's own dims of its rows, loaded ahead of their use.
template <int D, int NT>
struct Int4RawRows {
  uint4 x[NT][D / 32];
  __device__ __forceinline__ explicit Int4RawRows(const Int4QueryRows<NT>& r, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        x[nt][i] = *reinterpret_cast<const uint4*>(r.q[nt] + int4_word_dim<D>(lane & 3, i));
  }
};

// Fills mul and pow2 from the rows' values (all lanes).
template <int D, int NT>
__device__ __forceinline__ void int4_scale_rows(Int4QueryRows<NT>& r, const Int4RawRows<D, NT>& raw, const bool (&live)[NT],
                                                float scale) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t mx = 0u;  // |bf16| compares as its bits
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 x = raw.x[nt][i];
      mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu)),
                    x.w & 0x7fff7fffu);
    }
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float m = fmaxf(bf16_lo(mx), bf16_hi(mx)) * scale;
    const uint32_t ex = min(max(__float_as_uint(m) >> 23, 27u), 227u);  // 2^(+-100)
    r.pow2[nt] = __uint_as_float(ex << 23);
    r.mul[nt] = live[nt] ? scale * __uint_as_float((254u - ex) << 23) : 0.f;
  }
}

// Rotates the rows by their angles: cs(nt) points at the (cos, sin) of the lane's row (shared
// memory, 16-byte aligned). The rounding to f16 is off by 2^-11 of an operand.
template <int D, int NT, int HL, typename CsFn>
__device__ __forceinline__ void int4_build_query(Int4Query<D, NT, HL>& q, const Int4QueryRows<NT>& rows, int lane, CsFn cs) {
  constexpr int NG = Int4Geom<D>::NG, HALF = D / 2, W = D / 32;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2* ang = cs(nt);
    const float mul = rows.mul[nt];
    float s[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) s[j] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      asm volatile("" ::: "memory");  // one word's loads at a time: registers
      const int base = int4_word_dim<D>(t, i);
      const float sgn = base < HALF ? -1.f : 1.f;
      const uint4 x4 = *reinterpret_cast<const uint4*>(rows.q[nt] + base);
      const uint4 y4 = *reinterpret_cast<const uint4*>(rows.q[nt] + (base ^ HALF));
      const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
      float v[8];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float4 c = *reinterpret_cast<const float4*>(ang + (base & (HALF - 1)) + 2 * h);
        v[2 * h] = fmaf(bf16_lo(x[h]), c.x, bf16_lo(y[h]) * (sgn * c.y)) * mul;
        v[2 * h + 1] = fmaf(bf16_hi(x[h]), c.z, bf16_hi(y[h]) * (sgn * c.w)) * mul;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t b1 = pack_f16x2(v[2 * h + 1] * 0.0625f, v[2 * h + 5] * 0.0625f);
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&b1));
        const uint32_t b0 = pack_f16x2(v[2 * h] - r.x, v[2 * h + 4] - r.y);
        s[i % NG] += sum_op2<true>(b0) + 17.f * (r.x + r.y);  // the rounded values, as the products see them
        q.b[nt][2 * i + h][0] = HL == 1 && (g & 1) ? 0u : b0;
        q.b[nt][2 * i + h][1] = HL == 1 && (g & 1) ? 0u : b1;
      }
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      s[j] += __shfl_xor_sync(0xffffffffu, s[j], 1);
      s[j] += __shfl_xor_sync(0xffffffffu, s[j], 2);
      s[j] *= 1.f / 16777216.f;
    }
#pragma unroll
    for (int c = 0; c < HL; ++c) {  // column 2t + c's row sits in the lanes 4 (2t + c) ..
      const int src = 8 * t + 4 * c;
      q.f[nt][c] = __shfl_sync(0xffffffffu, rows.pow2[nt], src) * 16777216.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) q.sum[nt][c][j] = __shfl_sync(0xffffffffu, s[j], src);
    }
  }
}

// Running state: per row the reference maximum as -m (log2 units; 0 before the first key)
// and `top`, the value of score / f that refreshes it, the weight sum l and the
// zeros' sums z (partial over the lanes of equal t until int4_finish), and O^T / 2^24
// without the zeros: o[4 j + pp][nt] is the products' columns 2t, 2t + 1 for the lane's dim
// 2 pp of group j (int4_dims) in [0], [1] and for that plus 16 times the next in [2], [3]. With HL = 2
// the columns are the rows 2t, 2t + 1; with HL = 1 they are row t under group 0's and
// group 1's scales, and column 2t + j is the one that counts for group j. Weights times V
// scales go to f16 over `inv`'s power of two per group, which follows the scales as they
// grow: the largest scale is 2^4 to 2^5 then, at most 2^7 before the reference moves, and weights
// at most 2^8. What f16 has below is for the long tails: a product keeps its 11 bits from 2^-18
// of weight 1 times the largest scale, and is off by 2^-29 of that below (with the largest scale
// at 1 a tail of 131072 keys of weight 2^-25.5 was gone).
template <int D, int NT, int HL>
struct Int4State {
  float o[D / 16][NT][4];
  float neg_m[NT][HL], top[NT][HL], l[NT][HL], z[NT][HL][Int4Geom<D>::NG];
  float inv[Int4Geom<D>::NG], lim[Int4Geom<D>::NG];  // the same in all lanes; a scale above lim moves the reference
};

template <int D, int NT, int HL>
__device__ __forceinline__ void int4_init(Int4State<D, NT, HL>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i][nt][0] = st.o[i][nt][1] = st.o[i][nt][2] = st.o[i][nt][3] = 0.f;
#pragma unroll
    for (int c = 0; c < HL; ++c) {
      st.neg_m[nt][c] = 0.f;
      st.top[nt][c] = -INFINITY;
      st.l[nt][c] = 0.f;
#pragma unroll
      for (int j = 0; j < Int4Geom<D>::NG; ++j) st.z[nt][c][j] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < Int4Geom<D>::NG; ++j) {
    st.inv[j] = 1.f;
    st.lim[j] = 0.f;
  }
}

// O^T's running sums hold codes, not values: they grow with the keys and cancel against the
// zeros' part, and the products truncate them (2^-24 of the sum each time, always towards
// zero). Over 5000 keys of a 65000-key context that was 2.6e-3 of the output instead of the
// output rounding's 1.7e-3, over 8192 blocks of one warp of the shared-run decode 41% of it, so
// long runs move them to shared memory every kInt4Flush stages (64 blocks), where they are summed
// by rounding additions: `kept` is the warp's area, value n of lane l at 32 n + l (with HL = 1
// only the columns that count). It costs the shared-run decode 2 to 3%: 56.4 us against 54.2,
// 125.2 against 122.4.
constexpr int kInt4Flush = 32;
template <int D, int NT, int HL>
constexpr int int4_kept_floats() { return 32 * (D / 16) * NT * 2 * HL; }

// f(n, o): value n of the kept ones and its running sum.
template <int D, int NT, int HL, typename Fn>
__device__ __forceinline__ void int4_each_kept(Int4State<D, NT, HL>& st, Fn f) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < HL; ++c) f(((i * NT + nt) * 2 + r) * HL + c, i / 4, nt, c, st.o[i][nt][2 * r + (HL == 1 ? i / 4 : c)]);
}

// Moves the running sums to the kept ones (which are there already: `again`).
template <int D, int NT, int HL>
__device__ __forceinline__ void int4_flush(Int4State<D, NT, HL>& st, float* kept, bool again, int lane) {
  int4_each_kept<D, NT, HL>(st, [&](int n, int, int, int, float& o) {
    float* k = kept + 32 * n + lane;
    *k = again ? *k + o : o;
    o = 0.f;
  });
}

// And back, at the end.
template <int D, int NT, int HL>
__device__ __forceinline__ void int4_unflush(Int4State<D, NT, HL>& st, const float* kept, int lane) {
  int4_each_kept<D, NT, HL>(st, [&](int n, int, int, int, float& o) { o += kept[32 * n + lane]; });
}

constexpr float kInt4RescaleLog2 = 8.f;  // a maximum is refreshed when it grows by more
constexpr float kInt4ScaleTop = 128.f;   // the V scales' reference moves when one times inv is more

// Bytes h and h + 2 of a word as f16 pairs: low nibbles, and whole bytes.
__device__ __forceinline__ void int4_pair(uint32_t w, int h, uint32_t& nibbles, uint32_t& bytes) {
  bytes = h ? __byte_perm(w, 0u, 0x4341) : w & 0x00ff00ffu;
  nibbles = (h ? bytes : w) & 0x000f000fu;
}

// One tile: two blocks of one document. With `partial` (the same in all lanes) only the
// first nv[b] slots of block b are keys (0: the block is not there), and the other slots'
// scales and zeros may hold anything. `kept`: sums moved out of the state, to be rescaled
// with it (null: none).
template <int D, int NT, int HL>
__device__ __forceinline__ void int4_attend(const SharedRecord (&kr)[2], const SharedRecord (&vr)[2], bool partial, const int (&nv)[2],
                                            const Int4Query<D, NT, HL>& q, Int4State<D, NT, HL>& st, int lane,
                                            float* kept = nullptr) {
  using G = Int4Geom<D>;
  constexpr int NG = G::NG, W = D / 32;
  const int g = lane >> 2, t = lane & 3;

  // Scores over f of keys g and g + 8 of each block: p[block][key][tile][row]. The two blocks' and
  // the groups' products take turns: four sums side by side hide a product's latency.
  float p[2][2][NT][HL];
  uint32_t kw[2][2][W], km[2][2][NG];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r;
      if constexpr (W == 4) {
        const uint4 x = kr[b].v4(row * G::ROW + 16 * t);
        kw[b][r][0] = x.x, kw[b][r][1] = x.y, kw[b][r][2] = x.z, kw[b][r][3] = x.w;
        const uint2 u = kr[b].v2(G::META + row * 8);
        km[b][r][0] = u.x, km[b][r][NG - 1] = u.y;
      } else {
        const uint2 x = kr[b].v2(row * G::ROW + 8 * t);
        kw[b][r][0] = x.x, kw[b][r][1] = x.y;
        km[b][r][0] = kr[b].v1(G::META + row * 4);
      }
    }
  float acc[2][NT][NG][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t a[4];
        int4_pair(kw[b][0][i], h, a[0], a[2]);
        int4_pair(kw[b][1][i], h, a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (i < NG && h == 0) mma_16816_f16_first(acc[b][nt][i % NG], a, q.b[nt][2 * i + h][0], q.b[nt][2 * i + h][1]);
          else mma_16816_f16(acc[b][nt][i % NG], a, q.b[nt][2 * i + h][0], q.b[nt][2 * i + h][1]);
        }
      }
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < HL; ++c) {
          float s = meta_zero(km[b][r][0]) * q.sum[nt][c][0];
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            if (j > 0) s = fmaf(meta_zero(km[b][r][j]), q.sum[nt][c][j], s);
            s = fmaf(meta_scale(km[b][r][j]), acc[b][nt][j][2 * r + c], s);
          }
          p[b][r][nt][c] = s;
        }
  if (partial) {
    asm volatile("" ::: "memory");  // a branch, not selects on every tile
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < HL; ++c)
            if (g + 8 * r >= nv[b]) p[b][r][nt][c] = -INFINITY;
  }

  // V's scales and zeros of the same keys.
  uint32_t vm[2][2][NG];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (NG == 2) {
        const uint2 u = vr[b].v2(G::META + (g + 8 * r) * 8);
        vm[b][r][0] = u.x, vm[b][r][NG - 1] = u.y;
      } else {
        vm[b][r][0] = vr[b].v1(G::META + (g + 8 * r) * 4);
      }
    }
  if (partial) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < NG; ++j)
          if (g + 8 * r >= nv[b]) vm[b][r][j] = 0u;
  }
  float vs[2][2][NG];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < NG; ++j) vs[b][r][j] = meta_scale(vm[b][r][j]);

  // Running maximum and V-scale reference: refreshed together, when some row's maximum or
  // some scale outgrew its reference (a vote; the cross-lane maxima only then).
  float mx[NT][HL], sm[NG];
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < HL; ++c) {
      mx[nt][c] = fmaxf(fmaxf(p[0][0][nt][c], p[0][1][nt][c]), fmaxf(p[1][0][nt][c], p[1][1][nt][c]));
      grow |= mx[nt][c] > st.top[nt][c];
    }
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    sm[j] = fmaxf(fmaxf(vs[0][0][j], vs[0][1][j]), fmaxf(vs[1][0][j], vs[1][1][j]));
    grow |= sm[j] > st.lim[j];
  }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sm[j] = fmaxf(sm[j], __shfl_xor_sync(0xffffffffu, sm[j], o));
      if (sm[j] > st.lim[j]) {
        // 2^(4 - e) for sm in [2^e, 2^(e+1)): between 2^4 and 2^5 now. Kept a normal number.
        const uint32_t ex = min(max(__float_as_uint(sm[j]) >> 23, 8u), 252u);
        const float inv = __uint_as_float((258u - ex) << 23);
        const float r = inv / st.inv[j];
        st.inv[j] = inv;
        st.lim[j] = kInt4ScaleTop / inv;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[4 * j + i][nt][e] *= r;
        if (kept)
          int4_each_kept<D, NT, HL>(st, [&](int n, int jj, int, int, float&) {
            if (jj == j) kept[32 * n + lane] *= r;
          });
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < HL; ++c) {
        float x = mx[nt][c];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (x > st.top[nt][c]) {
          x *= q.f[nt][c];
          const float alpha = st.top[nt][c] == -INFINITY ? 0.f : fast_ex2(-st.neg_m[nt][c] - x);
          st.neg_m[nt][c] = -x;
          st.top[nt][c] = __fdividef(x + kInt4RescaleLog2, q.f[nt][c]);
          st.l[nt][c] *= alpha;
#pragma unroll
          for (int j = 0; j < NG; ++j) st.z[nt][c][j] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (HL == 1 || (e & 1) == c) st.o[i][nt][e] *= alpha;
          if (kept)
            int4_each_kept<D, NT, HL>(st, [&](int n, int, int t2, int c2, float&) {
              if (t2 == nt && c2 == c) kept[32 * n + lane] *= alpha;
            });
        }
      }
  }

  // Weights; their sum and the zeros' part in fp32.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < HL; ++c) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float x = fast_ex2(fmaf(p[b][r][nt][c], q.f[nt][c], st.neg_m[nt][c]));
          p[b][r][nt][c] = x;
          st.l[nt][c] += x;
#pragma unroll
          for (int j = 0; j < NG; ++j) st.z[nt][c][j] = fmaf(x, meta_zero(vm[b][r][j]), st.z[nt][c][j]);
        }
    }

  // O^T += C_v^T P^T: rows are dims, the k-order tokens 2t, 2t + 1 (b0), 2t + 8, 2t + 9 (b1).
  // Weights times scales (exact over their reference) are rounded to f16 once: off by 2^-11 of
  // a term, next to the codes' 4 bits.
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t pb[NT][NG][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float s[NG];
#pragma unroll
      for (int j = 0; j < NG; ++j) s[j] = vs[b][r][j] * st.inv[j];
      if constexpr (HL == 1) {  // both groups' columns at once
        const float x = p[b][r][0][0];
        pb[0][0][r] = transpose_8x8(pack_f16x2(x * s[0], x * s[NG - 1]));
        pb[0][NG - 1][r] = pb[0][0][r];
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < NG; ++j) pb[nt][j][r] = transpose_8x8(pack_f16x2(p[b][r][nt][0] * s[j], p[b][r][nt][HL - 1] * s[j]));
      }
    }
    // V's words, token rows g and g + 8 in lane g, become pairs of tokens (2t, 2t + 1) of the
    // same four dims: column g is a half of word W (g / 2) + i.
    uint32_t x[2][W];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (W == 4) {
        const uint4 y = vr[b].v4(int4_v_row(g + 8 * r) * G::ROW + 16 * t);
        x[r][0] = y.x, x[r][1] = y.y, x[r][2] = y.z, x[r][3] = y.w;
      } else {
        const uint2 y = vr[b].v2(int4_v_row(g + 8 * r) * G::ROW + 8 * t);
        x[r][0] = y.x, x[r][1] = y.y;
      }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t u = transpose_8x8(x[0][i]), v = transpose_8x8(x[1][i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[4];
        int4_pair(u, h, a[0], a[1]);
        int4_pair(v, h, a[2], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_16816_f16(st.o[4 * (i % NG) + 2 * (i / NG) + h][nt], a, pb[nt][i % NG][0], pb[nt][i % NG][1]);
      }
    }
  }
}

// Sums the lanes' parts of l and z: after it every lane holds the rows' full sums.
template <int D, int NT, int HL>
__device__ __forceinline__ void int4_finish(Int4State<D, NT, HL>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < HL; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.l[nt][c] += __shfl_xor_sync(0xffffffffu, st.l[nt][c], o);
#pragma unroll
        for (int j = 0; j < Int4Geom<D>::NG; ++j) st.z[nt][c][j] += __shfl_xor_sync(0xffffffffu, st.z[nt][c][j], o);
      }
}

// Weighted values, unnormalised, of the lane's dims of group j and its row c of tile nt:
// int4_dims(j, g) + 0..3 and int4_dims(j, g) + kInt4Dims2 + 0..3.
constexpr int kInt4Dims2 = 8;
__device__ __forceinline__ int int4_dims(int j, int g) { return 64 * j + 16 * (g >> 1) + 4 * (g & 1); }
template <int D, int NT, int HL>
__device__ __forceinline__ void int4_out8(const Int4State<D, NT, HL>& st, int j, int nt, int c, float (&v)[8]) {
  const float r = 1.f / st.inv[j];
  const int col = HL == 1 ? j : c;
#pragma unroll
  for (int pp = 0; pp < 4; ++pp) {
    v[2 * pp] = fmaf(st.o[4 * j + pp][nt][col] * 16777216.f, r, st.z[nt][c][j]);
    v[2 * pp + 1] = fmaf((st.o[4 * j + pp][nt][col + 2] - st.o[4 * j + pp][nt][col]) * 1048576.f, r, st.z[nt][c][j]);
  }
}

}  // namespace lazy
