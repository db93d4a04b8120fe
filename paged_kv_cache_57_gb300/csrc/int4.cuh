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
// an f16 is the subnormal c 2^-24, one 4 bits higher 16 c 2^-24, both exact, and the
// products are summed in fp32. (w & 0x000f000f) and (w & 0x00f000f0) are such pairs, so
// eight codes cost four masks and a shift. The factor 16 of every second element is
// taken off the other operand (q / 16, exact) or the output; 2^24 off the sums.
//
// Keys (or V's dims) are the A operand's 16 rows and the query heads its 8 columns: a
// product takes 256 codes, twice what heads as rows would, and groups of up to 8 heads
// pad nothing further. S^T = C q^T comes out with keys as rows; the weights become the
// B operand of O^T = C_v^T P^T by an 8 x 8 transpose (movmatrix).
#pragma once

#include "common.cuh"

namespace lazy {

template <int D>
struct Int4Geom {
  static constexpr int NG = D / 64;             // groups of a row
  static constexpr int ROW = D / 2;             // code bytes of a row
  static constexpr int META = kBlock * ROW;     // offset of the (scale, zero) words
  static constexpr int REC = META + kBlock * NG * 4;  // one (block, KV head)
};

// V row that holds token t of a block, and back. Lane t of a quad takes tokens 2t, 2t+1,
// 2t+8, 2t+9 (the B operand's rows) from rows t, t+4, t+8, t+12: consecutive lanes read
// consecutive rows.
__host__ __device__ __forceinline__ int int4_v_row(int t) { return (t & 8) + 4 * (t & 1) + ((t & 7) >> 1); }
__host__ __device__ __forceinline__ int int4_v_token(int r) { return (r & 8) + 2 * (r & 3) + ((r >> 2) & 1); }

__device__ __forceinline__ float meta_scale(uint32_t m) { return __uint_as_float(m << 16); }
__device__ __forceinline__ float meta_zero(uint32_t m) { return __uint_as_float(m & 0xffff0000u); }

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A record in shared memory.
struct SharedRecord {
  const uint8_t* p;
  __device__ __forceinline__ uint4 v4(int off) const { return *reinterpret_cast<const uint4*>(p + off); }
  __device__ __forceinline__ uint2 v2(int off) const { return *reinterpret_cast<const uint2*>(p + off); }
  __device__ __forceinline__ uint32_t v1(int off) const { return *reinterpret_cast<const uint32_t*>(p + off); }
};

// Copies one record (a multiple of 16 bytes at 16-byte boundaries) to shared memory;
// completion is signalled on `bar` as transaction bytes.
__device__ __forceinline__ void bulk_copy(uint8_t* dst, const uint8_t* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// K and V records of block `phys` (base pointers at the KV head) into a ring slot: K, then
// V. An id outside the pool is not loaded (the barrier is just arrived).
template <int D>
__device__ __forceinline__ void load_int4_block(uint8_t* slot, uint64_t* bar, int phys, int num_pool_blocks,
                                                const uint8_t* kp, const uint8_t* vp, size_t blk_bytes) {
  constexpr int REC = Int4Geom<D>::REC;
  if (phys < num_pool_blocks) {
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(bar, 2 * REC);
    bulk_copy(slot, kp + (size_t)phys * blk_bytes, REC, bar);
    bulk_copy(slot + REC, vp + (size_t)phys * blk_bytes, REC, bar);
  } else {
    mbar_arrive(bar);
  }
}

// Query fragments of NT tiles of 8 rows (query heads), for the k-order of the codes: lane
// (g, t) = (lane / 4, lane % 4) holds row g's dims of words D/32 t .. D/32 t + D/32 - 1 of
// a K row. k-step 2i + h: word i, nibbles 2h, 2h + 4 in b0 and 2h + 1, 2h + 5 (over 16) in
// b1. `f` scales a row's products (2^24 and the row's power of two) and `sum` holds its
// sums per group, both for the rows 2t, 2t + 1 that the lane sees in the product.
template <int D, int NT>
struct Int4Query {
  uint32_t b[NT][D / 16][2];
  float f[NT][2];
  float sum[NT][2][Int4Geom<D>::NG];
};

// Rows are read from shared memory as raw, scaled fp32 values (each row over 2^e_row, so
// that its largest is near 1) and rotated by the row's angles: value(row, dim) and
// cs(row, frequency) give them, row_scale(row) = 2^e_row.
template <int D, int NT, typename ValueFn, typename CsFn, typename ScaleFn>
__device__ __forceinline__ void int4_build_query(Int4Query<D, NT>& q, int lane, ValueFn value, CsFn cs,
                                                 ScaleFn row_scale) {
  constexpr int NG = Int4Geom<D>::NG, HALF = D / 2, W = D / 32;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = 8 * nt + g;
    float s[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) s[j] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int base = 64 * (i % NG) + 8 * ((W * t + i) / NG);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // nibbles 2h, 2h + 4, 2h + 1, 2h + 5
          const int d = base + 2 * h + 4 * (e & 1) + (e >> 1);
          const float2 c = cs(row, d & (HALF - 1));
          const float sn = d < HALF ? -c.y : c.y;
          v[e] = fmaf(value(row, d), c.x, value(row, d ^ HALF) * sn);
        }
        const uint32_t b0 = pack_f16x2(v[0], v[1]), b1 = pack_f16x2(v[2] * 0.0625f, v[3] * 0.0625f);
        q.b[nt][2 * i + h][0] = b0;
        q.b[nt][2 * i + h][1] = b1;
        s[i % NG] += sum_op2<true>(b0) + 16.f * sum_op2<true>(b1);  // the rounded values, as the products see them
      }
    }
    const float rs = row_scale(row);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      s[j] += __shfl_xor_sync(0xffffffffu, s[j], 1);
      s[j] += __shfl_xor_sync(0xffffffffu, s[j], 2);
      s[j] *= rs;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {  // row 2t + c sits in the lanes 4 (2t + c) ..
      const int src = 8 * t + 4 * c;
      q.f[nt][c] = __shfl_sync(0xffffffffu, rs, src) * 16777216.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) q.sum[nt][c][j] = __shfl_sync(0xffffffffu, s[j], src);
    }
  }
}

// Running state of NT tiles of 8 rows: per row the reference maximum m (log2 units), the
// weight sum l and the zeros' sums z (partial over the lanes of equal t until
// int4_finish), and O^T / 2^24 without the zeros: o[4 j + pp][nt], word j of the lane's
// V words (group j), dims 64 j + 8 g + 2 pp in [0], [1] (rows 2t, 2t + 1) and the next
// dim, times 16, in [2], [3]. Weights times V scales go to f16 over `inv`'s power of two
// per group, which follows the scales as they grow: at most 2^8 (weights) x 2^7.
template <int D, int NT>
struct Int4State {
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2], z[NT][2][Int4Geom<D>::NG];
  float inv[Int4Geom<D>::NG], lim[Int4Geom<D>::NG];  // the same in all lanes; a scale above lim moves the reference
};

template <int D, int NT>
__device__ __forceinline__ void int4_init(Int4State<D, NT>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i][nt][0] = st.o[i][nt][1] = st.o[i][nt][2] = st.o[i][nt][3] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      st.m[nt][c] = -INFINITY;
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

constexpr float kInt4RescaleLog2 = 8.f;    // a maximum is refreshed when it grows by more
constexpr float kInt4ScaleHeadroom = 128.f;  // and the V scales' reference by more than this

// One tile of TB blocks of one document. Only the first nv[b] slots of block b are keys
// (0: the block is not there): the other slots' scales and zeros may hold anything.
template <int D, int NT, int TB>
__device__ __forceinline__ void int4_attend(const SharedRecord (&kr)[TB], const SharedRecord (&vr)[TB], const int (&nv)[TB],
                                            const Int4Query<D, NT>& q, Int4State<D, NT>& st, int lane) {
  using G = Int4Geom<D>;
  constexpr int NG = G::NG, W = D / 32;
  const int g = lane >> 2, t = lane & 3;
  bool partial = false;
#pragma unroll
  for (int b = 0; b < TB; ++b) partial |= nv[b] < kBlock;  // warp-uniform

  // S^T: rows g and g + 8 of each block, columns (query rows) 2t and 2t + 1.
  float p[TB][NT][4];
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    uint32_t w0[W], w1[W], m0[NG], m1[NG];
    if constexpr (W == 4) {
      const uint4 x = kr[b].v4(g * G::ROW + 16 * t), y = kr[b].v4((g + 8) * G::ROW + 16 * t);
      w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
      w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
      const uint2 u = kr[b].v2(G::META + g * 8), v = kr[b].v2(G::META + (g + 8) * 8);
      m0[0] = u.x, m0[NG - 1] = u.y, m1[0] = v.x, m1[NG - 1] = v.y;
    } else {
      const uint2 x = kr[b].v2(g * G::ROW + 8 * t), y = kr[b].v2((g + 8) * G::ROW + 8 * t);
      w0[0] = x.x, w0[1] = x.y, w1[0] = y.x, w1[1] = y.y;
      m0[0] = kr[b].v1(G::META + g * 4), m1[0] = kr[b].v1(G::META + (g + 8) * 4);
    }
    float acc[NT][NG][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < NG; ++j) acc[nt][j][0] = acc[nt][j][1] = acc[nt][j][2] = acc[nt][j][3] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = w0[i] >> (8 * h), y = w1[i] >> (8 * h);
        const uint32_t a[4] = {x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816_f16(acc[nt][i % NG], a, q.b[nt][2 * i + h][0], q.b[nt][2 * i + h][1]);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t* m = e < 2 ? m0 : m1;
        float s = meta_scale(m[0]) * acc[nt][0][e], zs = meta_zero(m[0]) * q.sum[nt][e & 1][0];
#pragma unroll
        for (int j = 1; j < NG; ++j) {
          s = fmaf(meta_scale(m[j]), acc[nt][j][e], s);
          zs = fmaf(meta_zero(m[j]), q.sum[nt][e & 1][j], zs);
        }
        p[b][nt][e] = fmaf(q.f[nt][e & 1], s, zs);
      }
    if (partial) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + 8 * (e >> 1) >= nv[b]) p[b][nt][e] = -INFINITY;
    }
  }

  // V's scales and zeros of the same keys.
  float vs[TB][2][NG], vz[TB][2][NG];
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t m[NG];
      if constexpr (NG == 2) {
        const uint2 u = vr[b].v2(G::META + (g + 8 * r) * 8);
        m[0] = u.x, m[NG - 1] = u.y;
      } else {
        m[0] = vr[b].v1(G::META + (g + 8 * r) * 4);
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const bool live = !partial || g + 8 * r < nv[b];
        vs[b][r][j] = live ? meta_scale(m[j]) : 0.f;
        vz[b][r][j] = live ? meta_zero(m[j]) : 0.f;
      }
    }

  // Running maximum and V-scale reference: refreshed together, when some row's maximum or
  // some scale outgrew its reference (a vote; the cross-lane maxima only then).
  float mx[NT][2], sm[NG];
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      mx[nt][c] = -INFINITY;
#pragma unroll
      for (int b = 0; b < TB; ++b) mx[nt][c] = fmaxf(mx[nt][c], fmaxf(p[b][nt][c], p[b][nt][c + 2]));
      grow |= mx[nt][c] > st.m[nt][c] + kInt4RescaleLog2;
    }
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    sm[j] = 0.f;
#pragma unroll
    for (int b = 0; b < TB; ++b) sm[j] = fmaxf(sm[j], fmaxf(vs[b][0][j], vs[b][1][j]));
    grow |= sm[j] > st.lim[j];
  }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sm[j] = fmaxf(sm[j], __shfl_xor_sync(0xffffffffu, sm[j], o));
      if (sm[j] > st.lim[j]) {
        // 2^-(e + 1) for sm in [2^e, 2^(e+1)): between 1/2 and 1 now. Kept a normal number.
        const uint32_t ex = min(max(__float_as_uint(sm[j]) >> 23, 8u), 246u);
        const float inv = __uint_as_float((253u - ex) << 23);
        const float r = inv / st.inv[j];
        st.inv[j] = inv;
        st.lim[j] = kInt4ScaleHeadroom / inv;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[4 * j + i][nt][e] *= r;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = mx[nt][c];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (x > st.m[nt][c] + kInt4RescaleLog2) {
          const float alpha = fast_ex2(st.m[nt][c] - x);  // 0 while the row had no key
          st.m[nt][c] = x;
          st.l[nt][c] *= alpha;
#pragma unroll
          for (int j = 0; j < NG; ++j) st.z[nt][c][j] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            st.o[i][nt][c] *= alpha;
            st.o[i][nt][c + 2] *= alpha;
          }
        }
      }
  }

  // Weights; their sum and the zeros' part in fp32, times the scales in f16 (11 bits: an
  // error of 2^-12 of a term, next to the 4 bits of the codes).
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    uint32_t pb[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mu = st.m[nt][e & 1] == -INFINITY ? 0.f : st.m[nt][e & 1];
        p[b][nt][e] = fast_ex2(p[b][nt][e] - mu);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        st.l[nt][c] += p[b][nt][c] + p[b][nt][c + 2];
#pragma unroll
        for (int j = 0; j < NG; ++j)
          st.z[nt][c][j] = fmaf(p[b][nt][c], vz[b][0][j], fmaf(p[b][nt][c + 2], vz[b][1][j], st.z[nt][c][j]));
      }
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float s = vs[b][r][j] * st.inv[j];
          pb[nt][j][r] = transpose_8x8(pack_f16x2(p[b][nt][2 * r] * s, p[b][nt][2 * r + 1] * s));
        }
    }
    // O^T += C_v^T P^T: rows are dims, the k-order tokens 2t, 2t + 1 (b0), 2t + 8, 2t + 9 (b1).
    uint32_t w[4][NG];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (NG == 2) {
        const uint2 x = vr[b].v2((4 * u + t) * G::ROW + 8 * g);
        w[u][0] = x.x, w[u][NG - 1] = x.y;
      } else {
        w[u][0] = vr[b].v1((4 * u + t) * G::ROW + 4 * g);
      }
    }
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t x = __byte_perm(w[0][j], w[1][j], hf ? 0x7632 : 0x5410);
        const uint32_t y = __byte_perm(w[2][j], w[3][j], hf ? 0x7632 : 0x5410);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t xs = x >> (8 * h), ys = y >> (8 * h);
          const uint32_t a[4] = {xs & 0x000f000fu, xs & 0x00f000f0u, ys & 0x000f000fu, ys & 0x00f000f0u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816_f16(st.o[4 * j + 2 * hf + h][nt], a, pb[nt][j][0], pb[nt][j][1]);
        }
      }
  }
}

// Sums the lanes' parts of l and z: after it every lane holds the rows' full sums.
template <int D, int NT>
__device__ __forceinline__ void int4_finish(Int4State<D, NT>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.l[nt][c] += __shfl_xor_sync(0xffffffffu, st.l[nt][c], o);
#pragma unroll
        for (int j = 0; j < Int4Geom<D>::NG; ++j) st.z[nt][c][j] += __shfl_xor_sync(0xffffffffu, st.z[nt][c][j], o);
      }
}

// The lane's 8 dims 64 j + 8 g + 0..7 of row 8 nt + 2t + c: weighted values, unnormalised.
template <int D, int NT>
__device__ __forceinline__ void int4_out8(const Int4State<D, NT>& st, int j, int nt, int c, float (&v)[8]) {
  const float r = 1.f / st.inv[j];
#pragma unroll
  for (int pp = 0; pp < 4; ++pp) {
    v[2 * pp] = fmaf(st.o[4 * j + pp][nt][c] * 16777216.f, r, st.z[nt][c][j]);
    v[2 * pp + 1] = fmaf(st.o[4 * j + pp][nt][c + 2] * 1048576.f, r, st.z[nt][c][j]);
  }
}

}  // namespace lazy
