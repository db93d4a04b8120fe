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
constexpr int kMembers = LAZY_PLAN_MAX_MEMBERS;
constexpr int kItemInts = LAZY_PLAN_ITEM_INTS;

template <int D, int NT, int HL>
struct Int4Cfg {
  static constexpr int ROWS = Int4Rows<NT, HL>::ALL;
  static constexpr int QS = D + 4;   // fp32 query rows
  static constexpr int RED = D + 4;  // merge rows: o[D], m, l
  static constexpr int SLOT = Int4Loader<D>::STAGE;  // a ring stage: two blocks' K and V records
#ifndef INT4_RING
#define INT4_RING 2
#endif
  static constexpr int RING = NT == 1 ? INT4_RING : 4;  // stages per warp
  static constexpr int BUF = kWarps * RING * SLOT > kWarps * ROWS * RED * 4 ? kWarps * RING * SLOT : kWarps * ROWS * RED * 4;
  static constexpr int SMEM = BUF + ROWS * QS * 4 + kWarps * (D / 2) * 8 + ROWS * 4;
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

// A warp's partial of its rows to shared memory: o[D], m, l per row.
template <int D, int NT, int HL>
__device__ __forceinline__ void int4_store_partial(const Int4State<D, NT, HL>& st, float* red, int stride, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < HL; ++c) {
      float* row = red + (8 * nt + HL * t + c) * stride;
#pragma unroll
      for (int j = 0; j < Int4Geom<D>::NG; ++j) {
        float v[8];
        int4_out8(st, j, nt, c, v);
        float* dst = row + int4_dims(j, g);
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(dst + kInt4Dims2) = make_float4(v[4], v[5], v[6], v[7]);
      }
      if (g == 0) {
        row[D] = st.m[nt][c];
        row[D + 1] = st.l[nt][c];
      }
    }
}

}  // namespace

// ------------------------------------------------------------------ per sequence
// One CTA per (sequence, KV head and tile of 4, 8 or 16 query heads, split), four warps with a
// quarter of the split's blocks each. A warp is its own loader: a ring of RING stages of
// two blocks, each refilled as soon as it was read.
template <int D, int NT, int HL, bool LAZY>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 2) decode_int4_kernel(const DecodeArgs a, int head_tiles) {
  using C = Int4Cfg<D, NT, HL>;
  using G = Int4Geom<D>;
  constexpr int HALF = D / 2, R = C::RING;
  extern __shared__ __align__(128) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + C::BUF);
  float2* cs_all = reinterpret_cast<float2*>(qs + C::ROWS * C::QS);
  float* row_scale = reinterpret_cast<float*>(cs_all + kWarps * HALF);
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

  // ------------------------------------------------------------ first loads
  const int per_warp = (n + kWarps - 1) / kWarps;
  const int kb0 = warp * per_warp;
  const int nk = max(0, min(n, kb0 + per_warp) - kb0);  // blocks of this warp
  const int ns = (nk + 1) / 2;                          // stages: blocks 2i, 2i + 1
  const Int4Loader<D> load(a.k_pool, a.v_pool, a.Hkv, kvh, lane);
  uint8_t* ring = smem + warp * R * C::SLOT;
  auto load_words = [&](int kc, uint32_t& w, uint32_t& wn) {
    const int k = kc + lane, b = b0 + kb0 + k;
    w = k < nk ? __ldg(&wrow[b]) : 0u;
    wn = (k < nk && b + 1 < nb) ? __ldg(&wrow[b + 1]) : 0u;
  };
  // Lane l describes block kc + l; r.nv: valid slots of the blocks l and l + 1, and kSpecial
  // where the pair is not two whole blocks of the document of block l - 1 (or l = 0).
  constexpr int kSpecial = 1 << 16;
  auto describe = [&](int kc, uint32_t w, uint32_t wn) {
    LaneBlock r = describe_block(kc + lane < nk, b0 + kb0 + kc + lane, nb, seq_len, w, wn, a.id_bits, a.num_pool_blocks, a.status);
    const int nv1 = __shfl_down_sync(0xffffffffu, r.nv, 1), p1 = __shfl_down_sync(0xffffffffu, r.p, 1);
    const int p_1 = __shfl_up_sync(0xffffffffu, r.p, 1);
    const bool plain = r.nv == kBlock && nv1 == kBlock && (!LAZY || (lane > 0 && p1 == r.p && p_1 == r.p));
    r.nv |= nv1 << 8 | (plain ? 0 : kSpecial);
    if (r.phys >= a.num_pool_blocks) r.phys = 0;  // no keys in it: any block of the pool
    return r;
  };
  uint32_t w_cur, wn_cur, w_nxt = 0, wn_nxt = 0;
  load_words(0, w_cur, wn_cur);
  if (nk > 32) load_words(32, w_nxt, wn_nxt);
  LaneBlock cur = describe(0, w_cur, wn_cur), nxt{0, 0, 0};
  bool nxt_ready = false;
  auto load_stage = [&](int sl, int phys, int at) {  // the pair that lanes at, at + 1 describe
    const int ph0 = __shfl_sync(0xffffffffu, phys, at), ph1 = __shfl_sync(0xffffffffu, phys, at + 1);
    load(smem_u32(ring) + sl * C::SLOT, ph0, ph1, lane);
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < ns) load_stage(i, cur.phys, 2 * i);
    cp_async_commit();
  }

  // ------------------------------------------------------------ queries
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
  float2* cs = cs_all + warp * HALF;
  Int4Query<D, NT, HL> q;
  auto rebuild = [&](int delta) {
    __syncwarp();
    for (int f = lane; f < HALF; f += 32) cs[f] = rope_cs(__ldg(&a.rope[f]), delta, a.status);
    __syncwarp();
    int4_build_query<D, NT, HL>(
        q, lane, [&](int r) { return qs + r * C::QS; }, [&](int) { return cs; }, [&](int r) { return row_scale[r]; });
  };

  // ------------------------------------------------------------ main loop
  Int4State<D, NT, HL> st;
  int4_init(st);
  int p_cur = INT_MIN;  // the document that q is rotated for
  if constexpr (!LAZY) rebuild(m_pos);  // control: the pool holds absolute-position keys
  for (int i = 0, slot = 0; i < ns; ++i) {
    const int at = (2 * i) & 31;
    if (at == 0 && i > 0) {  // advance the word chunk
      if (!nxt_ready) nxt = describe(2 * i, w_nxt, wn_nxt);
      cur = nxt;
      nxt_ready = false;
      if (2 * i + 32 < nk) load_words(2 * i + 32, w_nxt, wn_nxt);
    }
    cp_async_wait<R - 1>();
    __syncwarp();
    const uint8_t* stage = ring + slot * C::SLOT;
    const SharedRecord kr[2] = {{stage}, {stage + 2 * G::REC}}, vr[2] = {{stage + G::REC}, {stage + 3 * G::REC}};
    const int info = __shfl_sync(0xffffffffu, cur.nv, at);
    const bool special = __any_sync(0xffffffffu, info >= kSpecial);
    int nv[2] = {kBlock, kBlock}, p1 = 0, nv1 = 0;
    if (special) {
      nv[0] = info & 255;
      nv[1] = (info >> 8) & 255;
      if constexpr (LAZY) {
        // A tile lies in one document: where the second block starts another, the first is
        // attended alone, q is rotated anew, and the second follows.
        const int p = __shfl_sync(0xffffffffu, cur.p, at);
        p1 = __shfl_sync(0xffffffffu, cur.p, at + 1);
        if (p != p_cur) rebuild(m_pos - (p_cur = p));
        if (nv[1] > 0 && p1 != p) {
          nv1 = nv[1];
          nv[1] = 0;
        }
      }
    }
    while (true) {
      int4_attend<D, NT, HL>(kr, vr, special, nv, q, st, lane);
      if (!LAZY || nv1 == 0) break;
      nv[0] = 0;
      nv[1] = nv1;
      nv1 = 0;
      rebuild(m_pos - (p_cur = p1));
    }
    __syncwarp();
    // Refill the stage with the warp's pair R positions ahead.
    if (i + R < ns) {
      const int kn = 2 * (i + R);
      if ((kn >> 5) != (i >> 4) && !nxt_ready) {
        nxt = describe(kn & ~31, w_nxt, wn_nxt);
        nxt_ready = true;
      }
      load_stage(slot, (kn >> 5) == (i >> 4) ? cur.phys : nxt.phys, kn & 31);
    }
    cp_async_commit();  // a group a step, empty at the end
    if (++slot == R) slot = 0;
  }
  int4_finish(st);
  __syncthreads();  // every warp is done with its ring: the merge takes its place
  float* red = reinterpret_cast<float*>(smem);
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
// the item's blocks and a ring for them, a warp with one of the tiles, as in
// decode_shared.cu.
namespace {

constexpr int kShRows = 64;

template <int D>
struct Int4SharedCfg {
  using C = Int4Cfg<D, 2, 2>;
  static constexpr int SLOTS = 12;  // ring stages, shared out among the teams: two CTAs fit an SM
  static constexpr int MERGE = kShRows * C::RED * 4;  // [teams][16 RT] rows are 64 in all
  static constexpr int BUF = SLOTS * C::SLOT > MERGE ? SLOTS * C::SLOT : MERGE;
  static constexpr int SMEM = BUF + kShRows * C::QS * 4 + kMembers * (D / 2) * 8;
};

}  // namespace

template <int D, bool LAZY>
__global__ void __launch_bounds__(kThreads, 2) decode_shared_int4_kernel(const SharedDecodeArgs a, const uint8_t* k_pool,
                                                                         const uint8_t* v_pool) {
  constexpr int NT = 2;
  constexpr int HL = 2;
  using C = Int4Cfg<D, NT, HL>;
  using S = Int4SharedCfg<D>;
  using G = Int4Geom<D>;
  constexpr int HALF = D / 2;
  extern __shared__ __align__(128) uint8_t smem[];  // the teams' rings, then the merge area
  float* qs = reinterpret_cast<float*>(smem + S::BUF);               // [64][QS]
  float2* cs_tab = reinterpret_cast<float2*>(qs + kShRows * C::QS);  // [members][HALF]
  __shared__ int4 rec4[kItemInts / 4];
  __shared__ int m_delta[kMembers], m_ok[kMembers];
  __shared__ float row_scale[kShRows];
  const int* rec = reinterpret_cast<const int*>(rec4);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv, item = blockIdx.x / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kItemInts / 4)
    rec4[threadIdx.x] = __ldg(reinterpret_cast<const int4*>(a.items) + (size_t)item * (kItemInts / 4) + threadIdx.x);
  __syncthreads();
  const int src = rec[0], b0 = rec[1], nblk = rec[2], last_nv = rec[3], nmem = rec[4];
  const bool item_ok = src >= 0 && src < a.B && b0 >= 0 && nblk >= 1 && nblk <= a.max_blocks - b0 &&
                       last_nv >= 1 && last_nv <= kBlock && nmem >= 1 && nmem <= kMembers && nmem * a.G <= kShRows;
  if (!item_ok) {  // uniform over the CTA: nothing is loaded or written
    if (threadIdx.x == 0) raise_status(a.status, LAZY_DEV_LAYOUT);
    return;
  }
  auto mem_seq = [&](int m) { return rec[8 + 4 * m]; };
  auto mem_slot = [&](int m) { return rec[8 + 4 * m + 2]; };

  // ------------------------------------------------------------ teams and first loads
  const int rows = nmem * a.G;
  const int RT = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4), TEAMS = kWarps / RT;
  const int team = warp / RT, rt = warp % RT;
  const int R = S::SLOTS / TEAMS;  // ring stages of the team: 3, 6 or 12
  const int per_team = (nblk + TEAMS - 1) / TEAMS;
  const int kb0 = team * per_team;
  const int nk = max(0, min(nblk, kb0 + per_team) - kb0);  // blocks of the team
  uint8_t* ring = smem + team * R * C::SLOT;
  const uint32_t* wrow = a.words + (size_t)src * a.max_blocks + b0 + kb0;
  const uint32_t id_mask = (1u << a.id_bits) - 1u;
  const Int4Loader<D> load(k_pool, v_pool, a.Hkv, kvh, lane);
  auto rec_id = [&](int kb) { return rec[8 + 4 * kMembers + kb]; };
  // Lane l describes team block kc + l, as in decode_shared.cu: the block word decides, and
  // where the record names the block too the two must agree.
  auto describe = [&](int kc, int& phys, int& nv) {
    const int k = kc + lane;
    phys = nv = 0;  // no keys: any block of the pool
    if (k < nk) {
      const int ph = (int)(__ldg(&wrow[k]) & id_mask);
      if (kb0 + k < LAZY_PLAN_ITEM_BLOCK_IDS && rec_id(kb0 + k) != ph) {
        raise_status(a.status, LAZY_DEV_LAYOUT);
      } else if (ph < a.num_pool_blocks) {
        phys = ph;
        nv = kb0 + k == nblk - 1 ? last_nv : kBlock;
      } else {
        raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
      }
    }
  };
  const int ns = (nk + 1) / 2;  // stages: team blocks 2i, 2i + 1
  // A stage is loaded by one warp of the team, in turn.
  auto load_stage = [&](int sl, int ph0, int ph1) { load(smem_u32(ring) + sl * C::SLOT, ph0, ph1, lane); };
  // First loads straight from the record's ids when it names all of them.
  const bool rec_first = kb0 + 2 * min(R - 1, ns) <= LAZY_PLAN_ITEM_BLOCK_IDS;  // uniform over the team
  auto id_of = [&](int k) {
    const int id = k < nk ? rec_id(kb0 + k) : 0;
    return id >= 0 && id < a.num_pool_blocks ? id : 0;
  };
  if (rec_first)
    for (int i = 0; i < R - 1; ++i) {
      if (i < ns && i % RT == rt) load_stage(i, id_of(2 * i), id_of(2 * i + 1));
      cp_async_commit();
    }
  int c_phys, c_nv, n_phys = 0, n_nv = 0;
  describe(0, c_phys, c_nv);
  if (nk > 32) describe(32, n_phys, n_nv);
  if (!rec_first)
    for (int i = 0; i < R - 1; ++i) {
      const int ph0 = __shfl_sync(0xffffffffu, c_phys, 2 * i), ph1 = __shfl_sync(0xffffffffu, c_phys, 2 * i + 1);
      if (i < ns && i % RT == rt) load_stage(i, ph0, ph1);
      cp_async_commit();
    }

  // ------------------------------------------------------------ members and queries
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
  Int4Query<D, NT, HL> q;
  int4_build_query<D, NT, HL>(
      q, lane, [&](int r) { return qs + (16 * rt + r) * C::QS; },
      [&](int r) { return cs_tab + (16 * rt + r < rows ? (16 * rt + r) / a.G : 0) * HALF; },
      [&](int r) { return row_scale[16 * rt + r]; });

  // ------------------------------------------------------------ main loop
  Int4State<D, NT, HL> st;
  int4_init(st);
  bool n_ready = true;
  for (int i = 0, slot = 0, fill = R - 1; i < ns; ++i) {
    const int at = (2 * i) & 31;
    if (i > 0 && at == 0) {
      if (!n_ready) describe(2 * i, n_phys, n_nv);
      c_phys = n_phys;
      c_nv = n_nv;
      n_ready = false;
    }
    // Stage i has landed for the warp that loaded it and, behind the barrier, for the team,
    // all of whose warps are done with stage i - 1, which is refilled.
    if (R == 3) cp_async_wait<1>();
    else if (R == 6) cp_async_wait<4>();
    else cp_async_wait<10>();
    if (RT > 1) team_and(team, 32 * RT, true);
    else __syncwarp();
    if (i + R - 1 < ns) {
      const int kn = 2 * (i + R - 1);
      if ((kn >> 5) != (i >> 4) && !n_ready) {
        describe(kn & ~31, n_phys, n_nv);
        n_ready = true;
      }
      const int phys = (kn >> 5) == (i >> 4) ? c_phys : n_phys;
      const int ph0 = __shfl_sync(0xffffffffu, phys, kn & 31), ph1 = __shfl_sync(0xffffffffu, phys, (kn & 31) + 1);
      if ((i + R - 1) % RT == rt) load_stage(fill, ph0, ph1);
    }
    cp_async_commit();  // a group a step, empty where another warp loads
    const uint8_t* stage = ring + slot * C::SLOT;
    const SharedRecord kr[2] = {{stage}, {stage + 2 * G::REC}}, vr[2] = {{stage + G::REC}, {stage + 3 * G::REC}};
    const int nv[2] = {__shfl_sync(0xffffffffu, c_nv, at), __shfl_sync(0xffffffffu, c_nv, at + 1)};
    int4_attend<D, NT, HL>(kr, vr, __any_sync(0xffffffffu, nv[0] + nv[1] < 2 * kBlock), nv, q, st, lane);
    if (++slot == R) slot = 0;
    if (++fill == R) fill = 0;
  }
  int4_finish(st);
  __syncthreads();  // every team is done with its ring: the merge takes its place

  // ------------------------------------------------------------ partials
  float* red = reinterpret_cast<float*>(smem);
  const int trows = 16 * RT;
  int4_store_partial(st, red + (team * trows + 16 * rt) * C::RED, C::RED, lane);
  __syncthreads();
  constexpr int PER = D / 32;
  for (int r = warp; r < rows; r += kWarps) {
    const int m = r / a.G, h = r - m * a.G;
    if (mem_slot(m) < 0 || mem_slot(m) >= a.num_slots) continue;
    float M = -INFINITY, acc[PER], L = 0.f;
    if (m_ok[m])  // a member that failed its checks leaves an empty partial
      for (int tm = 0; tm < TEAMS; ++tm) M = fmaxf(M, red[(tm * trows + r) * C::RED + D]);
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = 0.f;
    if (m_ok[m])
      for (int tm = 0; tm < TEAMS; ++tm) {
        const float* row = red + (tm * trows + r) * C::RED;
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

template <int D, int NT, int HL, bool LAZY>
static cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t st) {
  using C = Int4Cfg<D, NT, HL>;
  const int ht = (a.G + C::ROWS - 1) / C::ROWS;
  cudaError_t e = set_smem_once<decode_int4_kernel<D, NT, HL, LAZY>>(C::SMEM);
  if (e != cudaSuccess) return e;
  decode_int4_kernel<D, NT, HL, LAZY><<<dim3(a.splits, a.Hkv * ht, a.B), kThreads, C::SMEM, st>>>(a, ht);
  return cudaGetLastError();
}

template <int D, bool LAZY>
static cudaError_t launch_decode_d(const DecodeArgs& a, cudaStream_t st) {
  if (a.G <= 4) return launch_decode_t<D, 1, 1, LAZY>(a, st);
  return a.G <= 8 ? launch_decode_t<D, 1, 2, LAZY>(a, st) : launch_decode_t<D, 2, 2, LAZY>(a, st);
}

cudaError_t launch_decode_int4(const DecodeArgs& a, bool lazy, cudaStream_t st) {
  if (a.D == 128) return lazy ? launch_decode_d<128, true>(a, st) : launch_decode_d<128, false>(a, st);
  return lazy ? launch_decode_d<64, true>(a, st) : launch_decode_d<64, false>(a, st);
}

template <int D, bool LAZY>
static cudaError_t launch_shared_t(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, cudaStream_t st) {
  constexpr int SMEM = Int4SharedCfg<D>::SMEM;
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
