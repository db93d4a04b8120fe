// decode_int4.cu -- the decodes over int4 pools: per sequence (lazy_attn_decode) and over
// shared document runs (lazy_attn_decode_shared). The arithmetic of a tile is in
// int4.cuh; the query rows of a KV head are its heads (per sequence), or members x heads
// (shared).
#include <algorithm>
#include <climits>

#include "decode_block.cuh"
#include "decode_units.cuh"
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
  static constexpr int RED = D + 4;  // merge rows: o[D], m, l
  static constexpr int SLOT = Int4Loader<D>::STAGE;  // a ring stage: two blocks' K and V records
  static constexpr int RING = 2;                // stages per warp
  static constexpr int CTAS = NT == 1 ? 4 : 2;  // per SM
  static constexpr int BUF = kWarps * RING * SLOT > kWarps * ROWS * RED * 4 ? kWarps * RING * SLOT : kWarps * ROWS * RED * 4;
  static constexpr int KEPT = int4_kept_floats<D, NT, HL>();  // per warp (int4.cuh)
  static constexpr int SMEM = BUF + kWarps * (D / 2) * 8 + kWarps * KEPT * 4;
};

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
        row[D] = st.top[nt][c] == -INFINITY ? -INFINITY : -st.neg_m[nt][c];
        row[D + 1] = st.l[nt][c];
      }
    }
}

}  // namespace

// ------------------------------------------------------------------ per sequence
// A unit is a sequence, a KV head and a tile of 4, 8 or 16 of its query heads. Tiles of 8
// where 4 would do take 83 us against 77 on 64 x 4160 tokens, tiles of 8 instead of 16 345
// against 258 on 32 heads per KV head.
// Units are cut into pieces or ranges (decode_units.cuh).
//
// Of a part the four warps take a quarter each. A warp is its own loader: a ring of RING
// stages of two blocks, each refilled as soon as it was read. 64 sequences of 4160 tokens, 32
// heads on 8, take 64 us a call, 4.8 TB/s of records: no pipe is full (integer 55%, issue slots
// 55%), and 16 warps an SM, which is what 128 registers allow, do not hide a tile's chain. With
// 32 heads on one KV head both tiles of 16 heads read the records (872 MB for 466), at 8 warps
// an SM: 250 us, issue slots 51%, tensor 38%.

template <int D, int NT, int HL, bool LAZY>
__global__ void __launch_bounds__(kThreads, Int4Cfg<D, NT, HL>::CTAS) decode_int4_kernel(const UnitDecodeArgs a) {
  using C = Int4Cfg<D, NT, HL>;
  using G = Int4Geom<D>;
  constexpr int HALF = D / 2, R = C::RING;
  constexpr int kSpecial = 1 << 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float2* cs_all = reinterpret_cast<float2*>(smem + C::BUF);
  // Per warp, the blocks of two word chunks (64): ids, and per pair its valid slots (8 bits
  // each) with kSpecial where the pair is not two whole blocks of the document of the block
  // before (or begins a chunk).
  __shared__ int2 d_phys[kWarps][32];
  __shared__ int d_nv[kWarps][32];
  wait_for_launch_before();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ht = a.plan.units / a.Hkv;

  UnitWalk w;
  if (!w.begin(a, warp, lane)) return;
  while (w.next(a)) {
    const int s = w.s, seq_len = w.seq_len, nb = w.nb, u = w.u, lo = w.lo, hi = w.hi;
    const int kvh = u / ht, head0 = (u - kvh * ht) * C::ROWS;
    const int heads = min(C::ROWS, a.G - head0);
    const size_t q0 = (size_t)s * a.Hq + (size_t)kvh * a.G + head0;  // the first row's head
    const int n = hi - lo;                                           // blocks of the part
    const int m_pos = a.q_pos[s];
    const uint32_t* wrow = a.words + (size_t)s * a.max_blocks;

    Int4QueryRows<NT> rows;
    bool live[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = HL == 1 ? lane >> 3 : 8 * nt + (lane >> 2);
      live[nt] = r < heads;
      rows.q[nt] = static_cast<const __nv_bfloat16*>(a.q) + (q0 + (live[nt] ? r : 0)) * D;
    }
    const Int4RawRows<D, NT> raw(rows, lane);  // loads that nothing waits for yet
    float2 rate[HALF / 32];
#pragma unroll
    for (int j = 0; j < HALF / 32; ++j) rate[j] = a.rope[lane + 32 * j];

    // ------------------------------------------------------------ first loads
    // quarters of whole stages
    const int per_warp = ((n + 2 * kWarps - 1) / (2 * kWarps)) * 2;
    const int kb0 = lo + warp * per_warp;
    const int nk = max(0, min(lo + n, kb0 + per_warp) - kb0);  // blocks of this warp
    const int ns = (nk + 1) / 2;                               // stages: blocks 2i, 2i + 1
    const Int4Loader<D> load(a.k_pool, a.v_pool, a.Hkv, kvh, lane);
    const uint32_t ring = smem_u32(smem) + warp * R * C::SLOT;
    uint32_t w_nxt = 0, wn_nxt = 0;
    auto load_words = [&](int kc) {
      const int k = kc + lane, b = kb0 + k;
      w_nxt = k < nk ? wrow[b] : 0u;
      wn_nxt = (k < nk && b + 1 < nb) ? wrow[b + 1] : 0u;
    };
    auto describe = [&](int kc) {  // the chunk of w_nxt
      const LaneBlock r = describe_block(kc + lane < nk, kb0 + kc + lane, nb, seq_len, w_nxt, wn_nxt, a.id_bits,
                                         a.num_pool_blocks, a.status);
      const int nv1 = __shfl_down_sync(0xffffffffu, r.nv, 1), p1 = __shfl_down_sync(0xffffffffu, r.p, 1);
      // a block without keys, left out perhaps, did not have q rotated for its document
      const int p_1 = __shfl_up_sync(0xffffffffu, r.nv > 0 ? r.p : INT_MIN, 1);
      const bool plain = r.nv == kBlock && nv1 == kBlock && (!LAZY || (lane > 0 && p1 == r.p && p_1 == r.p));
      const int k = (kc + lane) & 63;
      reinterpret_cast<int*>(d_phys[warp])[k] = r.phys < a.num_pool_blocks ? r.phys : 0;  // no keys in it: any block
      if (!(lane & 1)) d_nv[warp][k >> 1] = r.nv | nv1 << 8 | (plain ? 0 : kSpecial);
      __syncwarp();
    };
    load_words(0);
    describe(0);
    load_words(32);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < ns) load(ring + i * C::SLOT, d_phys[warp][i].x, d_phys[warp][i].y, lane);
      cp_async_commit();
    }

    // ------------------------------------------------------------ queries
    int4_scale_rows<D, NT>(rows, raw, live, a.scale_log2);
    float2* cs = cs_all + warp * HALF;
    float* kept = reinterpret_cast<float*>(cs_all + kWarps * HALF) + warp * C::KEPT;
    Int4Query<D, NT, HL> q;
    auto rebuild = [&](int delta) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < HALF / 32; ++j) cs[lane + 32 * j] = rope_cs(rate[j], delta, a.status);
      __syncwarp();
      int4_build_query<D, NT, HL>(q, rows, lane, [&](int) { return cs; });
    };
    // Rotated while the first records are on their way (one sequence of 16384 tokens from
    // HBM: 21.3 us against 23.0 behind them). q_pos is read again where the document changes:
    // the loop has no register for it. Control: the pool holds absolute-position keys.
    int p_cur = 0;  // the document that q is rotated for
    if (ns > 0) {
      if constexpr (LAZY) p_cur = decode_word(wrow[kb0], kb0, a.id_bits).p;
      rebuild(m_pos - p_cur);
    }

    // ------------------------------------------------------------ main loop
    Int4State<D, NT, HL> st;
    int4_init(st);
    for (int i = 0, slot = 0; i < ns; ++i) {
      if ((i & 15) == 0) {
        if (2 * i + 32 < nk) {  // a chunk of words ahead
          describe(2 * i + 32);
          load_words(2 * i + 64);
        }
        if (i > 0 && i % kInt4Flush == 0) int4_flush(st, kept, i > kInt4Flush, lane);
      }
      cp_async_wait<R - 1>();
      __syncwarp();
      const uint8_t* stage = smem + (warp * R + slot) * C::SLOT;
      const SharedRecord kr[2] = {{stage}, {stage + 2 * G::REC}}, vr[2] = {{stage + G::REC}, {stage + 3 * G::REC}};
      const int info = d_nv[warp][i & 31];
      const bool special = __any_sync(0xffffffffu, info >= kSpecial);
      int nv[2] = {kBlock, kBlock}, p1 = 0, nv1 = 0;
      if (special) {
        nv[0] = info & 255;
        nv[1] = (info >> 8) & 255;
        if constexpr (LAZY) {
          // A tile lies in one document: where the second block starts another, the first is
          // attended alone, q is rotated anew, and the second follows.
          const int b = kb0 + 2 * i, p0 = decode_word(wrow[b], b, a.id_bits).p;
          if (p0 != p_cur) rebuild(a.q_pos[s] - (p_cur = p0));
          p1 = nv[1] > 0 ? decode_word(wrow[b + 1], b + 1, a.id_bits).p : p0;
          if (p1 != p0) {
            nv1 = nv[1];
            nv[1] = 0;
          }
        }
      }
      while (true) {
        int4_attend<D, NT, HL>(kr, vr, special, nv, q, st, lane, i >= kInt4Flush ? kept : nullptr);
        if (!LAZY || nv1 == 0) break;
        nv[0] = 0;
        nv[1] = nv1;
        nv1 = 0;
        rebuild(a.q_pos[s] - (p_cur = p1));
      }
      __syncwarp();
      if (i + R < ns) {  // refill the stage with the warp's pair R positions ahead
        const int2 ph = d_phys[warp][(i + R) & 31];
        load(ring + slot * C::SLOT, ph.x, ph.y, lane);
      }
      cp_async_commit();  // a group a step, empty at the end
      if (++slot == R) slot = 0;
    }
    if (ns > kInt4Flush) int4_unflush(st, kept, lane);
    int4_finish(st);
    __syncthreads();  // every warp is done with its ring: the merge takes its place
    float* red = reinterpret_cast<float*>(smem);
    int4_store_partial(st, red + warp * C::ROWS * C::RED, C::RED, lane);
    __syncthreads();
    const bool whole = lo == 0 && hi == nb;
    const size_t slot0 = (2 * (size_t)blockIdx.x + (lo == 0 ? 1 : 0)) * C::ROWS;
    for (int idx = threadIdx.x; idx < heads * D; idx += kThreads) {
      const int row = idx / D, col = idx % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[(w * C::ROWS + row) * C::RED + D]);
      const float Mr = M == -INFINITY ? 0.f : M;  // no keys: all sums are 0 (or NaN, which stays)
      float acc = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* src = red + (w * C::ROWS + row) * C::RED;
        const float f = fast_ex2(src[D] - Mr);
        acc += f * src[col];
        L += f * src[D + 1];
      }
      if (whole) {
        static_cast<__nv_bfloat16*>(a.out)[(q0 + row) * D + col] = __float2bfloat16_rn(L == 0.f ? 0.f : acc / L);
      } else {
        a.ws_o[(slot0 + row) * D + col] = acc;
        if (col == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * (slot0 + row)) = make_float2(M, L);
      }
    }
    if (w.last()) return;
    __syncthreads();  // the next part's loads and queries take the merge's place
  }
}

// ------------------------------------------------------------------ shared runs
// One CTA per (work item, KV head, 32 of its up to 64 rows). Rows are members x heads; a
// warp takes a tile of 8 of them (of 4 where there are no more), and the warps form 4 / RT
// teams of RT = 1, 2 or 4 warps with a contiguous part of the item's blocks and a ring of
// stages each. Tiles of 16 rows would unpack each code half as often, but hold 240
// registers, two CTAs an SM: 197 us against 154 on 32 x 16384 tokens of Zipf-drawn
// documents with 8 query heads per KV head, in items of 32 blocks. In items of 64, the long
// and wide ones first, the 8-row tiles take 126 us, 1.7 TB/s of unique records: bound by the
// instructions of a tile, once per 8 rows (59% of the issue slots, integer 56%, tensor 25%).
namespace {

constexpr int kShRows = 32;    // rows of a CTA
constexpr int kShStages = 8;   // ring stages, shared out among the teams

template <int D>
struct Int4SharedCfg {
  static constexpr int SLOT = Int4Loader<D>::STAGE;
  static constexpr int RED = D + 4;                   // merge rows: o[D], m, l
  static constexpr int MERGE = kWarps * 8 * RED * 4;  // [teams][8 RT] rows are 32 in all
  static constexpr int BUF = kShStages * SLOT > MERGE ? kShStages * SLOT : MERGE;
  // the members' angles, then, once the queries are built, the warps' kept sums (int4.cuh)
  static constexpr int KEPT = int4_kept_floats<D, 1, 2>();
  static constexpr int ANGLES = kMembers * (D / 2) * 8;
  static constexpr int SMEM = BUF + (ANGLES > kWarps * KEPT * 4 ? ANGLES : kWarps * KEPT * 4);
};

// The n threads of team t meet (barrier 0 is the CTA's).
__device__ __forceinline__ void team_sync(int t, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(t + 1), "r"(n) : "memory");
}

// What the CTA's warps share of an item.
struct Int4Item {
  int rec[kItemInts];
  int delta[kMembers], ok[kMembers];  // rotation offset of each member; it passed its checks
  int2 d_phys[kWarps][32];            // per team: the blocks of two word chunks
  int2 d_nv[kWarps][32];              // and their valid slots
};

}  // namespace

// The item's rows row0 .. row0 + 8 RT - 1 (4 with HL = 1, where RT = 1), from `rows` of them.
// One body for every RT: one per RT made the four warps of a scheduler wait two cycles an
// instruction for their code.
template <int D, int HL, bool LAZY>
__device__ __forceinline__ void shared_int4_rows(const SharedDecodeArgs& a, const uint8_t* k_pool, const uint8_t* v_pool,
                                                 Int4Item& it, uint8_t* smem, float2* cs_tab, int kvh, int row0,
                                                 int rows, int RT) {
  using C = Int4SharedCfg<D>;
  using G = Int4Geom<D>;
  constexpr int HALF = D / 2;
  const int TEAMS = kWarps / RT, R = kShStages / TEAMS, AHEAD = R - 1;  // R = 2, 4 or 8
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / RT, rt = warp & (RT - 1);
  const int src = it.rec[0], b0 = it.rec[1], nblk = it.rec[2], last_nv = it.rec[3];

  // ------------------------------------------------------------ first loads
  // parts of whole stages
  const int per_team = (nblk + 2 * TEAMS - 1) / (2 * TEAMS) * 2;
  const int kb0 = team * per_team;
  const int nk = max(0, min(nblk, kb0 + per_team) - kb0);  // blocks of the team
  const int ns = (nk + 1) / 2;                             // stages: team blocks 2i, 2i + 1
  const Int4Loader<D> load(k_pool, v_pool, a.Hkv, kvh, lane);
  const uint32_t ring = smem_u32(smem) + team * R * C::SLOT;
  const uint32_t* wrow = a.words + (size_t)src * a.max_blocks + b0 + kb0;
  const uint32_t id_mask = (1u << a.id_bits) - 1u;
  const int* ids = it.rec + 8 + 4 * kMembers;  // the record's block ids
  uint32_t w_nxt = 0u;
  auto load_words = [&](int kc) {
    if (kc + lane < nk) w_nxt = wrow[kc + lane];
  };
  // Chunk kc of the team's words (w_nxt) to its descriptors, by every warp of the team alike.
  // The block word decides; where the record names the block too the two must agree.
  auto describe = [&](int kc) {
    const int k = kc + lane;
    int phys = 0, nv = 0;  // no keys: any block of the pool
    if (k < nk) {
      const int ph = (int)(w_nxt & id_mask);
      if (kb0 + k < LAZY_PLAN_ITEM_BLOCK_IDS && ids[kb0 + k] != ph) {
        raise_status(a.status, LAZY_DEV_LAYOUT);
      } else if (ph < a.num_pool_blocks) {
        phys = ph;
        nv = kb0 + k == nblk - 1 ? last_nv : kBlock;
      } else {
        raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
      }
    }
    if (rt == 0) {
      reinterpret_cast<int*>(it.d_phys[team])[k & 63] = phys;
      reinterpret_cast<int*>(it.d_nv[team])[k & 63] = nv;
    }
    __syncwarp();
  };
  load_words(0);
  // First loads straight from the record's ids when it names all of them.
  const bool rec_first = kb0 + 2 * min(AHEAD, ns) <= LAZY_PLAN_ITEM_BLOCK_IDS;  // uniform over the team
  auto id_of = [&](int k) {
    const int id = k < nk ? ids[kb0 + k] : 0;
    return id >= 0 && id < a.num_pool_blocks ? id : 0;
  };
  if (rec_first) {
    for (int i = 0; i < AHEAD; ++i) {
      if (i < ns && (i & (RT - 1)) == rt) load(ring + i * C::SLOT, id_of(2 * i), id_of(2 * i + 1), lane);
      cp_async_commit();
    }
  }
  describe(0);
  load_words(32);
  if (RT > 1) team_sync(team, 32 * RT);
  if (!rec_first) {
    for (int i = 0; i < AHEAD; ++i) {
      if (i < ns && (i & (RT - 1)) == rt) load(ring + i * C::SLOT, it.d_phys[team][i].x, it.d_phys[team][i].y, lane);
      cp_async_commit();
    }
  }

  // ------------------------------------------------------------ members
  const int nmem = it.rec[4];
  if (threadIdx.x < nmem) {
    const int m = threadIdx.x, seq = it.rec[8 + 4 * m], bm = it.rec[8 + 4 * m + 1], slot = it.rec[8 + 4 * m + 2];
    bool good = seq >= 0 && seq < a.B && bm >= 0 && bm <= a.max_blocks - nblk && slot >= 0 && slot < a.num_slots;
    int delta = 0;
    if (good) {
      const BlockInfo mi = decode_word(a.words[(size_t)seq * a.max_blocks + bm], bm, a.id_bits);
      good = mi.phys == decode_word(a.words[(size_t)src * a.max_blocks + b0], b0, a.id_bits).phys;
      const int qp = a.q_pos[seq];
      delta = LAZY ? qp - mi.p : qp;
    }
    if (!good) raise_status(a.status, LAZY_DEV_LAYOUT);
    it.ok[m] = good;
    it.delta[m] = delta;
  }
  __syncthreads();
  // the angles of the CTA's members
  const int m0 = row0 / a.G, m1 = (rows - 1) / a.G;
  for (int idx = m0 * HALF + threadIdx.x; idx < (m1 + 1) * HALF; idx += kThreads)
    cs_tab[idx] = rope_cs(a.rope[idx % HALF], it.delta[idx / HALF], a.status);
  __syncthreads();

  // ------------------------------------------------------------ queries
  auto mem_seq = [&](int m) { return it.rec[8 + 4 * m]; };
  auto mem_slot = [&](int m) { return it.rec[8 + 4 * m + 2]; };
  Int4QueryRows<1> qrows;
  const int r = row0 + (HL == 1 ? lane >> 3 : 8 * rt + (lane >> 2)), rc = r < rows ? r : row0;
  const int mem = rc / a.G;
  const bool live[1] = {r < rows && it.ok[mem]};
  qrows.q[0] = static_cast<const __nv_bfloat16*>(a.q) +
               ((live[0] ? (size_t)mem_seq(mem) * a.Hq + (rc - mem * a.G) : 0) + (size_t)kvh * a.G) * D;
  int4_scale_rows<D, 1>(qrows, Int4RawRows<D, 1>(qrows, lane), live, a.scale_log2);
  Int4Query<D, 1, HL> q;
  int4_build_query<D, 1, HL>(q, qrows, lane, [&](int) { return cs_tab + mem * HALF; });

  // ------------------------------------------------------------ main loop
  float* kept = reinterpret_cast<float*>(cs_tab) + warp * C::KEPT;
  if (per_team > 2 * kInt4Flush) __syncthreads();  // sums will be kept where the angles were
  Int4State<D, 1, HL> st;
  int4_init(st);
  const uint8_t* ring_p = smem + team * R * C::SLOT;
  for (int i = 0; i < ns; ++i) {
    // Stage i has landed for the warp that loaded it and, behind the barrier, for the team,
    // all of whose warps are done with stage i - 1, which is refilled.
    if (RT == 1) {
      cp_async_wait<0>();
      __syncwarp();
    } else {
      if (RT == 2) cp_async_wait<2>();
      else cp_async_wait<6>();
      team_sync(team, 32 * RT);
    }
    if ((i & 15) == 0) {  // a chunk of words ahead, over the one that all are done with
      describe(2 * i + 32);
      load_words(2 * i + 64);
      if (i > 0 && i % kInt4Flush == 0) int4_flush(st, kept, i > kInt4Flush, lane);
    }
    const int n = i + AHEAD;
    if (n < ns && (n & (RT - 1)) == rt) {
      const int2 ph = it.d_phys[team][n & 31];
      load(ring + (n & (R - 1)) * C::SLOT, ph.x, ph.y, lane);
    }
    cp_async_commit();  // a group a step, empty where another warp loads
    const uint8_t* stage = ring_p + (i & (R - 1)) * C::SLOT;
    const SharedRecord kr[2] = {{stage}, {stage + 2 * G::REC}}, vr[2] = {{stage + G::REC}, {stage + 3 * G::REC}};
    const int2 v = it.d_nv[team][i & 31];
    const int nv[2] = {v.x, v.y};
    int4_attend<D, 1, HL>(kr, vr, __any_sync(0xffffffffu, v.x + v.y < 2 * kBlock), nv, q, st, lane,
                          i >= kInt4Flush ? kept : nullptr);
  }
  if (ns > kInt4Flush) int4_unflush(st, kept, lane);
  int4_finish(st);
  __syncthreads();  // every team is done with its ring: the merge takes its place

  // ------------------------------------------------------------ partials
  float* red = reinterpret_cast<float*>(smem);
  int4_store_partial(st, red + (team * RT + rt) * 8 * C::RED, C::RED, lane);
  __syncthreads();
  constexpr int PER = D / 32;
  const int n = min(rows - row0, HL == 1 ? 4 : 8 * RT);
  for (int x = warp; x < n; x += kWarps) {
    const int m = (row0 + x) / a.G, h = row0 + x - m * a.G;
    if (mem_slot(m) < 0 || mem_slot(m) >= a.num_slots) continue;
    float M = -INFINITY, acc[PER], L = 0.f;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = 0.f;
    if (it.ok[m]) {  // a member that failed its checks leaves an empty partial
      for (int tm = 0; tm < TEAMS; ++tm) M = fmaxf(M, red[(tm * RT * 8 + x) * C::RED + D]);
      const float Mr = M == -INFINITY ? 0.f : M;
      for (int tm = 0; tm < TEAMS; ++tm) {
        const float* row = red + (tm * RT * 8 + x) * C::RED;
        const float w = fast_ex2(row[D] - Mr);
        L += w * row[D + 1];
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] += w * row[lane + 32 * c];
      }
      if (L != 0.f) M = Mr;  // all scores NaN: not an empty slot, which the combine would pass over
    }
    const size_t pidx = (size_t)mem_slot(m) * a.Hq + (size_t)kvh * a.G + h;
#pragma unroll
    for (int c = 0; c < PER; ++c) a.ws_o[pidx * D + lane + 32 * c] = acc[c];
    if (lane == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * pidx) = make_float2(M, L);
  }
}

template <int D, bool LAZY>
__global__ void __launch_bounds__(kThreads, 4) decode_shared_int4_kernel(const SharedDecodeArgs a, const uint8_t* k_pool,
                                                                         const uint8_t* v_pool, int halves) {
  using C = Int4SharedCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];            // the teams' rings, then the merge area
  float2* cs_tab = reinterpret_cast<float2*>(smem + C::BUF);  // [members][D / 2]
  __shared__ __align__(16) Int4Item it;
  wait_for_launch_before();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv, item = blockIdx.x / a.Hkv / halves, half = blockIdx.x / a.Hkv % halves;
  if (threadIdx.x < kItemInts / 4)
    reinterpret_cast<int4*>(it.rec)[threadIdx.x] =
        reinterpret_cast<const int4*>(a.items)[(size_t)item * (kItemInts / 4) + threadIdx.x];
  __syncthreads();
  const int src = it.rec[0], b0 = it.rec[1], nblk = it.rec[2], last_nv = it.rec[3], nmem = it.rec[4];
  const bool item_ok = src >= 0 && src < a.B && b0 >= 0 && nblk >= 1 && nblk <= a.max_blocks - b0 &&
                       last_nv >= 1 && last_nv <= kBlock && nmem >= 1 && nmem <= kMembers && nmem * a.G <= 2 * kShRows;
  if (!item_ok) {  // uniform over the CTA: nothing is loaded or written
    if (threadIdx.x == 0) raise_status(a.status, LAZY_DEV_LAYOUT);
    return;
  }
  const int row0 = half * kShRows, all = nmem * a.G, rows = min(all, row0 + kShRows);
  if (row0 >= all) return;
  const int n = rows - row0;
  if (n <= 4) shared_int4_rows<D, 1, LAZY>(a, k_pool, v_pool, it, smem, cs_tab, kvh, row0, rows, 1);
  else shared_int4_rows<D, 2, LAZY>(a, k_pool, v_pool, it, smem, cs_tab, kvh, row0, rows, n <= 8 ? 1 : (n <= 16 ? 2 : 4));
}

// ------------------------------------------------------------------ launchers

UnitPlan plan_decode_int4(int B, int G, int Hkv, int max_blocks, int num_splits, int sms) {
  const int rows = G <= 4 ? 4 : (G <= 8 ? 8 : 16);
  const int per_sm = rows < 16 ? Int4Cfg<128, 1, 1>::CTAS : Int4Cfg<128, 2, 2>::CTAS;
  return plan_units(B, rows, Hkv * ((G + rows - 1) / rows), max_blocks, num_splits, (int64_t)sms * per_sm, kMinPieceLog2);
}

template <int D, int NT, int HL, bool LAZY>
static cudaError_t launch_decode_t(const UnitDecodeArgs& a, cudaStream_t st) {
  using C = Int4Cfg<D, NT, HL>;
  cudaError_t e = set_smem_once<decode_int4_kernel<D, NT, HL, LAZY>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_behind(decode_int4_kernel<D, NT, HL, LAZY>, (unsigned)a.plan.ctas, kThreads, C::SMEM, st, a);
}

template <int D, bool LAZY>
static cudaError_t launch_decode_d(const UnitDecodeArgs& a, cudaStream_t st) {
  if (a.plan.rows == 4) return launch_decode_t<D, 1, 1, LAZY>(a, st);
  return a.plan.rows == 8 ? launch_decode_t<D, 1, 2, LAZY>(a, st) : launch_decode_t<D, 2, 2, LAZY>(a, st);
}

cudaError_t launch_decode_int4(const UnitDecodeArgs& a, bool lazy, cudaStream_t st) {
  if (a.D == 128) return lazy ? launch_decode_d<128, true>(a, st) : launch_decode_d<128, false>(a, st);
  return lazy ? launch_decode_d<64, true>(a, st) : launch_decode_d<64, false>(a, st);
}

template <int D, bool LAZY>
static cudaError_t launch_shared_t(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, cudaStream_t st) {
  constexpr int SMEM = Int4SharedCfg<D>::SMEM;
  cudaError_t e = set_smem_once<decode_shared_int4_kernel<D, LAZY>>(SMEM);
  if (e != cudaSuccess) return e;
  const int halves = std::min(kMembers * a.G, 2 * kShRows) > kShRows ? 2 : 1;
  const long long grid = (long long)a.num_items * a.Hkv * halves;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_behind(decode_shared_int4_kernel<D, LAZY>, (unsigned)grid, kThreads, SMEM, st, a,
                       static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool), halves);
}

cudaError_t launch_decode_shared_int4(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, bool lazy,
                                      cudaStream_t st) {
  if (a.num_items == 0) return cudaSuccess;
  if (a.D == 128)
    return lazy ? launch_shared_t<128, true>(a, k_pool, v_pool, st) : launch_shared_t<128, false>(a, k_pool, v_pool, st);
  return lazy ? launch_shared_t<64, true>(a, k_pool, v_pool, st) : launch_shared_t<64, false>(a, k_pool, v_pool, st);
}

}  // namespace lazy
