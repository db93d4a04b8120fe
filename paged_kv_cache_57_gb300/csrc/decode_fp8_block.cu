// decode_fp8_block.cu -- the decodes over pools of e4m3 codes with a scale per block and head:
// per sequence (lazy_attn_decode) and over shared document runs (lazy_attn_decode_shared). The
// arithmetic of a block is in fp8_block.cuh; the query rows of a KV head are its heads (per
// sequence), or members x heads (shared).
//
// Four warps form 4 / RT teams of RT = 1 (per sequence: always), 2 or 4. A team takes a contiguous part of
// the CTA's blocks through a ring of stages in shared memory; each of its warps has its own tile
// of 4, 8, 16 or 32 query rows. A block's K and V records are two bulk copies, which one lane starts
// and the stage's mbarrier counts, every wait with a limit: a warp's own cp.async of them, nine
// instructions and their addresses in every lane, took 94 us where these take 86.
//
// Measured (8 KV heads of 128 dims unless said; calls in a row). Per sequence: 64 of 4096 tokens, 32 heads, 545 MB,
// 85 us, 6.4 TB/s: memory; one of 16384, 64 heads, 13.7 us: the chain of a piece, the join and two
// launches; 48 of 256 to 131072, 32 heads on one, 829 MB, 227 us, 3.6 TB/s: instructions. There an
// mma.sync m16n8k16 holds its scheduler for 8 cycles, so that a block of 32 rows costs an SM 144 cycles of products
// beside 116 of softmax and loop, for 180 of memory. Shared runs: 64 sequences of 4096 tokens, Zipf-drawn, 48 us
// for 151 MB, of which the prologue of an item (record, members, angles, queries) and the join are about
// 12 (the rest was not taken apart); 32 of 16384, 64 heads, 112 us for 386 MB: alone, items of up to 16 rows take 68 us, bound by
// memory, the wider ones 71, by instructions.
#include <algorithm>
#include <climits>

#include "decode_units.cuh"
#include "fp8_block.cuh"

namespace lazy {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMembers = LAZY_PLAN_MAX_MEMBERS;
constexpr int kItemInts = LAZY_PLAN_ITEM_INTS;

template <int D, int NT, int HL>
struct Fp8Cfg {
  static constexpr int ROWS = Fp8Rows<NT, HL>::ALL;  // of a warp
  static constexpr int RED = D + 4;                  // merge rows: o[D], m, l
  static constexpr int SLOT = Fp8Ring<D>::STAGE;     // one block
  // Per SM, as registers allow. 32 rows as two warps of a team with 16 each, at three CTAs: 234 to 244 us for
  // 235 at the time, with twice the conversions.
  static constexpr int CTAS = NT == 1 ? 4 : (NT == 2 ? 3 : 2);
  static constexpr int RING = NT == 1 ? 2 : 4;  // stages of a warp
  static constexpr int SLOTS = kWarps * RING;
  static_assert(SLOTS <= kFp8Slots, "barriers");
  static constexpr int BUF = SLOTS * SLOT > kWarps * ROWS * RED * 4 ? SLOTS * SLOT : kWarps * ROWS * RED * 4;
};

}  // namespace

// ------------------------------------------------------------------ per sequence
// A unit is a sequence, a KV head and a tile of 4, 8, 16 or 32 of its query heads; the units
// are cut into pieces or ranges (decode_units.cuh). Of a part each warp takes a quarter, by itself.
// LONG: a warp may have more than kFp8Keep blocks of a part.
template <int D, int NT, int HL, bool LAZY, bool LONG>
__global__ void __launch_bounds__(kThreads, Fp8Cfg<D, NT, HL>::CTAS) decode_fp8_block_kernel(const UnitDecodeArgs a) {
  using C = Fp8Cfg<D, NT, HL>;
  constexpr int HALF = D / 2, R = C::RING;
  // Blocks are started PAIR at a time, AHEAD of the one in work; EARLY before the first. (One at a time took 32 rows'
  // 235 us for 230; in the shared decode pairs brought nothing.)
  constexpr int PAIR = R >= 4 ? 2 : 1, AHEAD = R - PAIR, EARLY = PAIR == 2 ? R : AHEAD;
  constexpr int kNewDoc = 32;
  extern __shared__ __align__(128) uint8_t smem[];
  float2* cs_all = reinterpret_cast<float2*>(smem + C::BUF);
  uint32_t* q_all = reinterpret_cast<uint32_t*>(cs_all + kWarps * HALF);
  __shared__ Fp8Bars bars;
  if (threadIdx.x < C::SLOTS) {
    mbar_init(&bars.full[threadIdx.x], 1);
    fence_barrier_init();
  }
  __syncthreads();
  wait_for_launch_before();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ht = a.plan.units / a.Hkv;

  uint32_t used = 0;  // blocks that went through the ring before this part
  UnitWalk w;
  if (!w.begin(a, warp, lane)) return;
  while (w.next(a)) {
    const int s = w.s, seq_len = w.seq_len, nb = w.nb, lo = w.lo, hi = w.hi;
    const int kvh = w.u / ht, head0 = (w.u - kvh * ht) * C::ROWS;
    const int heads = min(C::ROWS, a.G - head0);
    const size_t q0 = (size_t)s * a.Hq + (size_t)kvh * a.G + head0;  // the first row's head
    const int n = hi - lo;                                           // blocks of the part
    const int m_pos = a.q_pos[s];
    const uint32_t* wrow = a.words + (size_t)s * a.max_blocks;

    const int row0 = HL == 1 ? lane >> 3 : lane >> 2;  // the lane's first row, the others 8 on
    const __nv_bfloat16* q_first = static_cast<const __nv_bfloat16*>(a.q) + q0 * D;
    auto row = [&](int nt) { return q_first + (row0 + 8 * nt < heads ? row0 + 8 * nt : 0) * D; };
    bool live[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) live[nt] = row0 + 8 * nt < heads;
    const Fp8RawRows<D, NT> raw(row, lane);  // loads that nothing waits for yet
    float2 rate[HALF / 32];
#pragma unroll
    for (int j = 0; j < HALF / 32; ++j) rate[j] = a.rope[lane + 32 * j];

    // ------------------------------------------------------------ first loads
    const int per_warp = (n + kWarps - 1) / kWarps;
    const int kb0 = lo + warp * per_warp;
    const int nk = max(0, min(lo + n, kb0 + per_warp) - kb0);  // blocks of this warp
    const size_t head = (size_t)kvh * Fp8Geom<D>::REC;
    const Fp8Ring<D> ring{static_cast<const uint8_t*>(a.k_pool) + head, static_cast<const uint8_t*>(a.v_pool) + head,
                          (uint32_t)a.Hkv * Fp8Geom<D>::REC, smem + warp * R * C::SLOT, &bars, warp * R};
    // A chunk of 32 blocks in the lanes: id, and valid slots with kNewDoc where the block is not one of the
    // document of the block before (or begins a chunk).
    int c_phys = 0, c_info = 0;
    uint32_t w_nxt = 0, wn_nxt = 0;
    auto load_words = [&](int kc) {
      const int k = kc + lane, b = kb0 + k;
      w_nxt = k < nk ? wrow[b] : 0u;
      wn_nxt = (k < nk && b + 1 < nb) ? wrow[b + 1] : 0u;
    };
    auto describe = [&](int kc) {  // the chunk of w_nxt
      const LaneBlock r = describe_block(kc + lane < nk, kb0 + kc + lane, nb, seq_len, w_nxt, wn_nxt, a.id_bits,
                                         a.num_pool_blocks, a.status);
      // a block without keys is left out and did not have q rotated for its document
      const int p_1 = __shfl_up_sync(0xffffffffu, r.nv > 0 ? r.p : INT_MIN, 1);
      c_phys = r.phys < a.num_pool_blocks ? r.phys : 0;  // no keys in it: any block
      c_info = r.nv | (!LAZY || (lane > 0 && p_1 == r.p) ? 0 : kNewDoc);
    };
    auto fill = [&](int j) {  // the stages of blocks j .. j + PAIR - 1 are loaded, by the lanes that hold the blocks
      if ((j & 31) == 0 && j < nk) {
        describe(j);
        load_words(j + 32);
      }
      const int off = lane - (j & 31);
      if (off >= 0 && off < PAIR && j + off < nk) ring.fill((used + j + off) % R, c_phys, c_info);
    };
    load_words(0);
#pragma unroll 1
    for (int i = 0; i < EARLY; i += PAIR) fill(i);

    // ------------------------------------------------------------ queries
    Fp8Query<D, NT, HL> q;
    float mul[NT];
    fp8_scale_rows<D, NT, HL>(q, mul, raw, live, a.scale_log2, lane);
    q.s = q_all + warp * (Fp8Query<D, NT, HL>::BYTES / 4) + 4 * lane;
    float2* cs = cs_all + warp * HALF;
    auto rebuild = [&](int delta) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < HALF / 32; ++j) cs[lane + 32 * j] = rope_cs(rate[j], delta, a.status);
      __syncwarp();
      fp8_build_query<D, NT, HL>(mul, row, lane, [&](int) { return cs; }, [&](int nt, int k, int h, uint32_t x) { q.set(nt, k, h, x); });
    };
    // Rotated while the first records are on their way. Control: the pool holds absolute-position keys.
    int p_cur = 0;  // the document that q is rotated for
    if (nk > 0) {
      if constexpr (LAZY) p_cur = decode_word(wrow[kb0], kb0, a.id_bits).p;
      rebuild(m_pos - p_cur);
    }

    // ------------------------------------------------------------ main loop
    Fp8State<D, NT, HL> st;
    fp8_init(st);
    bool ok = true;
    Fp8Kept<D, NT, HL> kept;  // (LONG)
    kept.any = false;
    int i = 0;
#pragma unroll 1
    for (int end = LONG ? min(nk, kFp8Keep) : nk;; end = min(nk, end + kFp8Keep)) {
      for (; i < end; ++i) {
        const uint32_t n_th = used + i, slot = n_th % R;
        if (PAIR == 1 || (i % 2 == 0 && i > 0)) fill(i + AHEAD);
        ok = ring.wait_full(slot, n_th / R & 1, a.status);
        if (!ok) {
          ring.drain(n_th, used + min(nk, i + R), R, a.status);
          break;
        }
        const int info = bars.info[warp * R + slot];
        int nv = kBlock;
        if (info != kBlock) {
          nv = info & 31;
          if (LAZY && info > kNewDoc) {
            const int p = decode_word(wrow[kb0 + i], kb0 + i, a.id_bits).p;
            if (p != p_cur) rebuild(a.q_pos[s] - (p_cur = p));
          }
        }
        if (nv > 0) fp8_attend<D, NT, HL>(ring.base + slot * C::SLOT, nv, q, st, lane);
        __syncwarp();  // the stage is free
      }
      if (!LONG || !ok || end == nk) break;
      kept.keep(st);
    }
    if (LONG) kept.give_back(st);
    used += nk;
    fp8_finish(st);
    __syncthreads();  // every warp is done with its ring: the merge takes its place
    float* red = reinterpret_cast<float*>(smem);
    fp8_store_partial(st, red + warp * C::ROWS * C::RED, C::RED, lane);
    __syncthreads();
    const bool whole = lo == 0 && hi == nb;
    const size_t slot0 = (2 * (size_t)blockIdx.x + (lo == 0 ? 1 : 0)) * C::ROWS;
    for (int idx = threadIdx.x; idx < heads * D; idx += kThreads) {
      const int row = idx / D, col = idx % D;
      float M = -INFINITY;
#pragma unroll
      for (int tm = 0; tm < kWarps; ++tm) M = fmaxf(M, red[(tm * C::ROWS + row) * C::RED + D]);
      const float Mr = M == -INFINITY ? 0.f : M;  // no keys: all sums are 0 (or NaN, which stays)
      float acc = 0.f, L = 0.f;
#pragma unroll
      for (int tm = 0; tm < kWarps; ++tm) {
        const float* src = red + (tm * C::ROWS + row) * C::RED;
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
    if (w.last() || !__syncthreads_and(ok)) return;
    fence_proxy_async_smem();
    __syncthreads();  // the next part's loads and queries take the merge's place
  }
}

// ------------------------------------------------------------------ shared runs
// One CTA per (work item, KV head), for all of its up to 64 rows (members x heads).
namespace {

template <int D>
struct Fp8SharedCfg {
  static constexpr int SLOT = Fp8Ring<D>::STAGE;
  static constexpr int ROWS = 2 * kWarps * 8;  // of a CTA
  static constexpr int RED = D + 4;            // merge rows: o[D], m, l
  // Four CTAs an SM with 8 stages and the queries of 16 rows in shared memory: 115 us for 119 on the 32 long sequences,
  // 55 for 49 on the 64 short ones.
  static constexpr int CTAS = 3;     // per SM
  static constexpr int SLOTS = 16;   // stages of the teams' rings
  static_assert(SLOTS <= kFp8Slots, "barriers");
  static constexpr int BUF = SLOTS * SLOT > ROWS * RED * 4 ? SLOTS * SLOT : ROWS * RED * 4;
  static constexpr int SMEM = BUF + kMembers * (D / 2) * 8;  // and the members' angles
};

// What the CTA's warps share of an item.
struct Fp8Item {
  int rec[kItemInts];
  int delta[kMembers], ok[kMembers];  // rotation offset of each member; it passed its checks
  Fp8Bars bars;
};

}  // namespace

// The item's `rows` rows by teams of RT warps with NT tiles each.
template <int D, int NT, int HL, bool LAZY>
__device__ __forceinline__ void shared_fp8_rows(const SharedDecodeArgs& a, const uint8_t* k_pool, const uint8_t* v_pool,
                                                Fp8Item& it, uint8_t* smem, float2* cs_tab, int kvh, int rows, int RT) {
  using C = Fp8SharedCfg<D>;
  constexpr int HALF = D / 2, TILE = Fp8Rows<NT, HL>::ALL;
  const int TEAMS = kWarps / RT, R = C::SLOTS / TEAMS;  // a power of two
  const int AHEAD = RT == 1 ? R - 1 : R - 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / RT, rt = warp & (RT - 1);
  const int src = it.rec[0], b0 = it.rec[1], nblk = it.rec[2], last_nv = it.rec[3];

  // ------------------------------------------------------------ first loads
  const int per_team = (nblk + TEAMS - 1) / TEAMS;
  const int kb0 = team * per_team;
  const int nk = max(0, min(nblk, kb0 + per_team) - kb0);  // blocks of the team
  const size_t head = (size_t)kvh * Fp8Geom<D>::REC;
  const Fp8Ring<D> ring{k_pool + head, v_pool + head, (uint32_t)a.Hkv * Fp8Geom<D>::REC, smem + team * R * C::SLOT, &it.bars, team * R};
  const uint32_t* wrow = a.words + (size_t)src * a.max_blocks + b0 + kb0;
  const uint32_t id_mask = (1u << a.id_bits) - 1u;
  const int* ids = it.rec + 8 + 4 * kMembers;  // the record's block ids
  uint32_t w_nxt = 0u;
  int c_phys = 0, c_nv = 0;  // a chunk of 32 blocks in the lanes: id, valid slots
  auto load_words = [&](int kc) {
    if (kc + lane < nk) w_nxt = wrow[kc + lane];
  };
  // Chunk kc of the team's words (w_nxt), by every warp of the team alike. The block word decides; where
  // the record names the block too the two must agree.
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
    c_phys = phys;
    c_nv = nv;
  };
  load_words(0);
  // What the queries need: loads that nothing waits for yet, so that all of the prologue's share one latency
  // behind the record's. A member's seq, first block and slot, checked:
  const int nmem = it.rec[4], me = threadIdx.x;
  bool good = false;
  uint32_t mem_word = 0u, src_word = 0u;
  int mem_pos = 0;
  if (me < nmem) {
    const int seq = it.rec[8 + 4 * me], bm = it.rec[8 + 4 * me + 1], slot = it.rec[8 + 4 * me + 2];
    good = seq >= 0 && seq < a.B && bm >= 0 && bm <= a.max_blocks - nblk && slot >= 0 && slot < a.num_slots;
    if (good) {
      mem_word = a.words[(size_t)seq * a.max_blocks + bm];
      src_word = a.words[(size_t)src * a.max_blocks + b0];
      mem_pos = a.q_pos[seq];
    }
  }
  static_assert(kThreads % HALF == 0, "a thread's angles are one frequency's");
  const float2 rate = a.rope[threadIdx.x % HALF];
  const __nv_bfloat16* qrow[NT];
  int mem[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rt * TILE + (HL == 1 ? lane >> 3 : 8 * nt + (lane >> 2)), rc = r < rows ? r : 0;
    mem[nt] = rc / a.G;
    const int seq = it.rec[8 + 4 * mem[nt]];
    qrow[nt] = static_cast<const __nv_bfloat16*>(a.q) +
               ((seq >= 0 && seq < a.B ? (size_t)seq * a.Hq + (rc - mem[nt] * a.G) : 0) + (size_t)kvh * a.G) * D;
  }
  auto row = [&](int nt) { return qrow[nt]; };
  const Fp8RawRows<D, NT> raw(row, lane);
  auto fill = [&](int j) {  // block j's stage is loaded, by the warp whose turn it is
    if ((j & 31) == 0 && j < nk) {
      describe(j);
      load_words(j + 32);
    }
    if (j < nk && (j & (RT - 1)) == rt) {
      const int slot = j & (R - 1);
      if (RT > 1 && j >= R && !ring.wait_empty(slot, (j / R + 1) & 1, a.status)) return false;
      const int ph = __shfl_sync(0xffffffffu, c_phys, j & 31), nv = __shfl_sync(0xffffffffu, c_nv, j & 31);
      if (lane == 0) ring.fill(slot, ph, nv);
    }
    return true;
  };
  bool ok = true;
  if (kb0 + min(AHEAD, nk) <= LAZY_PLAN_ITEM_BLOCK_IDS) {  // straight from the record, which names them
    for (int j = rt; j < min(AHEAD, nk); j += RT)
      if (lane == 0) {
        const int id = ids[kb0 + j];
        ring.fill(j, id >= 0 && id < a.num_pool_blocks ? id : 0, 0);
      }
    describe(0);
    load_words(32);
    __syncwarp();
    if (lane < AHEAD && (lane & (RT - 1)) == rt) it.bars.info[team * R + lane] = c_nv;  // seen behind the barriers below
  } else {
    for (int j = 0; j < AHEAD; ++j) ok &= fill(j);
  }

  // ------------------------------------------------------------ members and queries
  if (me < nmem) {
    const BlockInfo mi = decode_word(mem_word, it.rec[8 + 4 * me + 1], a.id_bits);
    good = good && mi.phys == decode_word(src_word, b0, a.id_bits).phys;
    if (!good) raise_status(a.status, LAZY_DEV_LAYOUT);
    it.ok[me] = good;
    it.delta[me] = !good ? 0 : (LAZY ? mem_pos - mi.p : mem_pos);
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nmem * HALF; idx += kThreads) cs_tab[idx] = rope_cs(rate, it.delta[idx / HALF], a.status);
  bool live[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) live[nt] = rt * TILE + (HL == 1 ? lane >> 3 : 8 * nt + (lane >> 2)) < rows && it.ok[mem[nt]];
  Fp8Query<D, NT, HL> q;
  float mul[NT];
  fp8_scale_rows<D, NT, HL>(q, mul, raw, live, a.scale_log2, lane);
  __syncthreads();
  fp8_build_query<D, NT, HL>(mul, row, lane, [&](int nt) { return cs_tab + mem[nt] * HALF; },
                             [&](int nt, int k, int h, uint32_t x) { q.set(nt, k, h, x); });

  // ------------------------------------------------------------ main loop
  Fp8State<D, NT, HL> st;
  fp8_init(st);
  for (int i = 0; i < nk; ++i) {
    const int slot = i & (R - 1);
    ok = ok && fill(i + AHEAD) && ring.wait_full(slot, i / R & 1, a.status);
    if (!ok) {
      ring.drain(i, min(nk, i + AHEAD + 1), R, a.status);
      break;
    }
    const int nv = it.bars.info[team * R + slot];
    if (nv > 0) fp8_attend<D, NT, HL>(ring.base + slot * C::SLOT, nv, q, st, lane);
    __syncwarp();
    if (RT > 1 && lane == 0) ring.release(slot);
  }
  fp8_finish(st);
  __syncthreads();  // every team is done with its ring: the merge takes its place

  // ------------------------------------------------------------ partials
  float* red = reinterpret_cast<float*>(smem);
  fp8_store_partial(st, red + warp * TILE * C::RED, C::RED, lane);
  __syncthreads();
  constexpr int PER = D / 32;
  for (int x = warp; x < rows; x += kWarps) {
    const int m = x / a.G, h = x - m * a.G;
    const int slot = it.rec[8 + 4 * m + 2];
    if (slot < 0 || slot >= a.num_slots) continue;
    float M = -INFINITY, acc[PER], L = 0.f;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = 0.f;
    if (it.ok[m]) {  // a member that failed its checks leaves an empty partial
      for (int tm = 0; tm < TEAMS; ++tm) M = fmaxf(M, red[(tm * RT * TILE + x) * C::RED + D]);
      const float Mr = M == -INFINITY ? 0.f : M;
      for (int tm = 0; tm < TEAMS; ++tm) {
        const float* row = red + (tm * RT * TILE + x) * C::RED;
        const float w = fast_ex2(row[D] - Mr);
        L += w * row[D + 1];
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] += w * row[lane + 32 * c];
      }
      if (L != 0.f) M = Mr;  // all scores NaN: not an empty slot, which the combine would pass over
    }
    const size_t pidx = (size_t)slot * a.Hq + (size_t)kvh * a.G + h;
#pragma unroll
    for (int c = 0; c < PER; ++c) a.ws_o[pidx * D + lane + 32 * c] = acc[c];
    if (lane == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * pidx) = make_float2(M, L);
  }
}

template <int D, bool LAZY>
__global__ void __launch_bounds__(kThreads, Fp8SharedCfg<D>::CTAS) decode_shared_fp8_block_kernel(const SharedDecodeArgs a, const uint8_t* k_pool,
                                                                              const uint8_t* v_pool) {
  using C = Fp8SharedCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];            // the teams' rings, then the merge area
  float2* cs_tab = reinterpret_cast<float2*>(smem + C::BUF);  // [members][D / 2]
  __shared__ __align__(16) Fp8Item it;
  wait_for_launch_before();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv, item = blockIdx.x / a.Hkv;
  if (threadIdx.x < kItemInts / 4)
    reinterpret_cast<int4*>(it.rec)[threadIdx.x] =
        reinterpret_cast<const int4*>(a.items)[(size_t)item * (kItemInts / 4) + threadIdx.x];
  __syncthreads();
  const int src = it.rec[0], b0 = it.rec[1], nblk = it.rec[2], last_nv = it.rec[3], nmem = it.rec[4];
  const bool item_ok = src >= 0 && src < a.B && b0 >= 0 && nblk >= 1 && nblk <= a.max_blocks - b0 &&
                       last_nv >= 1 && last_nv <= kBlock && nmem >= 1 && nmem <= kMembers && nmem * a.G <= C::ROWS && nblk <= kFp8MaxRun;
  if (!item_ok) {  // uniform over the CTA: nothing is loaded or written
    if (threadIdx.x == 0) raise_status(a.status, LAZY_DEV_LAYOUT);
    return;
  }
  const int n = nmem * a.G, RT = n <= 16 ? 1 : (n <= 32 ? 2 : 4);
  if (threadIdx.x < C::SLOTS) {
    mbar_init(&it.bars.full[threadIdx.x], 1);
    mbar_init(&it.bars.empty[threadIdx.x], RT);
    fence_barrier_init();
  }
  __syncthreads();
  if (n <= 8) shared_fp8_rows<D, 1, 2, LAZY>(a, k_pool, v_pool, it, smem, cs_tab, kvh, n, 1);
  else shared_fp8_rows<D, 2, 2, LAZY>(a, k_pool, v_pool, it, smem, cs_tab, kvh, n, RT);
}

// ------------------------------------------------------------------ launchers

// 32 rows a warp read and convert a block once for twice the rows, but their queries take longer to build and to
// merge; worth it for long batches, going by the table's width: 48 sequences of 256 to 131072 tokens, 32 heads on
// one, 230 us, as two units of 16 rows 281; 45 of 40000 to 79000 195 and 207; but 53 of 1665 to 3331 34 and 26,
// one of 8000 25 and 13, one of 20 22 and 10. (64 rows as two warps with 32 each: 258 us where units of 32 take 184,
// 80 sequences of 10000 to 20000 tokens, 64 heads on one.)
constexpr int64_t kWideBlocks = 1 << 16;

// Pieces of at least 16 blocks; 32 for 32 rows (128 sequences of 1000 tokens 27 us, with 16 31). With 32 for the
// others one sequence of 16384 tokens, 32 heads on 2, takes 14.8 us, with 16 12.4 and with 8 13.2; two of 1475, 32 on
// 8, 13.1, 10.7 and 10.4; eight of 2048, 64 on 8, 15.9, 16.1 and 25.5 (more parts than a warp of the join merges).
UnitPlan plan_decode_fp8_block(int B, int G, int Hkv, int max_blocks, int num_splits, int sms) {
  const int most = (int64_t)B * max_blocks * Hkv >= kWideBlocks ? 32 : 16;
  int rows = 4;
  while (rows < G && rows < most) rows *= 2;
  const int per_sm = rows <= 8 ? Fp8Cfg<128, 1, 1>::CTAS : (rows == 16 ? Fp8Cfg<128, 2, 2>::CTAS : Fp8Cfg<128, 4, 2>::CTAS);
  return plan_units(B, rows, Hkv * ((G + rows - 1) / rows), max_blocks, num_splits, (int64_t)sms * per_sm, rows == 32 ? 5 : 4,
                    kWarps * kFp8MaxRun);
}

template <int D, int NT, int HL, bool LAZY, bool LONG>
static cudaError_t launch_decode_t(const UnitDecodeArgs& a, cudaStream_t st) {
  using C = Fp8Cfg<D, NT, HL>;
  constexpr int SMEM = C::BUF + kWarps * ((D / 2) * 8 + Fp8Query<D, NT, HL>::BYTES);
  cudaError_t e = set_smem_once<decode_fp8_block_kernel<D, NT, HL, LAZY, LONG>>(SMEM);
  if (e != cudaSuccess) return e;
  return launch_behind(decode_fp8_block_kernel<D, NT, HL, LAZY, LONG>, (unsigned)a.plan.ctas, kThreads, SMEM, st, a);
}

template <int D, bool LAZY, bool LONG>
static cudaError_t launch_decode_l(const UnitDecodeArgs& a, cudaStream_t st) {
  switch (a.plan.rows) {
    case 4: return launch_decode_t<D, 1, 1, LAZY, LONG>(a, st);
    case 8: return launch_decode_t<D, 1, 2, LAZY, LONG>(a, st);
    case 16: return launch_decode_t<D, 2, 2, LAZY, LONG>(a, st);
    default: return launch_decode_t<D, 4, 2, LAZY, LONG>(a, st);
  }
}

template <int D, bool LAZY>
static cudaError_t launch_decode_d(const UnitDecodeArgs& a, cudaStream_t st) {
  return longest_part(a.plan, a.B, a.max_blocks) > kWarps * kFp8Keep ? launch_decode_l<D, LAZY, true>(a, st) : launch_decode_l<D, LAZY, false>(a, st);
}

cudaError_t launch_decode_fp8_block(const UnitDecodeArgs& a, bool lazy, cudaStream_t st) {
  if (a.D == 128) return lazy ? launch_decode_d<128, true>(a, st) : launch_decode_d<128, false>(a, st);
  return lazy ? launch_decode_d<64, true>(a, st) : launch_decode_d<64, false>(a, st);
}

template <int D, bool LAZY>
static cudaError_t launch_shared_t(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, cudaStream_t st) {
  constexpr int SMEM = Fp8SharedCfg<D>::SMEM;
  cudaError_t e = set_smem_once<decode_shared_fp8_block_kernel<D, LAZY>>(SMEM);
  if (e != cudaSuccess) return e;
  return launch_behind(decode_shared_fp8_block_kernel<D, LAZY>, (unsigned)(a.num_items * a.Hkv), kThreads, SMEM, st, a,
                       static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool));
}

cudaError_t launch_decode_shared_fp8_block(const SharedDecodeArgs& a, const void* k_pool, const void* v_pool, bool lazy,
                                           cudaStream_t st) {
  if (a.num_items == 0) return cudaSuccess;
  if (a.D == 128)
    return lazy ? launch_shared_t<128, true>(a, k_pool, v_pool, st) : launch_shared_t<128, false>(a, k_pool, v_pool, st);
  return lazy ? launch_shared_t<64, true>(a, k_pool, v_pool, st) : launch_shared_t<64, false>(a, k_pool, v_pool, st);
}

}  // namespace lazy
