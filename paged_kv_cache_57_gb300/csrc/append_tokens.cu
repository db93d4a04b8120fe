// append_tokens.cu -- block words, lengths and slots for the new tokens of a batch's sequences
// (lazy_attn_append_tokens).
//
// A sequence's own tokens (from tail_start on) lie in whole blocks behind its cited documents'
// blocks: token i of them is row i % 16 of block b0 + i / 16. So all that couples the sequences
// is two sums over the batch, of rows and of blocks taken from the free list. One CTA forms them
// (append_scan_kernel); the rows, each found by a search in the rows' sums, are written by the
// same CTA where they are few, else by a second launch over the device (append_rows_kernel),
// started behind the first one's back. Nothing but latency bounds the small case: the loads of
// four numbers a sequence, three barriers, a search and a store; the large one its stores.
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace lazy {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowsPerThread = 4;  // a 16-byte store of slots and one of positions
constexpr int kOneDoc = 1 << 30;   // a document without an end

__device__ __forceinline__ int blocks_for(int tokens) { return (int)(((unsigned)tokens + kBlock - 1) / kBlock); }

// What a sequence asks for.
struct Want {
  int rows, blocks;  // new tokens; blocks from the free list
  int b0;            // block of its own first token
  bool ok;           // the tokens can be added, room in the free list and the rows permitting
};

__device__ __forceinline__ Want want_of(const AppendArgs& a, int s, int& len, int& pos) {
  Want w{0, 0, 0, false};
  const int n = a.new_lens[s], start = a.tail_start[s];
  len = a.seq_lens[s];
  pos = a.pos[s];
  if (n <= 0) {
    if (n < 0) raise_status(a.status, LAZY_DEV_BAD_LEN);
    return w;
  }
  w.rows = n;
  if (len < 0 || len > kBlock * a.max_blocks) {
    raise_status(a.status, LAZY_DEV_BAD_LEN);
    return w;
  }
  const int64_t tail64 = (int64_t)pos - start, end = tail64 + n;
  // its own tokens begin a block, behind other documents or from the sequence's first block on
  bool good = pos >= 0 && tail64 >= 0 && tail64 <= len && (tail64 == 0 || ((len - tail64) & (kBlock - 1)) == 0) && (int64_t)pos + n <= INT_MAX;
  if (good) {
    const int tail = (int)tail64;
    w.b0 = blocks_for(len) - blocks_for(tail);
    const int64_t last = (end + kBlock - 1) / kBlock;
    good = w.b0 + last <= a.max_blocks;
    w.blocks = (int)(last - blocks_for(tail));
    if (good && w.blocks > 0) {  // the offsets of the new blocks must fit their field
      int64_t lo = (int64_t)kBlock * w.b0 - start, hi = lo;
      if (!a.key_positions) {
        const int first = kBlock * blocks_for(tail), fin = kBlock * (int)(last - 1);
        if (first / a.doc_tokens == fin / a.doc_tokens) {
          hi = lo + fin % a.doc_tokens;
          lo += first % a.doc_tokens;
        } else {
          hi = lo + a.doc_tokens - kBlock;
        }
      }
      const int64_t most = (1ll << (31 - a.id_bits)) - 1;
      good = lo >= -most - 1 && hi <= most;
    }
  }
  if (!good) {
    raise_status(a.status, LAZY_DEV_LAYOUT);
    w.blocks = 0;
  }
  w.ok = good;
  return w;
}

// The inclusive sums of x and y over the CTA; `part` is shared memory of 2 x 32 numbers.
__device__ __forceinline__ void scan2(int64_t& x, int64_t& y, int64_t (&part)[2][32], int64_t& all_x, int64_t& all_y) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  if (lane == 31) part[0][warp] = x, part[1][warp] = y;
  __syncthreads();
  int64_t px = lane < warps ? part[0][lane] : 0, py = lane < warps ? part[1][lane] : 0;  // every warp for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, px, o), v = __shfl_up_sync(0xffffffffu, py, o);
    if (lane >= o) px += u, py += v;
  }
  all_x = __shfl_sync(0xffffffffu, px, 31);
  all_y = __shfl_sync(0xffffffffu, py, 31);
  const int64_t bx = __shfl_sync(0xffffffffu, px, warp > 0 ? warp - 1 : 0), by = __shfl_sync(0xffffffffu, py, warp > 0 ? warp - 1 : 0);
  if (warp > 0) x += bx, y += by;
}

// Rows r .. r + n - 1 of the batch: slots and positions, and the words of the blocks that begin there.
// `cu` are the rows' sums, wherever they are.
template <int N>
__device__ __forceinline__ void write_rows(const AppendArgs& a, const int32_t* cu, int r, int n) {
  int lo = 0, hi = a.B;  // the last sequence that begins at or before r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  const int total = cu[a.B];
  int slot[N], local[N];
  int s = lo, begin = 0, end = -1, start = 0, tail = 0, b0 = 0, first = 0;
  bool ok = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    slot[i] = -1;
    local[i] = 0;
    const int row = r + i;
    if (i >= n || row >= total) continue;
    while (end < 0 || row >= end) {  // the row's sequence
      if (end >= 0) ++s;
      begin = cu[s];
      end = cu[s + 1];
      if (row >= end) continue;
      const int q = a.q_start[s], p = a.pos_out[s];
      start = a.tail_start[s];
      ok = p != q;
      tail = q - start;
      b0 = (a.seq_lens_out[s] - (p - start)) / kBlock;
      first = a.block_indptr[s];
    }
    if (!ok) continue;
    const int at = tail + row - begin, j = at / kBlock, have = blocks_for(tail);
    uint32_t* word = a.words + (size_t)s * a.max_blocks + b0 + j;
    const uint32_t id_mask = (1u << a.id_bits) - 1u;
    const int phys = j < have ? (int)(*word & id_mask) : a.free_blocks[first + j - have];
    const bool good = phys >= 0 && phys < a.num_pool_blocks;
    if (!good) raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
    if (at % kBlock == 0) {
      const int doc = start + (a.key_positions ? kBlock * j : at / a.doc_tokens * a.doc_tokens);
      *word = (uint32_t)(kBlock * (b0 + j) - doc) << a.id_bits | (good ? (uint32_t)phys : id_mask);
    }
    if (good) slot[i] = phys * kBlock + at % kBlock;
    local[i] = at % a.doc_tokens;
  }
  if (N == 4 && n == 4 && a.vec) {
    *reinterpret_cast<int4*>(a.slots + r) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    if (a.local_pos) *reinterpret_cast<int4*>(a.local_pos + r) = make_int4(local[0], local[1], local[2], local[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) {
      a.slots[r + i] = slot[i];
      if (a.local_pos) a.local_pos[r + i] = local[i];
    }
}

}  // namespace

// One CTA. ROWS: it writes the rows too.
template <bool ROWS>
__global__ void append_scan_kernel(const AppendArgs a) {
  extern __shared__ int32_t cu_s[];  // ROWS: the rows' sums
  __shared__ int64_t part[2][32];
  __shared__ int64_t given_s;  // blocks before the first sequence that goes without
  wait_for_launch_before();
  if (!ROWS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int first_raw = a.first_free ? *a.first_free : 0;
  const bool bad_first = first_raw < 0 || first_raw > a.num_free;
  const int first = bad_first ? a.num_free : first_raw;  // nothing is taken then
  if (threadIdx.x == 0) {
    given_s = INT64_MAX;
    if (bad_first) raise_status(a.status, LAZY_DEV_LAYOUT);
  }
  int64_t rows = 0, blocks = 0;  // of the sequences before the chunk
  for (int c = 0; c < a.B || c == 0; c += blockDim.x) {
    const int s = c + threadIdx.x;
    int len = 0, pos = 0;
    Want w{0, 0, 0, false};
    if (s < a.B) w = want_of(a, s, len, pos);
    int64_t r = w.rows, b = w.blocks, all_r, all_b;
    scan2(r, b, part, all_r, all_b);
    r += rows;
    b += blocks;
    const bool fits_rows = r <= a.num_rows, fits_blocks = w.blocks == 0 || first + b <= a.num_free;
    const bool ok = w.ok && fits_rows && fits_blocks;
    if (w.ok && !ok) {
      raise_status(a.status, fits_rows ? LAZY_DEV_NO_BLOCKS : LAZY_DEV_BAD_LEN);
      if (w.blocks > 0) atomicMin(reinterpret_cast<unsigned long long*>(&given_s), (unsigned long long)(b - w.blocks));
    }
    __syncthreads();
    const int64_t given = given_s;
    if (s < a.B) {
      // (every value of the sequence that an output may take the place of has been read)
      a.seq_lens_out[s] = ok ? kBlock * w.b0 + (pos - a.tail_start[s]) + w.rows : len;
      a.pos_out[s] = ok ? pos + w.rows : pos;
      a.q_start[s] = pos;
      const int cu = (int)(r < INT_MAX ? r : INT_MAX);
      a.cu_rows[s + 1] = cu;
      if (ROWS) cu_s[s + 1] = cu;
      a.block_indptr[s + 1] = first + (int)(b < given ? b : given);
    }
    if (c == 0 && threadIdx.x == 0) {
      a.cu_rows[0] = 0;
      if (ROWS) cu_s[0] = 0;
      a.block_indptr[0] = first;
    }
    rows += all_r;
    blocks += all_b;
    __syncthreads();  // `part` and given_s are the next chunk's
  }
  if (ROWS)
    for (int r = threadIdx.x; r < a.num_rows; r += blockDim.x) write_rows<1>(a, cu_s, r, 1);
}

__global__ void __launch_bounds__(kRowThreads) append_rows_kernel(const AppendArgs a) {
  const int64_t r = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) * kRowsPerThread;
  wait_for_launch_before();
  if (r < a.num_rows) write_rows<kRowsPerThread>(a, a.cu_rows, (int)r, (int)min((int64_t)kRowsPerThread, a.num_rows - r));
}

cudaError_t launch_append_tokens(AppendArgs a, int* launches, cudaStream_t st) {
  constexpr int kMostRows = 4096, kMostSeqs = 8192;  // for one CTA; its sums fit the default shared memory
  if (a.doc_tokens == 0) a.doc_tokens = kOneDoc;
  const bool one = a.num_rows <= kMostRows && a.B <= kMostSeqs;
  const int work = one && a.num_rows > a.B ? a.num_rows : a.B;
  const unsigned threads = work >= 1024 ? 1024 : (work <= 32 ? 32 : (work + 31) / 32 * 32);
  *launches = 1;
  if (one) return launch_behind(append_scan_kernel<true>, 1, threads, (a.B + 1) * sizeof(int32_t), st, a);
  cudaError_t e = launch_behind(append_scan_kernel<false>, 1, threads, 0, st, a);
  if (e != cudaSuccess || a.num_rows == 0) return e;
  *launches = 2;
  const int per = kRowThreads * kRowsPerThread;
  return launch_behind(append_rows_kernel, (unsigned)(((int64_t)a.num_rows + per - 1) / per), kRowThreads, 0, st, a);
}

}  // namespace lazy
