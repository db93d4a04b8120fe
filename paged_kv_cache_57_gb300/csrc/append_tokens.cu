// append_tokens.cu -- block words, lengths and slots for the new tokens of a batch's sequences
// (lazy_attn_append_tokens).
//
// A sequence's own tokens (from tail_start on) lie in whole blocks behind its cited documents'
// blocks: token i of them is row i % 16 of block b0 + i / 16. So all that couples the sequences
// is two sums over the batch, of rows and of blocks taken from the free list. One CTA forms them
// (append_scan_kernel), a thread a sequence, and where there is little to write, writes the rows too.
// Else a second launch does, started behind the first one's back: a thread a row (append_row_kernel), or, of many,
// warps of 256 rows (append_rows_kernel), that find their sequence by a search in the rows' sums. Latency bounds the
// small cases (64 sequences of a token 3.4 us a call in a graph, 7 a call from Python). 2.6 million rows take 11.0 us
// for 21 MB, of which the scan is a third; the rows' kernel is at no limit of the machine (issue slots 63%): its
// search and its sequence's numbers are dependent loads in front of a warp's 256 rows.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace lazy {

namespace {

constexpr int kRowThreads = 256;
// A thread a row up to what is resident at once: 6000 rows of 1021 sequences 8.5 us, in warps of 256 rows
// 15.9; 2.6 million rows of 48 20.4 and 11.0.
constexpr int kFewRows = 152 * 2048;
constexpr int kRowsPerWarp = 256;  // 2.6 million rows of 48 sequences 11.2 us, with 128 and 512 11.4, 1024 12.9
constexpr int kOwnRows = 8;        // rows that a sequence's thread writes by itself
constexpr int kOneDoc = 1 << 30;   // a document without an end

__device__ __forceinline__ int blocks_for(int tokens) { return (int)(((unsigned)tokens + kBlock - 1) / kBlock); }

// What a sequence asks for.
struct Want {
  int rows, blocks;  // new tokens; blocks from the free list
  int b0;            // block of its own first token
  int start;         // tail_start, which may be the place of pos_out
  bool ok;           // the tokens can be added, room in the free list and the rows permitting
};

__device__ __forceinline__ Want want_of(const AppendArgs& a, int s, int& len, int& pos) {
  const int n = a.new_lens[s], start = a.tail_start[s];
  Want w{0, 0, 0, start, false};
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

// Whether the n ids from free_blocks[at] on are blocks of the pool, for the lanes with `mine`. All lanes call it.
__device__ __forceinline__ bool ids_good(const AppendArgs& a, bool mine, int at, int n) {
  const int lane = threadIdx.x & 31;
  bool good = true;
  for (uint32_t left = __ballot_sync(0xffffffffu, mine); left; left &= left - 1) {
    const int l = __ffs(left) - 1, from = __shfl_sync(0xffffffffu, at, l), count = __shfl_sync(0xffffffffu, n, l);
    bool bad = false;
    for (int j = lane; j < count; j += 32) {
      const int id = a.free_blocks[from + j];
      bad |= id < 0 || id >= a.num_pool_blocks;
    }
    if (__any_sync(0xffffffffu, bad) && lane == l) good = false;
  }
  return good;
}

// a / d for 0 <= a < 2^31 by a multiplication (a.doc_mul, a.doc_shift: the launch fills them): division by invariant
// integers after Granlund and Montgomery (1994).
__device__ __forceinline__ int doc_of(const AppendArgs& a, int at) {
  return (int)((__umulhi((unsigned)at, a.doc_mul) + (unsigned)at) >> a.doc_shift);
}

// A sequence with rows, as they need it.
struct SeqRows {
  int shift;  // a row's place among the sequence's own tokens is row + shift; INT_MIN: its tokens were not added
  int start, b0;
  int first;  // free_blocks[first + j] is block j of its own, for j >= have
  int have;   // blocks of its own from earlier calls
};

__device__ __forceinline__ SeqRows seq_rows(const AppendArgs& a, int s, int begin) {
  const int q = a.q_start[s], p = a.pos_out[s], len = a.seq_lens_out[s], start = a.tail_start[s], first = a.block_indptr[s];
  const int tail = q - start, have = blocks_for(tail);
  return SeqRows{p != q ? tail - begin : INT_MIN, start, (len - (p - start)) / kBlock, first - have, have};
}

__device__ __forceinline__ int checked(const AppendArgs& a, int phys) {
  if (phys >= 0 && phys < a.num_pool_blocks) return phys;
  raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
  return -1;
}

// The word of the sequence's own block j with physical id `phys` (-1: bad).
__device__ __forceinline__ void put_word(const AppendArgs& a, const SeqRows& q, int s, int j, int phys) {
  const int doc = q.start + (a.key_positions ? kBlock * j : doc_of(a, kBlock * j) * a.doc_tokens);
  a.words[(size_t)s * a.max_blocks + q.b0 + j] =
      (uint32_t)(kBlock * (q.b0 + j) - doc) << a.id_bits | (phys >= 0 ? (uint32_t)phys : (1u << a.id_bits) - 1u);
}

// Physical id of the sequence's own block j (-1: bad); `begins`: the call takes it, and this row, its first,
// writes its word.
__device__ __forceinline__ int own_block(const AppendArgs& a, const SeqRows& q, int s, int j, bool begins) {
  if (j < q.have) return checked(a, (int)(a.words[(size_t)s * a.max_blocks + q.b0 + j] & ((1u << a.id_bits) - 1u)));
  const int phys = checked(a, a.free_blocks[q.first + j]);
  if (begins) put_word(a, q, s, j, phys);
  return phys;
}

__device__ __forceinline__ int2 one_row(const AppendArgs& a, const SeqRows& q, int s, int row) {
  if (q.shift == INT_MIN) return make_int2(-1, 0);
  const int at = row + q.shift, in = at % kBlock, phys = own_block(a, q, s, at / kBlock, in == 0);
  return make_int2(phys >= 0 ? phys * kBlock + in : -1, at - doc_of(a, at) * a.doc_tokens);
}

__device__ __forceinline__ void put_row(const AppendArgs& a, int r, int2 x) {
  a.slots[r] = x.x;
  if (a.local_pos) a.local_pos[r] = x.y;
}

// The rows of a warp's sequences, each lane's own: s with the rows begin .. end - 1 (none: end <= begin). All
// lanes call it. Few rows are their lane's, more are shared out.
__device__ __forceinline__ void write_seqs(const AppendArgs& a, const SeqRows& q, int s, int begin, int end) {
  const int n = end - begin, lane = threadIdx.x & 31;
  if (n > 0 && n <= kOwnRows) {  // in one block of its own or two, of one document each
    const bool ok = q.shift != INT_MIN;
    const int at = ok ? begin + q.shift : 0, in = at % kBlock, j = at / kBlock;
    int p0 = -1, p1 = -1;
    if (ok) {
      if (in + n > kBlock) p1 = own_block(a, q, s, j + 1, true);
      p0 = own_block(a, q, s, j, in == 0);
    }
    int local = at - doc_of(a, at) * a.doc_tokens;
    for (int i = 0; i < n; ++i) {
      const int ph = in + i < kBlock ? p0 : p1;
      put_row(a, begin + i, make_int2(ph >= 0 ? ph * kBlock + (in + i) % kBlock : -1, ok ? local : 0));
      if (++local == a.doc_tokens) local = 0;
    }
  }
  for (uint32_t left = __ballot_sync(0xffffffffu, n > kOwnRows); left; left &= left - 1) {
    const int l = __ffs(left) - 1;
    auto of = [&](int x) { return __shfl_sync(0xffffffffu, x, l); };
    const SeqRows p{of(q.shift), of(q.start), of(q.b0), of(q.first), of(q.have)};
    const int sl = of(s), from = of(begin), to = of(end);
    for (int r = from + lane; r < to; r += 32) put_row(a, r, one_row(a, p, sl, r));
  }
}

// The last sequence that begins at or before row r. `cu` are the rows' sums, wherever they are.
__device__ __forceinline__ int seq_of(const int32_t* cu, int B, int r) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

// One CTA. ROWS: it writes the rows too.
template <bool ROWS>
__global__ void append_scan_kernel(const AppendArgs a) {
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
    Want w{0, 0, 0, 0, false};
    if (s < a.B) w = want_of(a, s, len, pos);
    int64_t r = w.rows, b = w.blocks, all_r, all_b;
    scan2(r, b, part, all_r, all_b);
    r += rows;
    b += blocks;
    const bool fits_rows = r <= a.num_rows, fits_blocks = w.blocks == 0 || first + b <= a.num_free;
    bool ok = w.ok && fits_rows && fits_blocks;
    if (w.ok && !ok) {
      raise_status(a.status, fits_rows ? LAZY_DEV_NO_BLOCKS : LAZY_DEV_BAD_LEN);
      if (w.blocks > 0) atomicMin(reinterpret_cast<unsigned long long*>(&given_s), (unsigned long long)(b - w.blocks));
    }
    // A word marks a bad id by the greatest of its field. Where that is a block of the pool, a sequence
    // that is given a bad id gets no tokens: the next call's would go into that block.
    if (a.num_pool_blocks >> a.id_bits != 0 && !ids_good(a, ok && w.blocks > 0, (int)(first + b - w.blocks), w.blocks)) {
      raise_status(a.status, LAZY_DEV_BAD_BLOCK_ID);
      ok = false;
    }
    __syncthreads();
    const int64_t given = given_s;
    if (s < a.B) {
      // (every value of the sequence that an output may take the place of has been read)
      a.seq_lens_out[s] = ok ? kBlock * w.b0 + (pos - w.start) + w.rows : len;
      a.pos_out[s] = ok ? pos + w.rows : pos;
      a.q_start[s] = pos;
      const int cu = (int)(r < INT_MAX ? r : INT_MAX);
      a.cu_rows[s + 1] = cu;
      a.block_indptr[s + 1] = first + (int)(b < given ? b : given);
    }
    if (c == 0 && threadIdx.x == 0) {
      a.cu_rows[0] = 0;
      a.block_indptr[0] = first;
    }
    if (ROWS) {  // (one chunk)
      const int tail = pos - w.start, have = blocks_for(tail);
      const int begin = (int)min(r - w.rows, (int64_t)a.num_rows);  // the rows' sum may leave 32 bits
      const SeqRows q{ok ? tail - begin : INT_MIN, w.start, w.b0, first + (int)(b - w.blocks) - have, have};
      write_seqs(a, q, s, begin, s < a.B ? (int)min(r, (int64_t)a.num_rows) : begin);
    }
    rows += all_r;
    blocks += all_b;
    __syncthreads();  // `part` and given_s are the next chunk's
  }
  if (ROWS)
    for (int r = (int)min(rows, (int64_t)a.num_rows) + threadIdx.x; r < a.num_rows; r += blockDim.x) put_row(a, r, make_int2(-1, 0));
}

// A row a thread.
__global__ void __launch_bounds__(kRowThreads) append_row_kernel(const AppendArgs a) {
  const int r = blockIdx.x * kRowThreads + threadIdx.x;
  wait_for_launch_before();
  if (r >= a.num_rows) return;
  int2 x = make_int2(-1, 0);
  if (r < a.cu_rows[a.B]) {
    const int s = seq_of(a.cu_rows, a.B, r);
    x = one_row(a, seq_rows(a, s, a.cu_rows[s]), s, r);
  }
  put_row(a, r, x);
}

// A warp takes kRowsPerWarp rows in a row, four a lane at a time.
__global__ void __launch_bounds__(kRowThreads) append_rows_kernel(const AppendArgs a) {
  const int64_t warp0 = ((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kRowsPerWarp;
  wait_for_launch_before();
  int64_t r = warp0 + 4 * (threadIdx.x & 31);
  if (r >= a.num_rows) return;
  const int total = a.cu_rows[a.B];
  int s = -1, end = INT_MIN;
  SeqRows q{INT_MIN, 0, 0, 0, 0};
  if (r < total) {
    s = seq_of(a.cu_rows, a.B, (int)r);
    end = a.cu_rows[s + 1];
    q = seq_rows(a, s, a.cu_rows[s]);
  }
  auto reach = [&](int row) {  // the sequence of a later row
    if (row < end) return;
    int begin;
    do {
      ++s;
      begin = a.cu_rows[s];
      end = a.cu_rows[s + 1];
    } while (row >= end);
    q = seq_rows(a, s, begin);
  };
#pragma unroll 1
  for (int i = 0; i < kRowsPerWarp / 128 && r < a.num_rows; ++i, r += 128) {
    const int row = (int)r, n = (int)min((int64_t)4, a.num_rows - r);
    int slot[4], local[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) slot[k] = -1, local[k] = 0;
    if (row < total) reach(row);
    if (row + 3 < end && q.shift != INT_MIN) {  // one sequence's: in one of its blocks or two, of one document each
      const int at = row + q.shift, in = at % kBlock, j = at / kBlock;
      const int p0 = own_block(a, q, s, j, in == 0), p1 = in > kBlock - 4 ? own_block(a, q, s, j + 1, true) : -1;
      const int l0 = at - doc_of(a, at) * a.doc_tokens;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int ph = in + k < kBlock ? p0 : p1;
        slot[k] = ph >= 0 ? ph * kBlock + (in + k) % kBlock : -1;
        local[k] = l0 + k < a.doc_tokens ? l0 + k : l0 + k - a.doc_tokens;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n && row + k < total) {
          reach(row + k);
          const int2 x = one_row(a, q, s, row + k);
          slot[k] = x.x;
          local[k] = x.y;
        }
    }
    if (n == 4 && a.vec) {
      *reinterpret_cast<int4*>(a.slots + r) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.local_pos) *reinterpret_cast<int4*>(a.local_pos + r) = make_int4(local[0], local[1], local[2], local[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) {
          a.slots[r + k] = slot[k];
          if (a.local_pos) a.local_pos[r + k] = local[k];
        }
    }
  }
}

cudaError_t launch_append_tokens(AppendArgs a, int* launches, cudaStream_t st) {
  if (a.doc_tokens == 0) a.doc_tokens = kOneDoc;
  // at / d = (umulhi(at, mul) + at) >> shift for at < 2^31: shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1
  const uint64_t d = (uint64_t)a.doc_tokens;
  a.doc_shift = 0;
  while ((1ull << a.doc_shift) < d) ++a.doc_shift;
  a.doc_mul = (uint32_t)(((1ull << 32) * ((1ull << a.doc_shift) - d)) / d + 1);
  // One CTA writes rows at an SM's rate: 1021 sequences of up to 8 took 10.7 us that way, for 8.5; but 64
  // sequences of a token 6.8, with a second launch 8.5.
  const bool one = a.B <= 256 && a.num_rows <= 1024;
  const unsigned threads = a.B >= 1024 ? 1024 : (one && a.num_rows > a.B ? 256 : (a.B <= 32 ? 32 : (a.B + 31) / 32 * 32));
  *launches = 1;
  if (one) return launch_behind(append_scan_kernel<true>, 1, threads, 0, st, a);
  cudaError_t e = launch_behind(append_scan_kernel<false>, 1, threads, 0, st, a);
  if (e != cudaSuccess || a.num_rows == 0) return e;
  *launches = 2;
  if (a.tail_start == a.pos_out) a.tail_start = a.q_start;  // (= pos) was overwritten; q_start has its values
  if (a.num_rows <= kFewRows)
    return launch_behind(append_row_kernel, (unsigned)((a.num_rows + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st, a);
  const int per = kRowThreads / 32 * kRowsPerWarp;
  return launch_behind(append_rows_kernel, (unsigned)(((int64_t)a.num_rows + per - 1) / per), kRowThreads, 0, st, a);
}

}  // namespace lazy
