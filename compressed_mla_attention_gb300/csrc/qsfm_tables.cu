// Block tables and slots of the paged cache from request lengths (sm_103a).
//
// The bookkeeping between two steps of a serving loop: which blocks the
// requests give back and take, and the pool row of every new cache row. With
// the cache rows of request b before and after the step, p_b and r_b, its
// blocks before and after, h_b = ceil(p_b / 128) and n_b = ceil(r_b / 128),
//   G_b = sum_{i<b} g_i                 blocks given back before request b, g_i of
//                                       the columns n_i .. h_i - 1 that hold one,
//   T_b = sum_{i<b} max(0, n_i - h_i)   blocks taken before it,
//   N_b = sum_{i<b} max(0, r_i - p_i)   new rows before it,
// the i-th block taken is the i-th from the top of the stack "free list, then
// the blocks given back in order", so each output element follows from the
// three prefix sums alone and no thread waits for another's write. A column may
// hold no block: -1 where the pool was short or the block lies behind a window and
// is somebody else's by now. So g_i is counted, a warp per request that shrinks.
//
// Every CTA computes the prefix sums over the batch for itself (up to 160 KB of
// shared memory; the lengths come from L2) and takes a share of the output
// elements: a thread has four consecutive new rows at a time, finds the request
// of the first by a binary search in shared memory and stores 16 bytes. Reads
// and writes are of disjoint places: columns below h_b are read, columns from
// h_b on written; free entries below the count are read, entries from it on
// written. Only free_count itself is both, so with more than one CTA its update
// in place is a launch of its own (one CTA, the sums again).
// Bound by latency up to some ten thousand rows (the launch, one round trip for
// the lengths, the scan, the search and one or two round trips for a block id),
// then by the stores. Times inside a graph: 2 requests with one new row each 3.2 us,
// 128 requests 6.1 us, 500 requests with half a million new rows 11.3 us (4 MB of
// slots and positions). Counting what is given back takes 1.1 and 3.8 us of the last
// two (25 of the 500 requests end, 13 thousand columns, read by every CTA).
#include <cuda_runtime.h>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabRows = 4;  // consecutive rows of a thread
// Rows one CTA takes alone: more CTAs read the lengths as often, and an update
// in place costs a second launch.
constexpr int kTabAlone = 4 * kTabThreads * kTabRows;

// Prefix sums; the row counts of absurd lengths stop at the largest int (the
// table has at most 2^30 entries, so the block counts cannot pass it).
struct Sums {
  int rows, taken, given;
};
__device__ __forceinline__ int add_rows(int a, int b) { return int(min(unsigned(a) + unsigned(b), 0x7fffffffu)); }
__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return {add_rows(a.rows, b.rows), a.taken + b.taken, a.given + b.given};
}

// Sums of the threads before this one, and of all: within the warps by
// shuffles, then over the warps' totals, which every warp adds up for itself.
__device__ __forceinline__ Sums scan_before(const Sums& mine, Sums* s_warps, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](Sums v) {  // of this lane and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums w{__shfl_up_sync(0xffffffffu, v.rows, o), __shfl_up_sync(0xffffffffu, v.taken, o),
                   __shfl_up_sync(0xffffffffu, v.given, o)};
      if (lane >= o) v = add(w, v);
    }
    return v;
  };
  auto of_lane = [&](const Sums& v, int from) {
    return Sums{__shfl_sync(0xffffffffu, v.rows, from), __shfl_sync(0xffffffffu, v.taken, from),
                __shfl_sync(0xffffffffu, v.given, from)};
  };
  const Sums in_warp = scan(mine);
  if (lane == 31) s_warps[warp] = in_warp;
  __syncthreads();
  const Sums warps = scan(lane < kTabThreads / 32 ? s_warps[lane] : Sums{0, 0, 0});
  total = of_lane(warps, 31);
  const Sums earlier = of_lane(warps, warp > 0 ? warp - 1 : 0);
  const Sums up{__shfl_up_sync(0xffffffffu, in_warp.rows, 1), __shfl_up_sync(0xffffffffu, in_warp.taken, 1),
                __shfl_up_sync(0xffffffffu, in_warp.given, 1)};
  Sums before{0, 0, 0};
  if (warp > 0) before = earlier;
  if (lane > 0) before = add(before, up);
  return before;
}

// Request of element i of the ranges whose starts are at[0 .. n - 1]
// (at[0] = 0): the last b with at[b] <= i; empty ranges are passed over.
__device__ __forceinline__ int find_request(const int* at, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// update: 0 leaves free_count alone, 1 updates it (and free_count_out), 2 does
// nothing else.
__global__ void __launch_bounds__(kTabThreads, 2) block_table_kernel(const qsfm_block_table_params p, const int update,
                                                                  int* fault) {
  __shared__ Sums s_warps[kTabThreads / 32];
  extern __shared__ int s_dyn[];
  int* s_rows = s_dyn;             // N_b
  int* s_taken = s_dyn + p.batch;  // T_b
  int* s_given = s_taken + p.batch;  // G_b
  int* s_prev = s_given + p.batch;   // p_b
  int* s_need = s_prev + p.batch;    // n_b
  const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x;
  const int cap_rows = p.max_blocks * kBlock;  // rows a table row can hold

  const int per = (p.batch + kTabThreads - 1) / kTabThreads;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  const int stack = *p.free_count;  // in flight with the lengths
  bool wide = false, shrinks = false;
  for (int b = b0; b < b1; ++b) {
    const int n0 = max(0, __ldg(p.prev_lens + b)), n1 = max(0, __ldg(p.lens + b));
    int prev = n0 / p.cmp_ratio, rows = n1 / p.cmp_ratio;
    if (cta == 0 && update < 2 && p.residual != nullptr) p.residual[b] = n1 - rows * p.cmp_ratio;
    wide |= prev > cap_rows || rows > cap_rows;
    // a table row that is too narrow: its last columns are missing, the rows
    // behind them get slots of -1
    const int held = (min(prev, cap_rows) + kBlock - 1) / kBlock, need = (min(rows, cap_rows) + kBlock - 1) / kBlock;
    s_prev[b] = prev;
    s_need[b] = need;
    s_rows[b] = max(0, rows - prev);
    s_taken[b] = max(0, need - held);
    s_given[b] = 0;
    shrinks |= held > need;
  }
  if (wide && cta == 0 && update < 2) atomicOr(fault, QSFM_FAULT_ORI_TABLE_COL);
  auto held_of = [&](int b) { return (min(s_prev[b], cap_rows) + kBlock - 1) / kBlock; };
  auto in_pool = [&](int block) { return block >= 0 && block < p.num_blocks; };
  if (__syncthreads_or(shrinks)) {
    constexpr int kWarps = kTabThreads / 32;
    const int lane = tid & 31;
    // neighbouring requests go to different warps
    for (int base = tid >> 5; base < p.batch; base += 32 * kWarps) {
      const int mine = base + lane * kWarps;
      uint32_t todo = __ballot_sync(0xffffffffu, mine < p.batch && held_of(mine) > s_need[mine]);
      for (; todo != 0; todo &= todo - 1) {
        const int b = base + (__ffs(todo) - 1) * kWarps, end = held_of(b);
        const int32_t* columns = p.block_table + size_t(b) * p.max_blocks;
        int blocks = 0;
        bool foreign = false;
        constexpr int kAtOnce = 16;  // columns that a lane has in flight
        for (int c = s_need[b] + lane; c < end; c += 32 * kAtOnce) {
          int block[kAtOnce];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) block[k] = c + 32 * k < end ? columns[c + 32 * k] : -1;
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            blocks += in_pool(block[k]) ? 1 : 0;
            foreign |= block[k] < -1 || block[k] >= p.num_blocks;
          }
        }
        blocks = __reduce_add_sync(0xffffffffu, blocks);
        if (lane == 0) s_given[b] = blocks;
        if (foreign && cta == 0 && update < 2) atomicOr(fault, QSFM_FAULT_ORI_BLOCK_ID);
      }
    }
    __syncthreads();
  }
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Sums own{s_rows[b], s_taken[b], s_given[b]};
    s_rows[b] = mine.rows;
    s_taken[b] = mine.taken;
    s_given[b] = mine.given;
    mine = add(mine, own);
  }
  Sums total;
  const Sums before = scan_before(mine, s_warps, total);
  for (int b = b0; b < b1; ++b) {
    s_rows[b] = add_rows(s_rows[b], before.rows);
    s_taken[b] += before.taken;
    s_given[b] += before.given;
    if (cta == 0 && update < 2 && p.cu_rows != nullptr) p.cu_rows[b] = s_rows[b];
  }
  __syncthreads();

  const int count = max(0, min(stack, p.free_capacity));
  const long long left = (long long)count + total.given - total.taken;  // negative: the pool is short
  if (cta == 0 && tid == 0) {
    if (update < 2) {
      if (p.cu_rows != nullptr) p.cu_rows[p.batch] = total.rows;
      if (left < 0 || left > p.free_capacity || stack != count) atomicOr(fault, QSFM_FAULT_BLOCK_POOL);
      if (total.rows > p.max_rows) atomicOr(fault, QSFM_FAULT_SLOT);
    }
    if (update > 0)
      *(p.free_count_out != nullptr ? p.free_count_out : p.free_count) =
          int(left < 0 ? 0 : left > p.free_capacity ? p.free_capacity : left);
  }
  if (update == 2) return;

  // a block id of the list or of a held column: -1 where it is none
  auto checked = [&](int block) {
    if (in_pool(block)) return block;
    atomicOr(fault, QSFM_FAULT_ORI_BLOCK_ID);
    return -1;
  };
  // the i-th block given back, and the i-th taken (-1: none left)
  auto given_block = [&](int i) {
    const int b = find_request(s_given, p.batch, i);
    const int blocks = (b + 1 < p.batch ? s_given[b + 1] : total.given) - s_given[b];
    int c = held_of(b);
    const int first = s_need[b], after = s_given[b] + blocks - 1 - i;  // columns with a block behind it
    const int32_t* columns = p.block_table + size_t(b) * p.max_blocks;
    if (blocks == c - first) return columns[c - 1 - after];
    // some columns hold none: from the last one down (the front ones are those behind a window),
    // 0.16 us per eight columns: a request of 1024 that ends with holes takes 20 us more at most
    for (int left = after; c > first;) {
      constexpr int kAtOnce = 8;
      int block[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) block[k] = c - 1 - k >= first ? columns[c - 1 - k] : -1;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (in_pool(block[k]) && left-- == 0) return block[k];
      c -= kAtOnce;
    }
    return -1;
  };
  auto taken_block = [&](int i) {
    const int from_top = total.given - 1 - i;  // of the blocks given back; then the free list
    return from_top >= 0 ? given_block(from_top) : count + from_top >= 0 ? checked(p.free_list[count + from_top]) : -1;
  };

  // Rows, taken and returned blocks start at different warps, so that their
  // dependent loads overlap when there are few of each.
  const int step = ctas * kTabThreads, me = cta * kTabThreads + tid;
  const int me_taken = me >= step / 2 ? me - step / 2 : me + step / 2, me_given = step - 1 - me;
  const bool vec = ((reinterpret_cast<uintptr_t>(p.slot_map) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
  for (int i0 = kTabRows * me; i0 < p.max_rows; i0 += kTabRows * step) {
    int slot[kTabRows], pos[kTabRows];
    int b = 0, next = 0, col_of = -1, block = -1;  // request of the row, start of the next, the block at hand
    if (i0 < total.rows) {
      b = find_request(s_rows, p.batch, i0);
      next = b + 1 < p.batch ? s_rows[b + 1] : total.rows;
    }
#pragma unroll
    for (int k = 0; k < kTabRows; ++k) {
      const int i = i0 + k;
      slot[k] = -1;
      pos[k] = -1;
      if (i >= total.rows) continue;
      while (i >= next) {  // empty requests are passed over; i < total.rows ends it
        ++b;
        next = b + 1 < p.batch ? s_rows[b + 1] : total.rows;
        col_of = -1;
      }
      const int row = s_prev[b] + (i - s_rows[b]);
      const int col = row / kBlock;
      pos[k] = row * p.cmp_ratio;
      if (col >= p.max_blocks) continue;
      if (col != col_of) {
        const int held = held_of(b);
        block = col < held ? checked(p.block_table[size_t(b) * p.max_blocks + col])
                           : taken_block(s_taken[b] + col - held);
        col_of = col;
      }
      if (block >= 0) slot[k] = block * kBlock + row % kBlock;
    }
    if (vec && i0 + kTabRows <= p.max_rows) {
      *reinterpret_cast<int4*>(p.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (p.positions != nullptr)
        *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kTabRows; ++k) {
        if (i0 + k >= p.max_rows) break;
        p.slot_map[i0 + k] = slot[k];
        if (p.positions != nullptr) p.positions[i0 + k] = pos[k];
      }
    }
  }
  for (int i = me_taken; i < total.taken; i += step) {
    const int b = find_request(s_taken, p.batch, i);
    p.block_table[size_t(b) * p.max_blocks + held_of(b) + (i - s_taken[b])] = taken_block(i);
  }
  // blocks given back and not taken again go onto the free list
  const int pushed = min(max(0, total.given - total.taken), p.free_capacity - count);
  for (int i = me_given; i < pushed; i += step) p.free_list[count + i] = given_block(i);
}

}  // namespace

cudaError_t launch_block_tables(const qsfm_block_table_params& p, int* fault, cudaStream_t s) {
  const size_t smem = 5 * size_t(p.batch) * sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024 - sizeof(Sums) * kTabThreads / 32)  // beyond what every kernel may use
    e = cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             5 * 8192 * int(sizeof(int)));
  if (e != cudaSuccess) return e;
  int ctas = 1;
  if (p.max_rows > kTabAlone) {
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int per = kTabThreads * kTabRows;
    ctas = (p.max_rows + per - 1) / per;
    if (ctas > 2 * sms) ctas = 2 * sms;
  }
  const bool in_place = p.free_count_out == nullptr || p.free_count_out == p.free_count;
  const int update = ctas > 1 && in_place ? 0 : 1;
  block_table_kernel<<<ctas, kTabThreads, smem, s>>>(p, update, fault);
  if (update == 0) block_table_kernel<<<1, kTabThreads, smem, s>>>(p, 2, fault);
  return cudaGetLastError();
}

}  // namespace qsfm
