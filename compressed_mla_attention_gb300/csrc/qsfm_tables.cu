// Block tables and slots of the paged cache from request lengths (sm_103a).
//
// The bookkeeping between two steps of a serving loop: which blocks the
// requests give back and take, and the pool row of every new cache row. With
// the cache rows of request b before and after the step, p_b and r_b, its
// blocks before and after, h_b = ceil(p_b / 128) and n_b = ceil(r_b / 128),
//   G_b = sum_{i<b} max(0, h_i - n_i)   blocks given back before request b,
//   T_b = sum_{i<b} max(0, n_i - h_i)   blocks taken before it,
//   N_b = sum_{i<b} max(0, r_i - p_i)   new rows before it,
// the i-th block taken is the i-th from the top of the stack "free list, then
// the blocks given back in order", so each output element follows from the
// three prefix sums alone and no thread waits for another's write.
//
// One launch of one cluster: every CTA computes the prefix sums over the
// batch for itself (8 KB to 100 KB of shared memory; the lengths come from L2)
// and takes a share of the output elements, each of which finds its request
// by a binary search in shared memory. The cluster barrier separates the
// reads of free_count from its update in place. Everything else is read and
// written at disjoint places: columns below h_b are read, columns from h_b on
// written; entries below the count are read, entries from it on written.
// Bound by latency: the launch, one round trip for the lengths, the scan, the
// search and one or two round trips for a block id.
#include <cub/block/block_scan.cuh>
#include <cuda_runtime.h>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabMaxCtas = 8;  // the portable cluster size

// Prefix sums; the row counts of absurd lengths stop at the largest int (the
// table has at most 2^30 entries, so the block counts cannot pass it).
struct Sums {
  int rows, taken, given;
};
__device__ __forceinline__ int add_rows(int a, int b) { return int(min(unsigned(a) + unsigned(b), 0x7fffffffu)); }
struct AddSums {
  __device__ __forceinline__ Sums operator()(const Sums& a, const Sums& b) const {
    return {add_rows(a.rows, b.rows), a.taken + b.taken, a.given + b.given};
  }
};

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

__global__ void __launch_bounds__(kTabThreads) block_table_kernel(const qsfm_block_table_params p, int* fault) {
  using Scan = cub::BlockScan<Sums, kTabThreads>;
  __shared__ typename Scan::TempStorage scan_tmp;
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
  Sums mine{0, 0, 0};
  bool wide = false;
  for (int b = b0; b < b1; ++b) {
    const int n0 = max(0, __ldg(p.prev_lens + b)), n1 = max(0, __ldg(p.lens + b));
    int prev = n0 / p.cmp_ratio, rows = n1 / p.cmp_ratio;
    if (cta == 0 && p.residual != nullptr) p.residual[b] = n1 - rows * p.cmp_ratio;
    wide |= prev > cap_rows || rows > cap_rows;
    // a table row that is too narrow: its last columns are missing, the rows
    // behind them get slots of -1
    const int held = (min(prev, cap_rows) + kBlock - 1) / kBlock, need = (min(rows, cap_rows) + kBlock - 1) / kBlock;
    s_prev[b] = prev;
    s_need[b] = need;
    s_rows[b] = mine.rows;
    s_taken[b] = mine.taken;
    s_given[b] = mine.given;
    mine.rows = add_rows(mine.rows, max(0, rows - prev));
    mine.taken += max(0, need - held);
    mine.given += max(0, held - need);
  }
  if (wide && cta == 0) atomicOr(fault, QSFM_FAULT_ORI_TABLE_COL);
  Sums before, total;
  Scan(scan_tmp).ExclusiveScan(mine, before, Sums{0, 0, 0}, AddSums(), total);
  for (int b = b0; b < b1; ++b) {
    s_rows[b] = add_rows(s_rows[b], before.rows);
    s_taken[b] += before.taken;
    s_given[b] += before.given;
    if (cta == 0 && p.cu_rows != nullptr) p.cu_rows[b] = s_rows[b];
  }
  __syncthreads();

  const int count = max(0, min(stack, p.free_capacity));
  const long long left = (long long)count + total.given - total.taken;  // negative: the pool is short
  if (cta == 0 && tid == 0) {
    if (p.cu_rows != nullptr) p.cu_rows[p.batch] = total.rows;
    if (left < 0 || left > p.free_capacity || stack != count) atomicOr(fault, QSFM_FAULT_BLOCK_POOL);
    if (total.rows > p.max_rows) atomicOr(fault, QSFM_FAULT_SLOT);
  }
  if (ctas > 1) {  // every CTA has read the count
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
  }
  if (cta == 0 && tid == 0)
    *(p.free_count_out != nullptr ? p.free_count_out : p.free_count) =
        int(left < 0 ? 0 : left > p.free_capacity ? p.free_capacity : left);
  if (p.batch == 0) {
    for (int i = cta * kTabThreads + tid; i < p.max_rows; i += ctas * kTabThreads) {
      p.slot_map[i] = -1;
      if (p.positions != nullptr) p.positions[i] = -1;
    }
    return;
  }

  // the i-th block given back, and the i-th taken (-1: none left)
  auto given_block = [&](int i) {
    const int b = find_request(s_given, p.batch, i);
    return p.block_table[size_t(b) * p.max_blocks + s_need[b] + (i - s_given[b])];
  };
  auto taken_block = [&](int i) {
    const int from_top = total.given - 1 - i;  // of the blocks given back; then the free list
    return from_top >= 0 ? given_block(from_top) : count + from_top >= 0 ? p.free_list[count + from_top] : -1;
  };
  auto held_of = [&](int b) { return (min(s_prev[b], cap_rows) + kBlock - 1) / kBlock; };
  auto checked = [&](int block) {
    if (block >= p.num_blocks || block < -1) {
      atomicOr(fault, QSFM_FAULT_ORI_BLOCK_ID);
      return -1;
    }
    return block;
  };

  const int step = ctas * kTabThreads;
  for (int i = cta * kTabThreads + tid; i < p.max_rows; i += step) {
    int slot = -1, pos = -1;
    if (i < total.rows) {
      const int b = find_request(s_rows, p.batch, i);
      const int row = s_prev[b] + (i - s_rows[b]);
      const int col = row / kBlock, held = held_of(b);
      pos = row * p.cmp_ratio;
      if (col < p.max_blocks) {
        const int block = checked(col < held ? p.block_table[size_t(b) * p.max_blocks + col]
                                             : taken_block(s_taken[b] + col - held));
        if (block >= 0) slot = block * kBlock + row % kBlock;
      }
    }
    p.slot_map[i] = slot;
    if (p.positions != nullptr) p.positions[i] = pos;
  }
  for (int i = cta * kTabThreads + tid; i < total.taken; i += step) {
    const int b = find_request(s_taken, p.batch, i);
    p.block_table[size_t(b) * p.max_blocks + held_of(b) + (i - s_taken[b])] = checked(taken_block(i));
  }
  // blocks given back and not taken again go onto the free list
  const int pushed = min(max(0, total.given - total.taken), p.free_capacity - count);
  for (int i = cta * kTabThreads + tid; i < pushed; i += step) p.free_list[count + i] = given_block(i);
}

}  // namespace

cudaError_t launch_block_tables(const qsfm_block_table_params& p, int* fault, cudaStream_t s) {
  const size_t smem = 5 * size_t(p.batch) * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       5 * 8192 * int(sizeof(int)));
  if (e != cudaSuccess) return e;
  const int work = p.max_rows > 2 * p.batch ? p.max_rows : 2 * p.batch;
  int ctas = 1;
  while (ctas < kTabMaxCtas && ctas * kTabThreads < work) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_table_kernel, p, fault);
}

}  // namespace qsfm
