// kda_cache.hip -- slots of a cache of states: copies, forks, frees, compaction, beams (gfx950).
//
// A plan kernel (one workgroup: S flags and n slot numbers are a few kilobytes) settles
// which slot goes where, and a copy kernel moves the contents. Plans go by counts of free
// or used slots before a slot, so their results do not depend on the order in which lanes run.
#include "kda_device.h"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int PLAN = 1024;   // lanes of a plan kernel; each counts the flags of a run of slots

// Exclusive sum of v over the workgroup's PLAN lanes; the total in *total.
__device__ __forceinline__ int plan_scan(int v, int* buf, int* total) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(s, o, 64);
    if (lane >= o) s += t;
  }
  __syncthreads();   // buf may still be read from the scan before
  if (lane == 63) buf[w] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < PLAN / 64; ++i) {
    if (i < w) before += buf[i];
    all += buf[i];
  }
  *total = all;
  return before + s - v;
}

__global__ __launch_bounds__(PLAN) void kda_cache_fork_plan_kernel(int32_t* used, int32_t S, const int32_t* src,
                                                                   int32_t* dst, int64_t n) {
  __shared__ int buf[PLAN / 64];
  __shared__ int pre[PLAN + 1];   // free slots before lane t's run
  const int tid = threadIdx.x;
  const int run = (S + PLAN - 1) / PLAN;
  const int s0 = tid * run < S ? tid * run : S, s1 = s0 + run < S ? s0 + run : S;
  int c = 0, total;
  for (int s = s0; s < s1; ++s) c += used[s] == 0;
  pre[tid] = plan_scan(c, buf, &total);
  if (tid == 0) pre[PLAN] = total;
  __syncthreads();
  int base = 0;
  for (int64_t i0 = 0; i0 < n; i0 += PLAN) {   // used[] is as before the call throughout
    const int64_t i = i0 + tid;
    const int from = i < n ? src[i] : -2;
    const bool live = from == -1 || (from >= 0 && from < S && used[from] != 0);
    int all;
    const int rank = base + plan_scan(live, buf, &all);
    int to = -1;
    if (live && rank < total) {
      int lo = 0, hi = PLAN;   // pre[lo] <= rank < pre[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= rank) lo = mid;
        else hi = mid;
      }
      int k = rank - pre[lo];   // the run holds more than k free slots: the walk ends inside it
      to = lo * run;
      while (to < S && (used[to] != 0 || k > 0)) k -= used[to++] == 0;
    }
    if (i < n) dst[i] = to;
    base = base + all < total ? base + all : total;   // (stays within int for any n)
  }
  __syncthreads();   // every request has its slot: used[] may change
  for (int64_t i = tid; i < n; i += PLAN) {
    const int to = dst[i];
    if (to >= 0) used[to] = 1;
  }
}

__global__ __launch_bounds__(256) void kda_cache_free_kernel(int32_t* used, int32_t S, const int32_t* slots, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int s = slots[i];
    if (s >= 0 && s < S) used[s] = 0;
  }
}

// ws: number of moves, then their sources and their targets (S / 2 + 1 places each)
__global__ __launch_bounds__(PLAN) void kda_cache_compact_plan_kernel(int32_t* used, int32_t S, int32_t* remap,
                                                                      int32_t* table, int64_t n, int32_t* ws) {
  __shared__ int buf[PLAN / 64];
  const int tid = threadIdx.x;
  const int run = (S + PLAN - 1) / PLAN;
  const int s0 = tid * run < S ? tid * run : S, s1 = s0 + run < S ? s0 + run : S;
  int32_t* src = ws + 1;
  int32_t* dst = src + S / 2 + 1;
  int c = 0, n_used, holes;
  for (int s = s0; s < s1; ++s) c += used[s] != 0;
  const int before = plan_scan(c, buf, &n_used);   // used slots before this run
  // free slots below n_used, as many as used ones from n_used on
  int h = 0;
  for (int s = s0; s < s1 && s < n_used; ++s) h += used[s] == 0;
  const int hole0 = plan_scan(h, buf, &holes);
  int hole = hole0, k = before;   // k: used slots before s
  for (int s = s0; s < s1; ++s) {
    const bool u = used[s] != 0;
    if (s < n_used) {
      if (!u) dst[hole++] = s;
    } else if (u) {
      src[k - (n_used - holes)] = s;   // n_used - holes used slots lie below n_used
    }
    k += u;
  }
  __syncthreads();
  k = before;
  for (int s = s0; s < s1; ++s) {
    const bool u = used[s] != 0;
    remap[s] = !u ? -1 : s < n_used ? s : dst[k - (n_used - holes)];
    k += u;
    used[s] = s < n_used;
  }
  if (tid == 0) ws[0] = holes;
  __syncthreads();
  for (int64_t i = tid; i < n; i += PLAN) {
    const int s = table[i];
    table[i] = s >= 0 && s < S ? remap[s] : -1;
  }
}

// Copies the contents of listed slots in every layer; src -1 writes zeros (zeros set), a target
// outside the pool or a slot onto itself nothing. Unit: 16, 4 or 1 bytes. A workgroup takes
// pieces of PIECE units of one slot and layer. Bound by memory: 123 slots of 256 KiB in 6 layers
// take 78 us (5.0 TB/s); stored past the caches (a fork of 64 slots of 4 MiB 92.6 -> 83.8 us).
constexpr int PIECE = 1024;   // 256 lanes x 4 units
template <typename U>
__global__ __launch_bounds__(256) void kda_cache_copy_kernel(CachePool pool, size_t units, const int32_t* src,
                                                             const int32_t* dst, const int32_t* count, int64_t n,
                                                             bool zeros) {
  if (count) {   // n is the most there can be (kept to if another call writes the workspace)
    const int c = *count;
    n = c < 0 ? 0 : c < n ? c : n;
  }
  const int64_t pieces = (int64_t)((units + PIECE - 1) / PIECE);
  const int64_t items = n * pool.layers * pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t i = it / (pool.layers * pieces), r = it - i * (pool.layers * pieces);
    const int64_t layer = r / pieces;
    const size_t u0 = (size_t)(r - layer * pieces) * PIECE + threadIdx.x;
    const int64_t from = src[i], to = dst[i];
    if (to < 0 || to >= pool.slots || from >= pool.slots || from < (zeros ? -1 : 0) || from == to) continue;
    U* base = static_cast<U*>(pool.base) + (size_t)layer * pool.slots * units;
    U* out = base + (size_t)to * units;
    U v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const size_t u = u0 + 256 * j;
      v[j] = U{};
      if (from >= 0 && u < units) v[j] = base[(size_t)from * units + u];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const size_t u = u0 + 256 * j;
      if (u < units) __builtin_nontemporal_store(v[j], out + u);
    }
  }
}

hipError_t copy_slots(const CachePool& pool, const int32_t* src, const int32_t* dst, const int32_t* count, int64_t n,
                      bool zeros, hipStream_t stream) {
  const int unit = pool.slot_bytes % 16 == 0 ? 16 : pool.slot_bytes % 4 == 0 ? 4 : 1;
  const size_t units = pool.slot_bytes / unit;
  const double items = (double)n * pool.layers * (double)((units + PIECE - 1) / PIECE);
  const unsigned blocks = items < 8192.0 ? (unsigned)items : 8192u;
  if (blocks == 0) return hipSuccess;
  if (unit == 16)
    hipLaunchKernelGGL(kda_cache_copy_kernel<u32x4>, dim3(blocks), dim3(256), 0, stream, pool, units, src, dst, count, n, zeros);
  else if (unit == 4)
    hipLaunchKernelGGL(kda_cache_copy_kernel<uint32_t>, dim3(blocks), dim3(256), 0, stream, pool, units, src, dst, count, n, zeros);
  else
    hipLaunchKernelGGL(kda_cache_copy_kernel<uint8_t>, dim3(blocks), dim3(256), 0, stream, pool, units, src, dst, count, n, zeros);
  return hipGetLastError();
}

// The states of a sequence's W <= 64 beams after a step of beam search (rules in the header). A
// workgroup takes a piece of one sequence's slots in one layer and makes all copies of it; each
// settles for itself, in one wave, which slots become copies of which. No copy reads what another
// writes: sources are slots that a beam continues in, targets slots of beams that no one continues.
// Bound by memory where states are large (32 x 8 beams with 512 KiB in 2 layers: 45 us, 5.2 TB/s).
constexpr int BEAMS = 64;
template <typename U>
__global__ __launch_bounds__(256) void kda_cache_reorder_kernel(CachePool pool, size_t units, const int32_t* slots,
                                                                const int32_t* parents, int32_t* new_slots, int64_t N, int W) {
  __shared__ int from_s[BEAMS], to_s[BEAMS], n_s;
  const int64_t pieces = (int64_t)((units + PIECE - 1) / PIECE), items = N * pool.layers * pieces;
  const int tid = threadIdx.x;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t n = it / (pool.layers * pieces), r = it - n * (pool.layers * pieces);
    const int64_t layer = r / pieces, piece = r - layer * pieces;
    __syncthreads();   // the item before is done with the lists
    if (tid < 64) {    // lane j: new beam j, and old beam j
      const bool in = tid < W;
      const int slot = in ? slots[n * W + tid] : -1;
      int parent = in ? parents[n * W + tid] : -1;
      if (parent < 0 || parent >= W) parent = -1;
      bool first = parent >= 0, continued = false;
      for (int j = 0; j < W; ++j) {
        const int other = __builtin_amdgcn_readlane(parent, j);
        if (other == parent && j < tid) first = false;
        if (other == tid) continued = true;
      }
      const uint64_t below = ((uint64_t)1 << tid) - 1;
      const uint64_t moved = __ballot(in && !first), free = __ballot(in && !continued);   // as many
      // the free slots in ascending order of their beams
      if (in && !continued) to_s[__popcll(free & below)] = slot;
      const int rank = __popcll(moved & below);
      const int old = __shfl(slot, parent < 0 ? 0 : parent, 64);
      __builtin_amdgcn_wave_barrier();   // (a wave's accesses of shared memory are in order)
      const int now = in && !first ? to_s[rank] : old;
      if (in && !first) from_s[rank] = parent >= 0 ? old : -1;
      if (tid == 0) n_s = __popcll(moved);
      if (in && layer == 0 && piece == 0) new_slots[n * W + tid] = now;
    }
    __syncthreads();
    U* base = static_cast<U*>(pool.base) + (size_t)layer * pool.slots * units;
    const size_t u0 = (size_t)piece * PIECE + tid;
    for (int i = 0; i < n_s; ++i) {
      const int64_t from = from_s[i], to = to_s[i];
      if (from < 0 || from >= pool.slots || to < 0 || to >= pool.slots || from == to) continue;
      U v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const size_t u = u0 + 256 * j;
        v[j] = U{};
        if (u < units) v[j] = base[(size_t)from * units + u];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const size_t u = u0 + 256 * j;
        if (u < units) __builtin_nontemporal_store(v[j], base + (size_t)to * units + u);
      }
    }
  }
}

}  // namespace

hipError_t launch_cache_copy(const CachePool& pool, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream) {
  return copy_slots(pool, src, dst, nullptr, n, false, stream);
}

hipError_t launch_cache_fork(const CachePool& pool, int32_t* used, const int32_t* src, int32_t* dst, int64_t n,
                             hipStream_t stream) {
  hipLaunchKernelGGL(kda_cache_fork_plan_kernel, dim3(1), dim3(PLAN), 0, stream, used, (int32_t)pool.slots, src, dst, n);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? copy_slots(pool, src, dst, nullptr, n, true, stream) : e;
}

hipError_t launch_cache_free(int32_t* used, int64_t S, const int32_t* slots, int64_t n, hipStream_t stream) {
  const int64_t blocks = (n + 255) / 256;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(kda_cache_free_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream, used,
                     (int32_t)S, slots, n);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CachePool& pool, int32_t* used, int32_t* remap, int32_t* table, int64_t n,
                                int32_t* ws, hipStream_t stream) {
  const int32_t S = (int32_t)pool.slots;
  hipLaunchKernelGGL(kda_cache_compact_plan_kernel, dim3(1), dim3(PLAN), 0, stream, used, S, remap, table, n, ws);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? copy_slots(pool, ws + 1, ws + 1 + S / 2 + 1, ws, S / 2, false, stream) : e;
}

hipError_t launch_cache_reorder(const CachePool& pool, const int32_t* slots, const int32_t* parents, int32_t* new_slots,
                                int64_t N, int W, hipStream_t stream) {
  if (N == 0) return hipSuccess;
  const int unit = pool.slot_bytes % 16 == 0 ? 16 : pool.slot_bytes % 4 == 0 ? 4 : 1;
  const size_t units = pool.slot_bytes / unit;
  const double items = (double)N * pool.layers * (double)((units + PIECE - 1) / PIECE);
  const dim3 grid(items < 8192.0 ? (unsigned)items : 8192u), wg(256);
  if (unit == 16)
    hipLaunchKernelGGL(kda_cache_reorder_kernel<u32x4>, grid, wg, 0, stream, pool, units, slots, parents, new_slots, N, W);
  else if (unit == 4)
    hipLaunchKernelGGL(kda_cache_reorder_kernel<uint32_t>, grid, wg, 0, stream, pool, units, slots, parents, new_slots, N, W);
  else
    hipLaunchKernelGGL(kda_cache_reorder_kernel<uint8_t>, grid, wg, 0, stream, pool, units, slots, parents, new_slots, N, W);
  return hipGetLastError();
}

}  // namespace kda
