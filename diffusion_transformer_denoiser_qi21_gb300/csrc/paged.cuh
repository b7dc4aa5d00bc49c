// Device side of a batch over a paged K/V cache (qi21_paged), shared by the
// append and the attention kernels.
#pragma once

#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace qi21 {

constexpr unsigned int kStatusPage = 2u;  // a page or row outside the cache

// The sequence of row t: the b in [0, nseq) with cu[b] <= t < cu[b + 1], or
// nseq if there is none. By one whole warp: 32 probes per round narrow the
// count of ends cu[1 ..] that are <= t, one round per factor of 32 of nseq
// (a binary search by one thread would wait for a load per factor of 2).
// Ends after a few rounds whatever cu holds.
__device__ __forceinline__ int warp_find_seq(const int32_t* __restrict__ cu, int nseq, int t, int lane) {
  int lo = 0, hi = nseq;  // the count is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t i = lo + static_cast<int64_t>(lane + 1) * step;
    const bool le = i <= hi && __ldg(cu + i) <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    const int64_t end = lo + static_cast<int64_t>(n + 1) * step - 1;
    lo += n * step;
    hi = end < hi ? static_cast<int>(end) : hi;
  }
  if (lo < nseq && !(__ldg(cu + lo) <= t && t < __ldg(cu + lo + 1))) lo = nseq;
  return lo;
}

// Row (of the flattened pool) of own row `own` of sequence b; -1, with the
// status raised, if the row or its page is outside the cache.
__device__ __forceinline__ int64_t paged_row(const PagedArgs& p, int b, int own, unsigned int* status) {
  if (own >= 0 && own < p.table_rows) {
    const int pg = own / p.page_rows;
    const int id = __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + pg);
    if (id >= 0 && id < p.npages) return static_cast<int64_t>(id) * p.page_rows + (own - pg * p.page_rows);
  }
  atomicOr(status, kStatusPage);
  return -1;
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 16 bytes from global to shared memory, both addresses multiples of 16.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

constexpr float kPagedRescale = 8.0f;  // log2 units: p <= 2^8, in f16 range

// One attention call over a paged cache.
struct PagedAttnArgs {
  PagedArgs kv;
  const void* q;
  void* out;
  int64_t ldq, ldo;
  int rows, heads, group;  // group: query heads of a key head
  int causal;
  const uint32_t* vis;
  float scale_log2;
  int pre_tiles, pre_splits;  // few-row tiles of the prefix, and the parts of its keys
  int own_tiles, own_splits;
  int pre_keys, own_keys;     // keys of a few-row part
  int cluster;                // > 0: few-row tiles walk [prefix, own keys], split over a cluster
  int first;                  // this kernel is the call's first
  int slots;                  // parts per row; 1: the part is the result
  float* part_o;              // [slots][rows][heads][dim]
  float2* part_ml;            // [slots][rows][heads] (max in log2 units, sum)
};

// The x-th tile, counted over the sequences in order, of `tile` of the `per`
// pieces that a row has: its sequence b and its place `at` there, the
// sequence's first row and rows in this call, and its length as given; by
// one whole warp (128 sequences per round, all of their numbers loaded at
// once: a round is a wait for memory). b == nseq: there are fewer tiles.
struct SeqTile {
  int b, at, row0, rows, len;
};
__device__ __forceinline__ SeqTile warp_find_tile(const PagedAttnArgs& a, int x, int per, int tile, int lane) {
  int before = 0;
  for (int b0 = 0; b0 < a.kv.nseq; b0 += 128) {
    const int b = b0 + 4 * lane;  // this lane's four sequences
    int c[5], len[4], n[4];
#pragma unroll
    for (int k = 0; k < 5; ++k) c[k] = b + k <= a.kv.nseq ? __ldg(a.kv.cu + b + k) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) len[k] = b + k < a.kv.nseq ? __ldg(a.kv.lens + b + k) : 0;
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // ends that do not fit the call's rows: no rows
      n[k] = b + k < a.kv.nseq && c[k] >= 0 && c[k + 1] <= a.rows && c[k + 1] > c[k] ? c[k + 1] - c[k] : 0;
      mine += (n[k] * per + tile - 1) / tile;
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > x);
    if (past) {
      const int l = __ffs(past) - 1;
      SeqTile r{b, x - before - (sum - mine), c[0], n[0], len[0]};  // lane l's is right
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int t = (n[k] * per + tile - 1) / tile;
        if (r.b == b + k && r.at >= t) r = SeqTile{b + k + 1, r.at - t, c[k + 1], n[k + 1], len[k + 1]};
      }
      r.b = __shfl_sync(0xffffffffu, r.b, l);
      r.at = __shfl_sync(0xffffffffu, r.at, l);
      r.row0 = __shfl_sync(0xffffffffu, r.row0, l);
      r.rows = __shfl_sync(0xffffffffu, r.rows, l);
      r.len = __shfl_sync(0xffffffffu, r.len, l);
      return r;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return SeqTile{a.kv.nseq, 0, 0, 0, 0};
}

// Programmatic launch: a call's kernels may start while the one before them
// in the stream still runs. grid_wait returns when that one has ended and
// its writes are visible; grid_release lets the next one start.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch that may start while the kernel before it in the stream runs
// (grid_wait inside it).
template <class... A>
inline cudaError_t launch_early(void (*kernel)(A...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                                unsigned cluster, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Key `k` of [prefix, own rows] of a sequence: its K row of key head hk (the
// V row is kv_heads * D further), or null for a page outside the cache.
template <int D>
__device__ __forceinline__ const uint16_t* key_row(const PagedAttnArgs& a, const int32_t* own_pages, int hk, int k) {
  const bool pre = k < a.kv.prefix_len;
  if (!pre) k -= a.kv.prefix_len;
  const int pg = k / a.kv.page_rows;
  const int id = __ldg((pre ? a.kv.prefix_pages : own_pages) + pg);
  if (id < 0 || id >= a.kv.npages) return nullptr;
  return static_cast<const uint16_t*>(a.kv.pool) +
         (static_cast<int64_t>(id) * a.kv.page_rows + (k - pg * a.kv.page_rows)) * (2 * a.kv.kv_heads * D) + hk * D;
}

// Is a value of keys [k0, k1) not finite? By one whole warp.
template <bool BF, int D>
__device__ __noinline__ bool odd_values(const PagedAttnArgs& a, const int32_t* own_pages, int hk, int k0, int k1, int lane) {
  float odd = 0.f;
  for (int k = k0; k < k1; ++k) {
    const uint16_t* row = key_row<D>(a, own_pages, hk, k);
    if (row == nullptr) continue;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(row + a.kv.kv_heads * D) + lane * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 x = unpack2<BF>(v[i]);
      odd = fmaf(0.f, x.x, fmaf(0.f, x.y, odd));
    }
  }
  return __any_sync(0xffffffffu, odd != odd);
}

// The sums of one query row over keys [k0, k1) alone, weights 2^(s - m): a
// lane leaves values [lane D / 32, + D / 32). By one whole warp, key by key:
// for the rare row that odd_values above sends here.
template <bool BF, int D>
__device__ __noinline__ void redo_row(const PagedAttnArgs& a, const int32_t* own_pages, int hk, int t, int h, int k0, int k1,
                                      float m, int lane, float (&acc)[D / 32]) {
  float2 q[D / 64];
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                         static_cast<int64_t>(t) * a.ldq + h * D) + lane * (D / 64);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    q[i] = unpack2<BF>(qr[i]);
    acc[2 * i] = acc[2 * i + 1] = 0.f;
  }
  const float base = m == -INFINITY ? 0.f : m;
  for (int k = k0; k < k1; ++k) {
    const uint16_t* row = key_row<D>(a, own_pages, hk, k);
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(row) + lane * (D / 64);
    const uint32_t* vr = reinterpret_cast<const uint32_t*>(row + a.kv.kv_heads * D) + lane * (D / 64);
    float s = 0.f;
    if (row != nullptr)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const float2 x = unpack2<BF>(kr[i]);
        s = fmaf(q[i].x, x.x, fmaf(q[i].y, x.y, s));
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float p = exp2f(fmaf(s, a.scale_log2, -base));
    if (row != nullptr)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const float2 x = unpack2<BF>(vr[i]);
        acc[2 * i] = fmaf(p, x.x, acc[2 * i]);
        acc[2 * i + 1] = fmaf(p, x.y, acc[2 * i + 1]);
      }
  }
}

// Tiles of many rows on the tensor cores (k_paged_tc.cu).
enum WideMode : int { WIDE_PREFIX = 0, WIDE_JOINT = 1, WIDE_STAY = 2 };  // STAY: joint, for several items
// Tokens of a CTA's tile, 0 if the group does not fit one.
inline int wide_tokens(int group) { return group <= 128 ? 128 / group : 0; }
cudaError_t launch_attn_wide(const PagedAttnArgs& a, WideMode mode, bool pair, int tiles, int splits, cudaStream_t s);

}  // namespace qi21
