// Attention over a paged K/V cache whose prefix all sequences of the batch
// share. For query row t and head h of group g = h / (heads / kv_heads):
//   s_j = scale q . k_j,  p_j = exp(s_j - m),  out = sum_j p_j v_j / sum_j p_j
// over the keys j that the row sees. The sums over the prefix and over a
// sequence's own keys are taken apart (and each in splits, where that fills
// the GPU), every part leaving (m, sum p, sum p v) in f32, and joined with
// weights 2^(m_part - m): exact, as the parts differ only in the factor
// 2^m. So the rows of all sequences read the prefix once, together.
#include <algorithm>
#include <cmath>

#include "attn.cuh"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace qi21 {

static __device__ unsigned int s_paged_status = 0;

unsigned int paged_status_read_clear() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, s_paged_status, sizeof v);
  cudaMemcpyToSymbol(s_paged_status, &z, sizeof z);
  return v;
}

constexpr int kGran = 16;               // keys of a granule: never crosses a page
constexpr int kWarps = 4;               // of a CTA

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Loads from the shared memory of a CTA of the cluster.
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Is a value of the 16 x D granule at `addr` not finite? By one whole warp.
template <bool BF, int D>
__device__ __forceinline__ bool odd_granule(uint32_t addr, int lane) {
  float odd = 0.f;  // NaN once one is met
#pragma unroll
  for (int i = 0; i < kGran * D * 2 / 128; ++i) {
    const float2 v = unpack2<BF>(lds32(addr + i * 128 + lane * 4));
    odd = fmaf(0.f, v.x, fmaf(0.f, v.y, odd));
  }
  return __any_sync(0xffffffffu, odd != odd);
}

// c += a b, m16n8k16, f32 sums.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------- few rows a tile --
// A CTA takes a tile of 16 MT (row, head) pairs of one key head and a part of
// the keys, the prefix's or a sequence's own. Its four warps take granules
// of 16 keys in turn, each through a ring of its own (16-byte asynchronous
// copies, rows behind the end filled with zeros), so no warp waits for
// another: a granule is Q K^T, the running maximum and sum, and P V, by
// m16n8k16 MMAs with P taken from the score registers. The warps' parts are
// joined at the end. It is bound by the bytes of K and V: a tile has few
// rows, so the 128-row tensor-core tiles would be nearly empty. Two stages a
// warp rather than three leave room for three CTAs on an SM, whose starts
// and ends overlap.
//
// Small calls (a.cluster > 0) are one launch: a tile's CTAs walk [prefix, own
// keys] of its sequence, split evenly over a cluster of up to eight that
// joins its parts through distributed shared memory.
template <int D>
constexpr int kNarrowStages = D == 128 ? 2 : 3;
template <int D>
constexpr int kNarrowRing = kNarrowStages<D> * 2 * kGran * D * 2;  // of a warp
// The warps' f32 sums take the rings' place at the end, where they need more.
template <int D, int MT>
constexpr int kNarrowSums = 16 * MT * (D + 4) * 4 > kNarrowRing<D> ? 16 * MT * (D + 4) * 4 : kNarrowRing<D>;
template <int D, int MT>
constexpr int kNarrowPart = kWarps * kNarrowSums<D, MT>;  // offset of a CTA's part: sums, then (max, sum)
template <int D, int MT>
constexpr int kNarrowSmem = kNarrowPart<D, MT> + 16 * MT * (D * 4 + 8);

template <bool BF, int D, int MT>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_narrow(const __grid_constant__ PagedAttnArgs a) {
  constexpr int R = 16 * MT;
  constexpr int NST = kNarrowStages<D>;
  constexpr int HALF = kGran * D * 2;  // bytes of a granule's K (or V)
  constexpr int CH = D / 8;            // 16-byte pieces of a row
  constexpr int RS = 32 / CH;          // rows that a warp copies at once
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the key heads of a tile run side by side: their rows share DRAM pages
  const int ncl = max(1, a.cluster);
  int x = static_cast<int>(blockIdx.x / static_cast<unsigned>(ncl));
  const int hk = x % a.kv.kv_heads;
  x /= a.kv.kv_heads;
  // the call's first kernel waits for what came before the call. A later one
  // reads nothing of the kernel before it, so only its last CTA waits, at its
  // end: the join waits for this kernel alone, which must end after that one
  const bool waits = !a.first && blockIdx.x == gridDim.x - 1;
  if (a.first) grid_wait();
  grid_release();

  // the tile: pairs [r0, npairs) of the rows [t0, ...) and the sources of its
  // keys, the prefix (np rows), own keys (len rows) or both
  const bool pre = x < a.pre_tiles * a.pre_splits;
  const int P = a.kv.prefix_len;
  const int np = pre || a.cluster ? P : 0;
  int t0 = 0, npairs, r0, split, slot, len = 0, nrows = 0;
  const int32_t* own_pages = nullptr;
  if (pre) {
    const int tile = x / a.pre_splits;
    split = x - tile * a.pre_splits;
    slot = split;
    npairs = min(max(__ldg(a.kv.cu + a.kv.nseq), 0), a.rows) * a.group;
    r0 = tile * R;
  } else {
    x -= a.pre_tiles * a.pre_splits;
    const int tile = x / a.own_splits;
    split = a.cluster ? static_cast<int>(cluster_rank()) : x - tile * a.own_splits;
    slot = a.pre_splits + split;
    const SeqTile q = warp_find_tile(a, tile, a.group, R, lane);
    t0 = q.row0;
    nrows = q.rows;
    npairs = nrows * a.group;  // 0 if there is no such tile
    r0 = q.at * R;
    own_pages = a.kv.table + static_cast<int64_t>(q.b) * a.kv.table_stride;
    len = q.len;
    if (npairs > 0 && (len < nrows || len > a.kv.table_rows) && threadIdx.x == 0) atomicOr(&s_paged_status, kStatusPage);
    len = min(max(len, 0), a.kv.table_rows);
  }
  if (r0 >= npairs) {  // all CTAs of a cluster
    if (waits) grid_wait();
    return;
  }

  // this thread's rows: lane / 4 and + 8 of every 16; the keys that they see of the
  // prefix and of the own ones, and the most and least of the tile
  const int tq = lane >> 2, tj = lane & 3;
  int lim_p[MT][2], lim_o[MT][2];
  uint32_t qf[MT][D / 16][4];
  int most_p = 0, most_o = 0, least_p = 0x7fffffff, least_o = 0x7fffffff;
#pragma unroll
  for (int me = 0; me < 2 * MT; ++me) {
    const int mt = me >> 1, e = me & 1;
    const int pr = r0 + 16 * mt + tq + 8 * e;
    const bool live = pr < npairs;
    const int i = live ? pr / a.group : 0;
    const int t = t0 + i;
    const int h = hk * a.group + (live ? pr - i * a.group : 0);
    int n = P + len;  // of [prefix, own keys]
    if (live && a.vis)
      n = static_cast<int>(min(__ldg(a.vis + t), static_cast<uint32_t>(n)));
    else if (a.causal && !pre)
      n = P + min(max(len - nrows + i + 1, 0), len);
    lim_p[mt][e] = live ? min(n, np) : 0;
    lim_o[mt][e] = live ? min(max(n - P, 0), len) : 0;
    most_p = max(most_p, lim_p[mt][e]);
    most_o = max(most_o, lim_o[mt][e]);
    if (live) {
      least_p = min(least_p, lim_p[mt][e]);
      least_o = min(least_o, lim_o[mt][e]);
    }
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                           static_cast<int64_t>(t) * a.ldq + h * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[mt][k][e] = live ? __ldg(qr + 8 * k + tj) : 0u;
      qf[mt][k][2 + e] = live ? __ldg(qr + 8 * k + 4 + tj) : 0u;
    }
  }
  most_p = __reduce_max_sync(0xffffffffu, most_p);
  most_o = __reduce_max_sync(0xffffffffu, most_o);
  least_p = __reduce_min_sync(0xffffffffu, least_p);
  least_o = __reduce_min_sync(0xffffffffu, least_o);

  // granules: the prefix's, then the own keys'; this warp's are g0, g0 + 4,
  // ... below g1
  const int gp = (most_p + kGran - 1) / kGran;
  const int ng = gp + (most_o + kGran - 1) / kGran;
  int g0, g1;
  if (a.cluster) {
    g0 = static_cast<int>(static_cast<int64_t>(ng) * split / ncl);
    g1 = static_cast<int>(static_cast<int64_t>(ng) * (split + 1) / ncl);
  } else {
    // equal parts of the longest sequence that the table can hold; a shorter
    // one is cut as often, but into parts of 256 keys at least
    int part = (pre ? a.pre_keys : a.own_keys) / kGran;
    if (!pre) part = min(part, max(256 / kGran, (ng + a.own_splits - 1) / a.own_splits));
    const int64_t k0 = static_cast<int64_t>(split) * part;
    g0 = static_cast<int>(min(k0, static_cast<int64_t>(ng)));
    g1 = static_cast<int>(min(k0 + part, static_cast<int64_t>(ng)));
  }
  const bool any = g0 < g1;
  g0 += warp;
  const uint32_t sring = smem_u32(smem) + warp * (NST * 2 * HALF);
  const int64_t row_bytes = 4 * static_cast<int64_t>(a.kv.kv_heads) * D;
  const int64_t v_off = 2 * static_cast<int64_t>(a.kv.kv_heads) * D;
  // copies: a lane moves piece cp_c of rows cp_r, cp_r + RS, ...
  const int cp_r = lane / CH, cp_c = lane % CH;
  const uint8_t* cp_src = static_cast<const uint8_t*>(a.kv.pool) + hk * (2 * D) + cp_c * 16 + cp_r * row_bytes;
  auto page_of = [&](int g) {
    return g < gp ? __ldg(a.kv.prefix_pages + g * kGran / a.kv.page_rows)
                  : __ldg(own_pages + (g - gp) * kGran / a.kv.page_rows);
  };
  auto fetch = [&](int g, int id, int st) {
    const bool ok = id >= 0 && id < a.kv.npages;
    if (!ok && lane == 0) atomicOr(&s_paged_status, kStatusPage);
    const int key = (g < gp ? g : g - gp) * kGran;
    const int left = ok ? (g < gp ? most_p : most_o) - key : 0;  // rows before the end
    const int64_t row = static_cast<int64_t>(ok ? id : 0) * a.kv.page_rows + key % a.kv.page_rows;
    const uint8_t* src = cp_src + row * row_bytes;
    const uint32_t dst = sring + st * 2 * HALF + cp_r * (D * 2);
    if (left >= kGran) {
#pragma unroll
      for (int i = 0; i < kGran / RS; ++i) {
        const uint32_t d = dst + i * (RS * D * 2) + ((cp_c ^ ((cp_r + i * RS) & 7)) << 4);
        cp_async16(d, src, true);
        cp_async16(d + HALF, src + v_off, true);
        src += RS * row_bytes;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kGran / RS; ++i) {
        const uint32_t d = dst + i * (RS * D * 2) + ((cp_c ^ ((cp_r + i * RS) & 7)) << 4);
        const bool live = cp_r + i * RS < left;
        cp_async16(d, live ? src : cp_src, live);
        cp_async16(d + HALF, live ? src + v_off : cp_src, live);
        src += RS * row_bytes;
      }
    }
  };

  float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
    m[mt][0] = m[mt][1] = -INFINITY;
    l[mt][0] = l[mt][1] = 0.f;
  }

  int nf = g0;  // next granule to fetch
  int nid = nf < g1 ? page_of(nf) : 0;
  auto fetch_next = [&](int st) {
    if (nf < g1) {
      const int id = nid, g = nf;
      nf += kWarps;
      if (nf < g1) nid = page_of(nf);
      fetch(g, id, st);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) fetch_next(s);
  int st = 0;
  // matrix addresses of this lane: K by rows (lane % 8 and the upper half),
  // V by rows for the transposed load
  const int kkey = (lane >> 4) * 8 + (lane & 7), kbit = (lane >> 3) & 1;
  const int vkey = ((lane >> 3) & 1) * 8 + (lane & 7), vbit = lane >> 4;
  const uint32_t kx = (kbit ^ (kkey & 7)) << 4, vx = (vbit ^ (vkey & 7)) << 4;
  const float c = a.scale_log2;
  for (int g = g0; g < g1; g += kWarps) {
    cp_async_wait<NST - 2>();
    __syncwarp();
    {
      int fs = st + NST - 1;
      if (fs >= NST) fs -= NST;
      fetch_next(fs);
    }
    const int cur = st;
    const uint32_t sk = sring + st * 2 * HALF + kkey * (D * 2), sv = sring + st * 2 * HALF + HALF + vkey * (D * 2);
    if (++st == NST) st = 0;

    float s[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t b[4];
      ldsm4<false>(sk + (kx ^ (k << 5)), b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816<BF>(s[mt][0], qf[mt][k], b[0], b[1]);
        mma16816<BF>(s[mt][1], qf[mt][k], b[2], b[3]);
      }
    }
    const bool of_p = g < gp;
    const int key = (of_p ? g : g - gp) * kGran;
    const bool partly = key + kGran > (of_p ? least_p : least_o);
    if (partly) {  // what a row does not see is taken out
      const int col = key + 2 * tj;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int lim[2] = {of_p ? lim_p[mt][0] : lim_o[mt][0], of_p ? lim_p[mt][1] : lim_o[mt][1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + 8 * n + (e & 1) >= lim[e >> 1]) s[mt][n][e] = -INFINITY;
      }
    }
    uint32_t p[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float al[2];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s0 = s[mt][0][2 * e], s1 = s[mt][0][2 * e + 1], s2 = s[mt][1][2 * e], s3 = s[mt][1][2 * e + 1];
        float mx = fmaxf(fmaxf(s0, s1), fmaxf(s2, s3));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * c;
        // the maximum (log2 units) is raised only past the threshold: o and l
        // share it
        al[e] = 1.f;
        if (mx > m[mt][e] + kPagedRescale) {
          al[e] = ex2(m[mt][e] - mx);
          m[mt][e] = mx;
          moved = true;
        }
        // a row that has seen no key yet has weights 2^(-inf - 0) = 0
        const float base = m[mt][e] == -INFINITY ? 0.f : -m[mt][e];
        const float p0 = ex2(fmaf(s0, c, base)), p1 = ex2(fmaf(s1, c, base));
        const float p2 = ex2(fmaf(s2, c, base)), p3 = ex2(fmaf(s3, c, base));
        // P is rounded to the values' type for the MMA (half a step of a
        // weight each, of either sign); l sums the f32 weights
        p[mt][e] = pack2<BF>(p0, p1);
        p[mt][2 + e] = pack2<BF>(p2, p3);
        l[mt][e] = fmaf(l[mt][e], al[e], (p0 + p1) + (p2 + p3));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[mt][n][0] *= al[0];
          o[mt][n][1] *= al[0];
          o[mt][n][2] *= al[1];
          o[mt][n][3] *= al[1];
        }
      }
    }
    const uint32_t sgv = sring + cur * 2 * HALF + HALF;  // the granule's V
    if (partly && odd_granule<BF, D>(sgv, lane)) {
      // a weight of 0 does not take out a value that is not finite (0 times
      // it is a NaN): this granule's sums key by key, over what a row sees
#pragma unroll 1
      for (int k = 0; k < kGran; ++k) {
        const int from = (lane & ~3) | ((k & 7) >> 1);
        const uint32_t vr = sgv + k * (D * 2) + tj * 4;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t lo = __shfl_sync(0xffffffffu, p[mt][e], from), hi = __shfl_sync(0xffffffffu, p[mt][2 + e], from);
            const float2 pp = unpack2<BF>(k < 8 ? lo : hi);
            const float pk = k & 1 ? pp.y : pp.x;
            if (key + k < (of_p ? lim_p[mt][e] : lim_o[mt][e])) {
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                const float2 v = unpack2<BF>(lds32(vr + ((n ^ (k & 7)) << 4)));
                o[mt][n][2 * e] = fmaf(pk, v.x, o[mt][n][2 * e]);
                o[mt][n][2 * e + 1] = fmaf(pk, v.y, o[mt][n][2 * e + 1]);
              }
            }
          }
      }
    } else {
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldsm4<true>(sv + (vx ^ (n << 5)), b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816<BF>(o[mt][2 * n], p[mt], b[0], b[1]);
          mma16816<BF>(o[mt][2 * n + 1], p[mt], b[2], b[3]);
        }
      }
    }
    __syncwarp();  // the stage is refilled next round
  }
  cp_async_wait<0>();

  // join the four warps: each leaves its sums in its ring
  constexpr int OP = D + 4;  // row pitch of the f32 sums: spreads the rows over the banks
  float* so = reinterpret_cast<float*>(smem + warp * kNarrowSums<D, MT>);
  if (kNarrowSums<D, MT> > kNarrowRing<D>)
    __syncthreads();  // they reach into another warp's ring
  else
    __syncwarp();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[mt][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (tj == 0) {
        s_m[warp][16 * mt + tq + 8 * e] = m[mt][e];
        s_l[warp][16 * mt + tq + 8 * e] = sum;
      }
    }
    float* row = so + (16 * mt + tq) * OP + 2 * tj;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      *reinterpret_cast<float2*>(row + 8 * n) = make_float2(o[mt][n][0], o[mt][n][1]);
      *reinterpret_cast<float2*>(row + 8 * OP + 8 * n) = make_float2(o[mt][n][2], o[mt][n][3]);
    }
  }
  __syncthreads();
  constexpr int TR = D / 4;  // threads of a row, 4 values each
  float* part = reinterpret_cast<float*>(smem + kNarrowPart<D, MT>);
  float2* part_ml = reinterpret_cast<float2*>(part + R * D);
  for (int r = threadIdx.x / TR; r < R; r += kWarps * 32 / TR) {
    const int pr = r0 + r;
    if (pr >= npairs) break;
    const int col = (threadIdx.x % TR) * 4;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][r]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][r] - base);
      const float4 v = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + w * kNarrowSums<D, MT>) + r * OP + col);
      ll += f * s_l[w][r];
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    if (ncl > 1) {
      *reinterpret_cast<float4*>(part + r * D + col) = acc;
      if (col == 0) part_ml[r] = make_float2(mm, ll);
      continue;
    }
    const int i = pr / a.group;
    const int t = t0 + i, h = hk * a.group + pr - i * a.group;
    if (a.slots == 1) {
      const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;  // a row that sees no key is 0
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + t * a.ldo + h * D + col);
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF>(acc.x * inv, acc.y * inv), pack2<BF>(acc.z * inv, acc.w * inv));
    } else {
      const int64_t at = (static_cast<int64_t>(slot) * a.rows + t) * a.heads + h;
      if (any) *reinterpret_cast<float4*>(a.part_o + at * D + col) = acc;  // without keys its weight is 0
      if (col == 0) a.part_ml[at] = make_float2(mm, ll);
    }
  }
  if (ncl > 1) {
    // the cluster's parts: CTA k finishes rows k, k + ncl, ...
    cluster_sync();
    for (int r = split + ncl * (threadIdx.x / TR); r < R && r0 + r < npairs; r += ncl * (kWarps * 32 / TR)) {
      const int col = (threadIdx.x % TR) * 4;
      float2 ml[8];
      float4 v[8];
      float mm = -INFINITY;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < ncl) {
          ml[k] = ld_cluster2(mapa_rank(part_ml + r, k));
          v[k] = ld_cluster4(mapa_rank(part + r * D + col, k));
          mm = fmaxf(mm, ml[k].x);
        }
      const float base = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < ncl) {
          const float f = ex2(ml[k].x - base);
          ll += f * ml[k].y;
          acc.x += f * v[k].x;
          acc.y += f * v[k].y;
          acc.z += f * v[k].z;
          acc.w += f * v[k].w;
        }
      const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
      const int i = (r0 + r) / a.group;
      const int t = t0 + i, h = hk * a.group + (r0 + r) - i * a.group;
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + t * a.ldo + h * D + col);
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF>(acc.x * inv, acc.y * inv), pack2<BF>(acc.z * inv, acc.w * inv));
    }
    cluster_sync();  // no CTA leaves while its part is read
  }
  if (waits) grid_wait();
}

// ----------------------------------------------------------------- join --
// The parts of one (row, head): weights 2^(m_s - m) of the slots, then the
// weighted sum of their f32 parts over the joined sum. `warps` warps of a CTA
// take the slots of a pair in turn, eight loads at a time (a lone row split
// over a hundred parts would else wait for them one after the other), and
// meet in shared memory. Bound by reading the parts, which the L2 still
// holds.
template <bool BF, int D>
__global__ void __launch_bounds__(256) attn_paged_join(const __grid_constant__ PagedAttnArgs a, int warps) {
  constexpr int V = D / 32;
  __shared__ __align__(16) float s_acc[8][D];
  __shared__ float2 s_ml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = warp % warps;
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * (8 / warps) + warp / warps;
  grid_wait();
  const int64_t pairs = static_cast<int64_t>(min(max(__ldg(a.kv.cu + a.kv.nseq), 0), a.rows)) * a.heads;
  const int64_t step = static_cast<int64_t>(a.rows) * a.heads;
  const bool live = pair < pairs;
  // this warp's slots: w, w + warps, ..., at most 16 (128 slots, 8 warps)
  const int mine = live ? (a.slots - w + warps - 1) / warps : 0;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < mine) ml = a.part_ml[(w + lane * warps) * step + pair];
  float mm = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float wt = ex2(ml.x - (mm == -INFINITY ? 0.f : mm));
  float ll = lane < mine ? wt * ml.y : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
  float acc[V] = {};
  for (int s = 0; s < mine; s += 8) {
    float ws[8];
    alignas(16) float v[8][V];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      ws[k] = __shfl_sync(0xffffffffu, wt, (s + k) & 31);
      if (s + k >= mine) ws[k] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = 0.f;
      if (ws[k] != 0.f) {  // a part without keys may hold no sums
        const float* src = a.part_o + ((w + (s + k) * warps) * step + pair) * D + lane * V;
        if constexpr (V == 4)
          *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(src);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += ws[k] * v[k][i];
  }
  if (warps > 1) {
    if (lane == 0) s_ml[warp] = make_float2(mm, ll);
#pragma unroll
    for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
    __syncthreads();
    if (w != 0) return;
    for (int k = 0; k < warps; ++k) mm = fmaxf(mm, s_ml[warp + k].x);
    const float base = mm == -INFINITY ? 0.f : mm;
    ll = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int k = 0; k < warps; ++k) {
      const float f = ex2(s_ml[warp + k].x - base);
      if (f == 0.f) continue;
      ll += f * s_ml[warp + k].y;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += f * s_acc[warp + k][lane * V + i];
    }
  }
  if (!live) return;
  const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
  const int64_t t = pair / a.heads;
  const int h = static_cast<int>(pair - t * a.heads);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + t * a.ldo + h * D + lane * V);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) dst[i] = pack2<BF>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
}

// ----------------------------------------------------------------- host --

// Parts per row at most: few rows may have many (long keys are split over
// the SMs), many rows few. rows * paged_slots(rows) does not fall as rows
// rise past kPartRows, and is at most kPartRows or 2 rows.
constexpr int kPartRows = 2048;
constexpr int kMaxSlots = 128;
// Bytes of the prefix that a small call may read once per sequence instead
// of once for all, and that few-row tiles of all rows may read instead of the
// tensor-core tiles, which take some 8 us to start and end (8 sequences of 4
// heads behind 2000 rows, 8 key heads: 10.9 us against 13.0; behind 8000:
// 19.0 against 13.9).
constexpr int64_t kReadAgain = 32 << 20;
constexpr int64_t kFewRowPrefix = 24 << 20;
static int paged_slots(int rows) { return std::min(kMaxSlots, std::max(2, kPartRows / std::max(1, rows))); }

size_t attn_paged_bytes(const PagedArgs& p, int rows, int heads) {
  const size_t most = std::max<size_t>(2 * static_cast<size_t>(rows),
                                       std::min<size_t>(kPartRows, static_cast<size_t>(rows) * kMaxSlots));
  return most * heads * (static_cast<size_t>(p.dim) * 4 + 8) + 256;
}

// The few-row tiles that run beside the tensor-core tiles, in microseconds:
// their CTAs (three on an SM), one CTA's time, and the SM time of their bytes.
struct Beside {
  double ctas, each, sm_us;
};

// Parts of a wide call's keys: the count that ends first by a model in
// microseconds. A CTA takes `fixed` to start and end and `per_block` for each
// of its key blocks. The few-row tiles beside take the SMs that it leaves;
// those that are left over when it ends take a CTA's time more (their
// lengths are known to the device alone: half the table's rows is assumed,
// so a count that makes the wide part itself 1.6 times longer than need be
// is out). A join takes 4 us (a call that is joined anyway has it whatever
// the count), and parts are written and read back at about 4 TB/s. Fewer
// parts pay `fixed` less often, more fill the GPU.
static int wide_splits(int64_t items, int ctas, int64_t blocks, double per_block, bool joined, const Beside& few,
                       int64_t rows_heads, int dim, int most) {
  const double fixed = 8.0, sms = sm_count();
  double least = 0.0;
  int best = 1;
  for (int pass = 0; pass < 2; ++pass) {  // the shortest wide part, then the choice
    double got = 0.0;
    for (int n = 1; n <= most && (n == 1 || n <= blocks); ++n) {
      const double one = static_cast<double>((blocks + n - 1) / n) * per_block + fixed;
      const double all = static_cast<double>(items) * n * ctas;
      const double alone = std::ceil(all / sms) * one;
      if (pass == 0) {
        if (n == 1 || alone < least) least = alone;
      } else if (alone <= 1.6 * least) {
        double t = std::max(alone, (all * one + few.sm_us) / sms);
        if (few.ctas > 0.0) {
          const double slots = 3.0 * std::max(0.0, sms - all);  // beside
          const double late = few.ctas - slots * (std::floor(alone / few.each) + 1.0);
          t = std::max(t, late > 0.0 ? alone + few.each * std::max(1.0, late / (3.0 * sms))
                                     : few.each * std::ceil(few.ctas / slots));
        }
        if (n > 1 || joined) t += 4.0 + n * static_cast<double>(rows_heads) * dim * 8 / 4e6;
        if (got == 0.0 || t < got) {
          got = t;
          best = n;
        }
      }
    }
  }
  return best;
}

// Parts of the keys of `tiles` few-row tiles of `keys` keys, `of_seq` of them
// with the same keys: the count that ends first by a model in microseconds.
// 64 keys (a granule of each warp) take a CTA 0.95, or their share of 6.6
// TB/s among the CTAs that run with it (`per_sm` on an SM; tiles with the
// same keys find them in the L2), both slowing it where they are alike. A
// CTA takes 2.3 more to start and end beside others, 3.5 in the last wave,
// which also waits for its slowest SM, the fuller it is the longer. (300
// sequences of 2000 keys, one key head: one part 53 us, three 62; 64 of them:
// five parts 15.9, eight 20; two of 60000, 32 key heads: 279, as two waves of
// CTAs of like length 320.)
static int few_row_parts(int64_t tiles, int64_t of_seq, int64_t keys, int dim, int per_sm, bool joined,
                         int64_t rows_heads, int most) {
  const double slots = static_cast<double>(per_sm) * sm_count(), alone = 0.95 / 64;
  auto share = [&](double ctas) { return ctas * (4 * dim) / 6.6e6 / std::min<double>(static_cast<double>(of_seq), 3.0); };
  double got = 0.0;
  int best = 1;
  for (int n = 1; n <= most && (n == 1 || keys > 256 * static_cast<int64_t>(n - 1)); ++n) {
    const double each = 64.0 * std::ceil(static_cast<double>(keys) / (64.0 * n)), all = static_cast<double>(tiles) * n;
    const double full = std::ceil(all / slots) - 1.0, last = all - full * slots;
    const double key = std::sqrt(std::hypot(alone * alone, share(last) * share(last))) * (1.0 + 0.2 * std::pow(last / slots, 4));
    const double t = full * (2.3 + each * std::max(alone, share(slots))) + 3.5 + each * key +
                     (n > 1 || joined ? 4.0 + n * static_cast<double>(rows_heads) * dim * 8 / 4e6 : 0.0);
    if (n == 1 || t < got) {
      got = t;
      best = n;
    }
  }
  return best;
}

template <bool BF, int D, int MT>
static cudaError_t launch_narrow(const PagedAttnArgs& a, unsigned grid, unsigned cluster, cudaStream_t s) {
  constexpr int smem = kNarrowSmem<D, MT>;
  static PerDevice<cudaError_t> once;
  const cudaError_t* attr = once.get([] {
    return cudaFuncSetAttribute(attn_paged_narrow<BF, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr == nullptr) return cudaErrorNoDevice;
  if (*attr != cudaSuccess) return *attr;
  return launch_early(attn_paged_narrow<BF, D, MT>, grid, kWarps * 32, smem, s, cluster, a);
}

template <bool BF, int D>
static cudaError_t launch_paged_t(PagedAttnArgs& a, cudaStream_t s) {
  const int hk = a.kv.kv_heads, P = a.kv.prefix_len;
  const int64_t pairs = static_cast<int64_t>(a.rows) * a.group, all = static_cast<int64_t>(a.rows) * a.heads;
  const int seqs = std::min(a.kv.nseq, a.rows);
  const int most = paged_slots(a.rows);
  const int tokens = wide_tokens(a.group);
  cudaError_t e = cudaSuccess;
  auto block_us = [](bool pair) { return D == 64 ? 0.7 : pair ? 0.8 : 0.75; };  // measured
  auto join = [&] {
    const int warps = a.slots > 32 ? 8 : a.slots > 16 ? 4 : a.slots > 8 ? 2 : 1;
    return launch_early(attn_paged_join<BF, D>, static_cast<unsigned>((all * warps + 7) / 8), 256, 0, s, 1, a, warps);
  };
  auto place_parts = [&] {
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<int64_t>(a.slots) * a.rows * a.heads * D);
  };
  if (tokens > 0 && pairs >= 64 * static_cast<int64_t>(seqs)) {
    // many rows per sequence: a sequence's tiles walk [prefix, own keys]. The
    // CTAs stay for several items, as pairs, if there are items enough (the
    // sequences taken as equal) and the keys fit the L2 (129 MB): then in
    // order of tiles, a sequence's last ones, which see the most keys, of all
    // heads first. Three prompts of 1250 rows behind 2048, 8 key heads: 158 us
    // against 172 with an item a CTA, and 167 with single CTAs; of 700 behind
    // 905, 32 key heads (54 MB): 66 against 79. Else the tiles of one head run
    // together, which read the same keys, and single CTAs need no partner in
    // step: four images of 1024 rows behind 4114, 32 heads (134 MB): 255
    // against 265 as pairs, and 284 if they stay
    const int64_t blocks = (static_cast<int64_t>(P) + 127) / 128 + (static_cast<int64_t>(a.kv.table_rows) + 127) / 128;
    const double kv_bytes = (P + static_cast<double>(a.kv.nseq) * a.kv.table_rows) * hk * (4 * D);
    const int64_t each = (a.rows + static_cast<int64_t>(seqs) - 1) / seqs;  // rows of a sequence
    auto items = [&](bool pair) { return seqs * ((each + tokens * (pair ? 2 : 1) - 1) / (tokens * (pair ? 2 : 1))) * hk; };
    const bool two_tiles = D == 128 && pairs > 128 * static_cast<int64_t>(seqs);
    const bool stay = kv_bytes <= (96 << 20) && items(two_tiles) > sm_count() / (two_tiles ? 2 : 1);
    const bool pair = two_tiles && stay;
    const int per = tokens * (pair ? 2 : 1);
    const int64_t tiles = a.rows / per + seqs;
    if (tiles > 0x3fffffff / kMaxSlots) return cudaErrorInvalidValue;
    a.slots = stay ? 1 : wide_splits(items(pair), pair ? 2 : 1, blocks, block_us(pair), false, Beside{0, 0, 0}, all, D, most);
    place_parts();
    e = launch_attn_wide(a, stay ? WIDE_STAY : WIDE_JOINT, pair, static_cast<int>(tiles), a.slots, s);
    return e != cudaSuccess || a.slots == 1 ? e : join();
  }
  // tiles of 16 rows, or of 32 where a sequence has more and there are tiles
  // enough for all SMs (its keys are then copied into shared memory half as
  // often: 64 sequences of 5 x 4 rows, 500 keys: 38 us against 44; with few
  // tiles the longer ones only take longer: 16 of 5 x 7 rows: 25 against 23)
  const bool two = pairs > 16 * static_cast<int64_t>(seqs) && (pairs / 32 + seqs) * hk >= 3 * static_cast<int64_t>(sm_count());
  const int R = two ? 32 : 16;
  auto narrow = [&](int64_t grid, int64_t cluster) {
    const unsigned g = static_cast<unsigned>(grid), c = static_cast<unsigned>(cluster);
    return two ? launch_narrow<BF, D, 2>(a, g, c, s) : launch_narrow<BF, D, 1>(a, g, c, s);
  };
  const int64_t own_tiles = pairs / R + seqs;
  a.own_tiles = static_cast<int>(own_tiles);
  // a small call: one launch in which every sequence reads the prefix itself,
  // while its CTAs have so few keys each that parts and their join take
  // longer (one sequence, 8 key heads, 2000 keys: 8.9 us against 9.1, 4000:
  // 12.0 against 9.4). Where SMs have several CTAs that is sooner if a prefix
  // is then read once (two sequences behind 1000 keys, 32 key heads: 10.8
  // against 9.4), later if not (one of 4000 keys: 14.1 against 16.6)
  const double again = static_cast<double>(own_tiles) * hk * P * (4 * D);  // bytes of that
  const int64_t keys = static_cast<int64_t>(P) + a.kv.table_rows;
  int64_t ncl = std::min<int64_t>(3 * static_cast<int64_t>(sm_count()) / (own_tiles * hk), keys / 64);
  ncl = ncl >= 8 ? 8 : ncl >= 4 ? 4 : ncl >= 2 ? 2 : 1;
  const int64_t each_most = ncl == 1 ? 1024 : own_tiles * hk * ncl <= sm_count() ? 384 : P > 0 ? 256 : 640;
  if (again <= kReadAgain && keys <= each_most * ncl && own_tiles * hk * ncl <= 0x7fffffff) {
    a.cluster = static_cast<int>(ncl);
    a.own_splits = 1;
    a.slots = 1;
    a.first = 1;
    return narrow(own_tiles * hk * ncl, ncl);
  }
  // few rows per sequence: the prefix for the rows of all sequences, each
  // sequence's own keys for its own
  const int per_sm = two ? 2 : D == 128 ? 3 : 4;  // few-row CTAs on an SM
  auto part_keys = [](int64_t keys, int64_t n) { return static_cast<int>(((keys + n - 1) / n + kGran - 1) / kGran * kGran); };
  // of the own keys beside tensor-core tiles: CTAs for two waves of three per
  // SM, none of fewer than 256 keys
  auto beside_parts = [&](int cap) {
    const int64_t n = std::min<int64_t>((6 * static_cast<int64_t>(sm_count()) + own_tiles * hk - 1) / (own_tiles * hk),
                                        (static_cast<int64_t>(a.kv.table_rows) + 255) / 256);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, cap)));
  };
  // bytes that few-row tiles of the prefix read
  const double again_few = static_cast<double>((pairs + R - 1) / R) * P * hk * (4 * D);
  const bool wide = P > 0 && tokens > 0 && pairs > R && again_few > kFewRowPrefix;
  const bool pair = D == 128 && pairs > 128;
  const int per = tokens * (pair ? 2 : 1);
  const int64_t each = (a.rows + static_cast<int64_t>(seqs) - 1) / seqs;
  const int64_t of_seq = (each * a.group + R - 1) / R, live = seqs * of_seq * hk;  // few-row tiles, the rows shared evenly
  int wide_tiles = 0;
  if (wide) {
    wide_tiles = (a.rows + per - 1) / per;
    // a few-row CTA takes 4 us to start and end and 0.95 per 64 keys
    const double half = 0.5 * a.kv.table_rows;
    const int cut = beside_parts(most - 1);
    const double keys_each = std::max(half / cut, std::min(half, 256.0));
    const Beside few{static_cast<double>(live) * std::ceil(half / keys_each),
                     4.0 + 0.95 * keys_each / 64, half * seqs * hk * (4.0 * D) / 30e3};
    a.pre_splits = wide_splits(static_cast<int64_t>(wide_tiles) * hk, pair ? 2 : 1, (static_cast<int64_t>(P) + 127) / 128,
                               block_us(pair), true, few, all, D, most - 1);
  } else if (P > 0) {
    a.pre_tiles = static_cast<int>((pairs + R - 1) / R);
    a.pre_splits = few_row_parts(static_cast<int64_t>(a.pre_tiles) * hk, a.pre_tiles, P, D, per_sm, true, all, most - 1);
    a.pre_keys = part_keys(P, a.pre_splits);
  }
  a.own_splits = wide ? beside_parts(most - a.pre_splits)
                      : few_row_parts(live, of_seq, a.kv.table_rows, D, per_sm, P > 0, all, most - a.pre_splits);
  a.own_keys = part_keys(a.kv.table_rows, a.own_splits);
  a.slots = a.pre_splits + a.own_splits;
  place_parts();
  const int64_t gx = hk * (static_cast<int64_t>(a.pre_tiles) * a.pre_splits +
                           static_cast<int64_t>(a.own_tiles) * a.own_splits);
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  if (wide && (e = launch_attn_wide(a, WIDE_PREFIX, pair, wide_tiles, a.pre_splits, s)) != cudaSuccess) return e;
  a.first = !wide;
  e = narrow(gx, 1);
  return e != cudaSuccess || a.slots == 1 ? e : join();
}

cudaError_t launch_attn_paged(const PagedArgs& p, int rows, int heads, const void* q, int64_t ldq, void* out,
                              int64_t ldo, bool causal, const uint32_t* vis, float scale, void* ws, cudaStream_t s) {
  PagedAttnArgs a{};
  a.kv = p;
  a.q = q;
  a.out = out;
  a.ldq = ldq;
  a.ldo = ldo;
  a.rows = rows;
  a.heads = heads;
  a.group = heads / p.kv_heads;
  a.causal = causal;
  a.vis = vis;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.part_o = static_cast<float*>(ws);
  const bool bf = p.dt == DT_BF16;
  if (p.dim == 128) return bf ? launch_paged_t<true, 128>(a, s) : launch_paged_t<false, 128>(a, s);
  return bf ? launch_paged_t<true, 64>(a, s) : launch_paged_t<false, 64>(a, s);
}

}  // namespace qi21
