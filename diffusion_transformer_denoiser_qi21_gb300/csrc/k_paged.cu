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
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// A CTA takes a tile of 16 MT (row, head) pairs of one key head and a run of
// keys, the prefix's or a sequence's own. Its four warps take granules of 16
// keys in turn, each through a ring of its own (16-byte asynchronous copies,
// rows behind the end filled with zeros), so no warp waits for another: a
// granule is Q K^T, the running maximum and sum, and P V, by m16n8k16 MMAs
// with P taken from the score registers. The warps' parts are joined at the
// end. It is bound by the bytes of K and V: a tile has few rows, so the
// 128-row tensor-core tiles would be nearly empty.
template <int D>
constexpr int kNarrowStages = D == 128 ? 3 : 4;
template <int D>
constexpr int kNarrowSmem = kWarps * kNarrowStages<D> * 2 * kGran * D * 2;

template <bool BF, int D, int MT>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_narrow(const __grid_constant__ PagedAttnArgs a) {
  constexpr int R = 16 * MT;
  constexpr int NST = kNarrowStages<D>;
  constexpr int HALF = kGran * D * 2;  // bytes of a granule's K (or V)
  constexpr int CH = D / 8;            // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y;
  int x = blockIdx.x;

  // the tile: pairs [r0, r0 + nr) of the rows [t0, ...), the keys' source
  // and their number for each row
  const bool pre = x < a.pre_tiles * a.pre_splits;
  int t0 = 0, npairs, r0, split, nsplit, slot, len = 0, nrows = 0;
  const int32_t* pages;
  const int P = a.kv.prefix_len;
  if (pre) {
    const int tile = x / a.pre_splits;
    split = x - tile * a.pre_splits;
    nsplit = a.pre_splits;
    slot = split;
    pages = a.kv.prefix_pages;
    npairs = min(max(__ldg(a.kv.cu + a.kv.nseq), 0), a.rows) * a.group;
    r0 = tile * R;
  } else {
    x -= a.pre_tiles * a.pre_splits;
    const int tile = x / a.own_splits;
    split = x - tile * a.own_splits;
    nsplit = a.own_splits;
    slot = a.pre_splits + split;
    int b, at;
    warp_find_tile(a, tile, a.group, R, lane, b, at);
    if (b >= a.kv.nseq) return;
    t0 = __ldg(a.kv.cu + b);
    nrows = seq_rows(a, b);
    npairs = nrows * a.group;
    r0 = at * R;
    pages = a.kv.table + static_cast<int64_t>(b) * a.kv.table_stride;
    len = __ldg(a.kv.lens + b);
    if ((len < nrows || len > a.kv.table_rows) && threadIdx.x == 0) atomicOr(&s_paged_status, kStatusPage);
    len = min(max(len, 0), a.kv.table_rows);
  }
  if (r0 >= npairs) return;

  // this thread's rows: lane / 4 and + 8 of each 16-row tile
  const int tq = lane >> 2, tj = lane & 3;
  int lim[MT][2];  // keys of this part that the row sees
  uint32_t qf[MT][D / 16][4];
  int most = 0;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pr = r0 + mt * 16 + tq + 8 * e;
      const bool live = pr < npairs;
      const int i = live ? pr / a.group : 0;
      const int t = t0 + i;
      const int h = hk * a.group + (live ? pr - i * a.group : 0);
      int n = 0;
      if (live) {
        if (pre)
          n = a.vis ? static_cast<int>(min(__ldg(a.vis + t), static_cast<uint32_t>(P))) : P;
        else if (a.vis)
          n = static_cast<int>(min(__ldg(a.vis + t), static_cast<uint32_t>(P) + len)) - P;
        else
          n = a.causal ? len - nrows + i + 1 : len;
        n = min(max(n, 0), pre ? P : len);
      }
      lim[mt][e] = n;
      most = max(most, n);
      const uint32_t* qr = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                             static_cast<int64_t>(t) * a.ldq + h * D);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[mt][k][e] = live ? __ldg(qr + 8 * k + tj) : 0u;
        qf[mt][k][2 + e] = live ? __ldg(qr + 8 * k + 4 + tj) : 0u;
      }
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));

  // this warp's granules of the split: g0, g0 + 4, ... below g1
  const int ng = (most + kGran - 1) / kGran;
  const int g0 = static_cast<int>(static_cast<int64_t>(ng) * split / nsplit) + warp;
  const int g1 = static_cast<int>(static_cast<int64_t>(ng) * (split + 1) / nsplit);
  const uint8_t* ring = smem + warp * (NST * 2 * HALF);
  const uint32_t sring = smem_u32(ring);
  const uint16_t* pool = static_cast<const uint16_t*>(a.kv.pool);
  const int64_t row_elems = 2 * static_cast<int64_t>(a.kv.kv_heads) * D;

  auto page_of = [&](int g) { return __ldg(pages + g * kGran / a.kv.page_rows); };
  auto fetch = [&](int g, int id, int st) {
    const bool ok = id >= 0 && id < a.kv.npages;
    if (!ok && lane == 0) atomicOr(&s_paged_status, kStatusPage);
    const int64_t row = static_cast<int64_t>(ok ? id : 0) * a.kv.page_rows + g * kGran % a.kv.page_rows;
    const uint16_t* base = pool + row * row_elems + hk * D;
    const uint32_t d0 = sring + st * 2 * HALF;
#pragma unroll
    for (int i = 0; i < 2 * kGran * CH / 32; ++i) {
      const int u = i * 32 + lane;
      const int kv = u / (kGran * CH), w = u % (kGran * CH);
      const int r = w / CH, c = w % CH;
      const bool live = ok && g * kGran + r < most;
      const uint16_t* src = live ? base + r * row_elems + (kv ? a.kv.kv_heads * D : 0) + c * 8 : pool;
      cp_async16(d0 + kv * HALF + r * (D * 2) + ((c ^ (r & 7)) << 4), src, live);
    }
  };

  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2];
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
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) {
    if (nf < g1) {
      const int id = nid, g = nf;
      nf += kWarps;
      if (nf < g1) nid = page_of(nf);
      fetch(g, id, s);
    }
    cp_async_commit();
  }
  int st = 0;
  for (int g = g0; g < g1; g += kWarps) {
    cp_async_wait<NST - 2>();
    __syncwarp();
    {
      int fs = st + NST - 1;
      if (fs >= NST) fs -= NST;
      if (nf < g1) {
        const int id = nid, gg = nf;
        nf += kWarps;
        if (nf < g1) nid = page_of(nf);
        fetch(gg, id, fs);
      }
      cp_async_commit();
    }
    const uint32_t sk = sring + st * 2 * HALF, sv = sk + HALF;
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
      const int key = (lane >> 4) * 8 + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
      ldsm4<false>(sk + key * (D * 2) + ((c ^ (key & 7)) << 4), b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816<BF>(s[mt][0], qf[mt][k], b[0], b[1]);
        mma16816<BF>(s[mt][1], qf[mt][k], b[2], b[3]);
      }
    }
    uint32_t p[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float al[2];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // scores in log2 units; what the row does not see is taken out
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& v = s[mt][n][2 * e + c];
            v = g * kGran + 8 * n + 2 * tj + c < lim[mt][e] ? v * a.scale_log2 : -INFINITY;
            mx = fmaxf(mx, v);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the maximum is raised only past the threshold: o and l share it
        al[e] = 1.f;
        if (mx > m[mt][e] + kPagedRescale) {
          al[e] = ex2(m[mt][e] - mx);
          m[mt][e] = mx;
          moved = true;
        }
        const float base = m[mt][e] == -INFINITY ? 0.f : m[mt][e];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(s[mt][n][2 * e] - base), p1 = ex2(s[mt][n][2 * e + 1] - base);
          sum += p0 + p1;
          // P is rounded to the values' type for the MMA (half a step of a
          // weight each, of either sign); l sums the f32 weights
          p[mt][2 * n + e] = pack2<BF>(p0, p1);
        }
        l[mt][e] = l[mt][e] * al[e] + sum;
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
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      const int key = ((lane >> 3) & 1) * 8 + (lane & 7), c = 2 * n + (lane >> 4);
      ldsm4<true>(sv + key * (D * 2) + ((c ^ (key & 7)) << 4), b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816<BF>(o[mt][2 * n], p[mt], b[0], b[1]);
        mma16816<BF>(o[mt][2 * n + 1], p[mt], b[2], b[3]);
      }
    }
    __syncwarp();  // the stage is refilled next round
  }
  cp_async_wait<0>();

  // join the four warps: each leaves its sums in its ring
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[mt][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (tj == 0) {
        s_m[warp][mt * 16 + tq + 8 * e] = m[mt][e];
        s_l[warp][mt * 16 + tq + 8 * e] = sum;
      }
    }
  constexpr int OP = D + 4;  // row pitch of the f32 sums: spreads the rows over the banks
  static_assert(16 * MT * OP * 4 <= NST * 2 * HALF, "the sums fit the ring");
  float* so = reinterpret_cast<float*>(smem + warp * (NST * 2 * HALF));
  __syncwarp();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      *reinterpret_cast<float2*>(so + (mt * 16 + tq) * OP + 8 * n + 2 * tj) = make_float2(o[mt][n][0], o[mt][n][1]);
      *reinterpret_cast<float2*>(so + (mt * 16 + tq + 8) * OP + 8 * n + 2 * tj) = make_float2(o[mt][n][2], o[mt][n][3]);
    }
  __syncthreads();
  constexpr int TR = D / 4;  // threads of a row, 4 values each
  for (int r = threadIdx.x / TR; r < R; r += kWarps * 32 / TR) {
    const int pr = r0 + r;
    if (pr >= npairs) break;
    const int c = (threadIdx.x % TR) * 4;
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
          reinterpret_cast<const float*>(smem + w * (NST * 2 * HALF)) + r * OP + c);
      ll += f * s_l[w][r];
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    const int i = pr / a.group;
    const int t = t0 + i, h = hk * a.group + pr - i * a.group;
    if (a.slots == 1) {
      const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;  // a row that sees no key is 0
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + t * a.ldo + h * D + c);
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF>(acc.x * inv, acc.y * inv), pack2<BF>(acc.z * inv, acc.w * inv));
    } else {
      const int64_t at = (static_cast<int64_t>(slot) * a.rows + t) * a.heads + h;
      *reinterpret_cast<float4*>(a.part_o + at * D + c) = acc;
      if (c == 0) a.part_ml[at] = make_float2(mm, ll);
    }
  }
}

// ----------------------------------------------------------------- join --
// One warp per (row, head): weights 2^(m_s - m) of the slots, then the
// weighted sum of their f32 parts over the joined sum. Bound by reading the
// parts, which the L2 still holds.
template <bool BF, int D>
__global__ void __launch_bounds__(256) attn_paged_join(const __grid_constant__ PagedAttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t pairs = static_cast<int64_t>(min(max(__ldg(a.kv.cu + a.kv.nseq), 0), a.rows)) * a.heads;
  if (pair >= pairs) return;
  const int64_t step = static_cast<int64_t>(a.rows) * a.heads;
  float mm = -INFINITY;
  for (int s = lane; s < a.slots; s += 32) mm = fmaxf(mm, a.part_ml[s * step + pair].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float base = mm == -INFINITY ? 0.f : mm;
  constexpr int V = D / 32;
  float acc[V] = {};
  float ll = 0.f;
  for (int s0 = 0; s0 < a.slots; s0 += 32) {
    float w = 0.f;
    if (s0 + lane < a.slots) {
      const float2 ml = a.part_ml[(s0 + lane) * step + pair];
      w = ex2(ml.x - base);
      ll += w * ml.y;
    }
    const int n = min(32, a.slots - s0);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      if (ws == 0.f) continue;  // a part without keys may hold no sums
      const float* src = a.part_o + ((s0 + s) * step + pair) * D + lane * V;
      if (V == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] += ws * v.x;
        acc[1] += ws * v.y;
        acc[2 % V] += ws * v.z;
        acc[3 % V] += ws * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] += ws * v.x;
        acc[1] += ws * v.y;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
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
static int paged_slots(int rows) { return std::min(kMaxSlots, std::max(2, kPartRows / std::max(1, rows))); }

size_t attn_paged_bytes(const PagedArgs& p, int rows, int heads) {
  const size_t most = std::max<size_t>(2 * static_cast<size_t>(rows),
                                       std::min<size_t>(kPartRows, static_cast<size_t>(rows) * kMaxSlots));
  return most * heads * (static_cast<size_t>(p.dim) * 4 + 8) + 256;
}

// Parts of a wide call's keys: the count that ends first, by a model of one
// item's time in key blocks (its blocks, and about four of set-up and end)
// over the waves of items, plus the parts' write and read back at about
// 6 TB/s against 0.8 us a block.
static int wide_splits(int64_t items, int64_t blocks, int64_t slots, int64_t rows_heads, int dim, int most) {
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= most && n <= blocks; ++n) {
    const double t = static_cast<double>((items * n + slots - 1) / slots) * ((blocks + n - 1) / n + 4) +
                     (n > 1 ? n * static_cast<double>(rows_heads) * dim * 8 / 4.8e6 : 0.0);
    if (n == 1 || t < least) {
      best = n;
      least = t;
    }
  }
  return best;
}

template <bool BF, int D>
static cudaError_t launch_paged_t(PagedAttnArgs& a, cudaStream_t s) {
  constexpr int smem = kNarrowSmem<D>;
  static PerDevice<cudaError_t> once;
  const cudaError_t* attr = once.get([] {
    return cudaFuncSetAttribute(attn_paged_narrow<BF, D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr == nullptr) return cudaErrorNoDevice;
  if (*attr != cudaSuccess) return *attr;
  const int hk = a.kv.kv_heads, P = a.kv.prefix_len;
  const int64_t pairs = static_cast<int64_t>(a.rows) * a.group, all = static_cast<int64_t>(a.rows) * a.heads;
  const int seqs = std::min(a.kv.nseq, a.rows);
  const int most = paged_slots(a.rows);
  const int tokens = a.kv.npages > 0 ? wide_tokens(a.group) : 0;
  cudaError_t e = cudaSuccess;
  auto join = [&] {
    attn_paged_join<BF, D><<<static_cast<unsigned>((all + 7) / 8), 256, 0, s>>>(a);
    return cudaGetLastError();
  };
  auto place_parts = [&] {
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<int64_t>(a.slots) * a.rows * a.heads * D);
  };
  if (tokens > 0 && pairs >= 64 * static_cast<int64_t>(seqs)) {
    // many rows per sequence: a sequence's tiles walk [prefix, own keys]
    const bool pair = D == 128 && pairs > 128 * static_cast<int64_t>(seqs);
    const int per = tokens * (pair ? 2 : 1);
    const int64_t tiles = a.rows / per + seqs;
    const int64_t blocks = (static_cast<int64_t>(P) + 127) / 128 + (static_cast<int64_t>(a.kv.table_rows) + 127) / 128;
    if (tiles > 0x3fffffff / kMaxSlots) return cudaErrorInvalidValue;
    a.slots = wide_splits(tiles * hk, blocks, sm_count() / (pair ? 2 : 1), all, D, most);
    place_parts();
    e = launch_attn_wide(a, WIDE_JOINT, pair, static_cast<int>(tiles), a.slots, s);
    return e != cudaSuccess || a.slots == 1 ? e : join();
  }
  // few rows per sequence: the prefix for the rows of all sequences, each
  // sequence's own keys for its own
  const int R = 16;
  a.own_tiles = static_cast<int>(pairs / R + seqs);
  // narrow splits: enough CTAs for two waves of two per SM, none of fewer
  // than 256 keys
  const int64_t want = 4 * static_cast<int64_t>(sm_count());
  auto splits = [&](int64_t tiles, int64_t keys, int cap) {
    const int64_t n = std::min<int64_t>((want + tiles * hk - 1) / (tiles * hk), (keys + 255) / 256);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, cap)));
  };
  const bool wide = P > 0 && tokens > 0 && pairs > R;
  const bool pair = D == 128 && pairs > 128;
  const int per = tokens * (pair ? 2 : 1);
  int wide_tiles = 0;
  if (wide) {
    wide_tiles = (a.rows + per - 1) / per;
    a.pre_splits = wide_splits(static_cast<int64_t>(wide_tiles) * hk, (static_cast<int64_t>(P) + 127) / 128,
                               sm_count() / (pair ? 2 : 1), all, D, most - 1);
  } else if (P > 0) {
    a.pre_tiles = static_cast<int>((pairs + R - 1) / R);
    a.pre_splits = splits(a.pre_tiles, P, most - 1);
  }
  a.own_splits = splits(a.own_tiles, a.kv.table_rows, most - a.pre_splits);
  a.slots = a.pre_splits + a.own_splits;
  place_parts();
  if (wide && (e = launch_attn_wide(a, WIDE_PREFIX, pair, wide_tiles, a.pre_splits, s)) != cudaSuccess) return e;
  const int64_t gx = static_cast<int64_t>(a.pre_tiles) * a.pre_splits + static_cast<int64_t>(a.own_tiles) * a.own_splits;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  attn_paged_narrow<BF, D, 1><<<dim3(static_cast<unsigned>(gx), hk), kWarps * 32, smem, s>>>(a);
  e = cudaGetLastError();
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
