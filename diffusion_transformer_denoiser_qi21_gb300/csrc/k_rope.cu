// Rotary positions of row vectors, and the append of new keys (turned on
// the way) and values to a paged K/V cache. Both move every value once and
// turn it by its row's angle:
//   (a, b) -> s (a cos - b sin, a sin + b cos),  angle_j = pos f_j
// (gradient: the angle negated). The angle of pair j is kept as turns per
// position in 64-bit fixed point, F_j = f_j / 2 pi * 2^64, so pos * F_j
// modulo 2^64 is the angle with its whole turns taken off, exactly, for
// every int64 position: one integer product instead of an f64 product and
// reduction (f64 arithmetic is slow here, and an f32 angle of position 10^6
// is off by 0.03 rad). cos and sin are then taken in f32 of the remainder
// of at most an eighth of a turn either way.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace qi21 {

static __device__ unsigned int s_rope_status = 0;

unsigned int rope_status_read_clear() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, s_rope_status, sizeof v);
  cudaMemcpyToSymbol(s_rope_status, &z, sizeof z);
  return v;
}

constexpr int kRopeThreads = 256;
// heads of a thread's batch: 64 bytes of 16-byte pieces
template <bool HALF>
constexpr int kRopeBatch = HALF ? 2 : 4;
constexpr int kRopeStages = 2;       // batches under way per thread (three: the same; four: one CTA an SM fewer, 83 us)
constexpr int kRopeMaxCs = 4096;     // (cos, sin) pairs of a CTA: 32 KB
constexpr int kRopeMaxRows = 64;     // rows of a CTA

struct RopeArgs {
  RopeDev r;
  const void* x;  // keys, in an append
  void* out;
  const void* v;  // append only
  int64_t ldx, ldo, ldv;
  const int64_t* pos;
  int rows, heads, dim;
  int rpc;         // rows of a CTA
  int units;       // of a head (see the kernel)
  int head_lanes;  // threads that share a row's column piece
  float sgn;       // -1 for the gradient
  int cs_floats;   // of a CTA's (cos, sin)
  PagedArgs p;     // append only
};

template <typename T>
__device__ __forceinline__ float widen(T v) {
  if constexpr (std::is_same<T, __half>::value)
    return __half2float(v);
  else if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return __bfloat162float(v);
  else
    return v;
}
// Two neighbouring values of a piece, rounded together: one conversion of
// both runs at the arithmetic rate, two single ones at a quarter of it.
template <typename T>
__device__ __forceinline__ void put2(T* e, float lo, float hi) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = pack2<std::is_same<T, __nv_bfloat16>::value>(lo, hi);
    memcpy(e, &w, 4);
  } else {
    e[0] = lo;
    e[1] = hi;
  }
}
template <typename T>
__device__ __forceinline__ T narrow(float v) {
  if constexpr (std::is_same<T, __half>::value)
    return __float2half_rn(v);
  else if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return __float2bfloat16_rn(v);
  else
    return v;
}

// E neighbouring values, moved as one piece of E * sizeof(T) bytes if VECT
// (then aligned to it), else one by one.
template <typename T, int E, bool VECT>
struct Piece {
  alignas(VECT ? sizeof(T) * E : sizeof(T)) T e[E];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VECT && sizeof(T) * E == 16)
      *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (VECT && sizeof(T) * E == 8)
      *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    else if constexpr (VECT && sizeof(T) * E == 4)
      *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
    else
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = p[i];
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VECT && sizeof(T) * E == 16)
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    else if constexpr (VECT && sizeof(T) * E == 8)
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
    else if constexpr (VECT && sizeof(T) * E == 4)
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(e);
    else
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = e[i];
  }
};

// cos and sin of `turns` / 2^64 of a turn. The nearest quarter is taken off,
// so the remainder has 30 bits and its f32 value is off by 2^-27 half turns.
__device__ __forceinline__ float2 cos_sin_turns(uint64_t turns) {
  const int h = static_cast<int>(turns >> 32);
  const unsigned qd = (static_cast<unsigned>(h) + (1u << 29)) >> 30;
  const int rest = static_cast<int>(static_cast<unsigned>(h) - (qd << 30));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  const float cc = (qd & 1) ? s : c, ss = (qd & 1) ? c : s;
  return make_float2((qd + 1) & 2 ? -cc : cc, qd & 2 ? -ss : ss);
}

// The places of rows [row0, row0 + n) in the cache, n <= 64, by one warp: the
// first row's sequence by a search of all of them, the others' by a search
// of the next 32 sequences' numbers, held by the lanes (and of all where that
// is short).
__device__ __forceinline__ void append_places(const PagedArgs& p, int row0, int n, int lane, int64_t* dst, int64_t* pos) {
  const int b0 = warp_find_seq(p.cu, p.nseq, row0, lane);
  const bool is = b0 + lane < p.nseq;
  const int beg = is ? __ldg(p.cu + b0 + lane) : 0x7fffffff;
  const int end = is ? __ldg(p.cu + b0 + lane + 1) : 0x7fffffff;
  const int len = is ? __ldg(p.lens + b0 + lane) : 0;
  for (int base = 0; base < n; base += 32) {
    const int t = row0 + base + lane;
    int k = 0;  // ends that are <= t, of the 32
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      if (__shfl_sync(0xffffffffu, end, k + s - 1) <= t) k += s;
    const bool past = __shfl_sync(0xffffffffu, end, 31) <= t;
    const int c0 = __shfl_sync(0xffffffffu, beg, k);  // of the row's sequence b0 + k
    const int c1 = __shfl_sync(0xffffffffu, end, k);
    int b = c0 <= t && t < c1 ? b0 + k : p.nseq;
    int own = __shfl_sync(0xffffffffu, len, k) - (c1 - t);
    for (unsigned left = __ballot_sync(0xffffffffu, past && base + lane < n); left; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const int at = warp_find_seq(p.cu, p.nseq, row0 + base + l, lane);
      if (lane == l) {
        b = at;
        if (b < p.nseq) own = __ldg(p.lens + b) - (__ldg(p.cu + b + 1) - t);
      }
    }
    if (base + lane < n) {
      dst[base + lane] = b < p.nseq ? paged_row(p, b, own, &s_rope_status) : -1;
      pos[base + lane] = static_cast<int64_t>(p.prefix_len) + own;
    }
  }
}

// A CTA takes rpc rows. A head is cut into units: one piece of E values, or
// in the HALF layout's turned part the two pieces whose values pair up. A
// thread has one unit of every head_lanes-th head of a row (of the keys'
// heads, then the values' in an append), so it reads the (cos, sin) of its
// columns once per row and turns several heads with them. Its pieces of the
// next two batches of heads are under way into a ring of its own in shared
// memory (registers hold one batch only, and the SM then waits for memory
// between its arithmetic: 88 us against 82 below), the first ones ahead of
// the angles, and four CTAs share an SM. What bounds it: the bytes of x and
// out. 32768 rows of 32 heads of 128 (bf16, 537 MB): 82 us, 6.6 TB/s; in a
// stream of calls, where a kernel starts while the one before it ends, 78 us,
// a copy's rate (4099 rows of 16 f32 heads: 12.2 us against 14.3); with (cos,
// sin) read per head, conflicting banks and the frequencies read per angle,
// 118.
template <typename T, bool HALF, int E, bool VECT, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float cs[];  // [rpc][cos, sin][rot / 2]
  __shared__ int64_t s_dst[kRopeMaxRows];  // append: row of the pool, or -1
  __shared__ int64_t s_pos[kRopeMaxRows];  // append without positions: the row's
  using P = Piece<T, E, VECT>;
  constexpr int Z = HALF ? E : (E + 1) / 2;  // pairs of a unit
  constexpr int NB = kRopeBatch<HALF>;
  const int tid = threadIdx.x;
  const int row0 = static_cast<int>(blockIdx.x) * a.rpc;
  const int nrow = min(a.rpc, a.rows - row0);
  const int hp = a.r.rot >> 1;
  const int heads = APPEND ? 2 * a.heads : a.heads;

  // this thread's unit and its first row and head
  const int tpr = a.units * a.head_lanes;  // threads of a row
  const int step = kRopeThreads / tpr;     // rows at once
  const int first = tid / tpr;
  const int lane_h = (tid - first * tpr) / a.units;
  const int unit = tid - first * tpr - lane_h * a.units;
  const int turn_units = HALF ? hp / E : (a.r.rot + E - 1) / E;
  const bool turns = unit < turn_units;
  const int col = turns || !HALF ? unit * E : a.r.rot + (unit - turn_units) * E;
  const int live = a.r.rot - col;  // values of an interleaved piece that turn
  const bool two = HALF && turns;
  const bool active = first < step;

  // A thread's batches (NB heads of a row) follow each other by rows, then
  // heads. 16-byte pieces go to a ring of the thread's own in shared memory,
  // kRopeStages batches ahead; smaller ones to registers, one batch ahead
  constexpr bool RING = VECT && sizeof(T) * E == 16;
  constexpr int NP = HALF ? 2 * NB : NB;  // pieces of a batch
  P b0[NB], b1[NB];
  uint4* ring = reinterpret_cast<uint4*>(cs + a.cs_floats) + tid;
  auto load = [&](int row, int h0, int st) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int h = h0 + k * a.head_lanes;
      if (h < heads) {
        const T* src = APPEND && h >= a.heads
                           ? static_cast<const T*>(a.v) + row * a.ldv + (h - a.heads) * a.dim + col
                           : static_cast<const T*>(a.x) + row * a.ldx + h * a.dim + col;
        if constexpr (RING) {
          cp_async16(smem_u32(ring + (st * NP + k) * kRopeThreads), src);
          if (two) cp_async16(smem_u32(ring + (st * NP + NB + k) * kRopeThreads), src + hp);
        } else {
          b0[k].load(src);
          if (two) b1[k].load(src + hp);
        }
      }
    }
  };
  // the batch under way furthest ahead, and its stage
  int fr = first, fh = lane_h;
  auto fetch_next = [&](int st) {
    if (active && fr < nrow) {
      load(row0 + fr, fh, st);
      fh += NB * a.head_lanes;
      if (fh >= heads) {
        fh = lane_h;
        fr += step;
      }
    }
    if constexpr (RING) cp_async_commit();
  };
  constexpr int ST = RING ? kRopeStages : 1;
  grid_wait();  // the above touches no memory of a kernel before this one
  grid_release();
#pragma unroll
  for (int k = 0; k < ST; ++k) fetch_next(k);
  int st = 0;

  if (APPEND) {
    if (tid < 32) append_places(a.p, row0, nrow, tid, s_dst, s_pos);
    if (a.pos == nullptr) __syncthreads();
  }
  // a thread keeps one pair: its frequency is read once (the parameter
  // memory serves lanes that read different words one after the other)
  if (hp > 0) {
    const int r1 = tid / hp, j = tid - r1 * hp;
    if (r1 < kRopeThreads / hp) {
      const uint64_t turns_j = a.r.turns[j];
      const int axis = a.r.axis[j];
      // a unit of 8 pairs is read as two pieces of 4: the pieces of
      // neighbouring units side by side keep the reads off each other's banks
      const int at = Z == 8 ? ((j & 4 ? turn_units : 0) + (j >> 3)) * 4 + (j & 3) : j;
      for (int r = r1; r < nrow; r += kRopeThreads / hp) {
        const int64_t ps = APPEND && a.pos == nullptr
                               ? s_pos[r]
                               : __ldg(reinterpret_cast<const long long*>(a.pos) +
                                       static_cast<int64_t>(row0 + r) * a.r.naxes + axis);
        const float2 z = cos_sin_turns(static_cast<uint64_t>(ps) * turns_j);
        cs[r * 2 * hp + at] = z.x * a.r.scale;
        cs[r * 2 * hp + at + hp] = z.y * a.r.scale * a.sgn;
      }
    }
  }
  __syncthreads();
  if (!active) return;

  for (int r = first; r < nrow; r += step) {
    alignas(16) float zc[Z], zs[Z];
    if (turns) {
      if constexpr (Z >= 4) {
        const float* src = cs + r * 2 * hp + unit * 4;
        if (HALF || live >= E) {
          // hp and with it every address is a multiple of 4 values here: in
          // the HALF layout by the choice of E, else if the head turns whole
          // units (a unit that turns in part reads its pairs one by one)
#pragma unroll
          for (int i = 0; i < Z; i += 4) {
            if ((hp & 3) == 0) {
              *reinterpret_cast<float4*>(zc + i) = *reinterpret_cast<const float4*>(src + i * turn_units);
              *reinterpret_cast<float4*>(zs + i) = *reinterpret_cast<const float4*>(src + hp + i * turn_units);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                zc[i + k] = src[i * turn_units + k];
                zs[i + k] = src[hp + i * turn_units + k];
              }
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < Z; ++k)
            if (2 * k < live) {
              zc[k] = src[k];
              zs[k] = src[hp + k];
            }
        }
      } else {
        const float* src = cs + r * 2 * hp + unit * Z;
#pragma unroll
        for (int k = 0; k < Z; ++k)
          if (HALF || 2 * k < live) {
            zc[k] = src[k];
            zs[k] = src[hp + k];
          }
      }
    }
    T* dst0;
    if (APPEND) {
      dst0 = static_cast<T*>(a.out) + s_dst[r] * a.ldo + col;
      if (s_dst[r] < 0) dst0 = nullptr;
    } else {
      dst0 = static_cast<T*>(a.out) + (row0 + r) * a.ldo + col;
    }
    for (int h0 = lane_h; h0 < heads; h0 += NB * a.head_lanes) {
      if constexpr (RING) {
        cp_async_wait<ST - 1>();
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          if (h0 + k * a.head_lanes >= heads) break;
          *reinterpret_cast<uint4*>(b0[k].e) = ring[(st * NP + k) * kRopeThreads];
          if (two) *reinterpret_cast<uint4*>(b1[k].e) = ring[(st * NP + NB + k) * kRopeThreads];
        }
        fetch_next(st);
        if (++st == ST) st = 0;
      } else if (r != first || h0 != lane_h) {
        fetch_next(0);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int h = h0 + k * a.head_lanes;
        if (h >= heads || (APPEND && dst0 == nullptr)) break;
        T* dst = dst0 + h * a.dim;  // the values' heads follow the keys' in a cache row
        if (turns && !(APPEND && h >= a.heads)) {
          if constexpr (HALF) {
            if constexpr (E == 1) {
              const float p = widen(b0[k].e[0]), q = widen(b1[k].e[0]);
              b0[k].e[0] = narrow<T>(p * zc[0] - q * zs[0]);
              b1[k].e[0] = narrow<T>(p * zs[0] + q * zc[0]);
            } else {
#pragma unroll
              for (int e = 0; e < E; e += 2) {
                const float p0 = widen(b0[k].e[e]), q0 = widen(b1[k].e[e]);
                const float p1 = widen(b0[k].e[e + 1]), q1 = widen(b1[k].e[e + 1]);
                put2(&b0[k].e[e], p0 * zc[e] - q0 * zs[e], p1 * zc[e + 1] - q1 * zs[e + 1]);
                put2(&b1[k].e[e], p0 * zs[e] + q0 * zc[e], p1 * zs[e + 1] + q1 * zc[e + 1]);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e + 1 < E; e += 2) {
              if (e < live) {
                const float p = widen(b0[k].e[e]), q = widen(b0[k].e[e + 1]);
                put2(&b0[k].e[e], p * zc[e / 2] - q * zs[e / 2], p * zs[e / 2] + q * zc[e / 2]);
              }
            }
          }
        }
        b0[k].store(dst);
        if (two) b1[k].store(dst + hp);
      }
    }
  }
}

template <typename T, bool HALF, int E, bool VECT, bool APPEND>
static cudaError_t launch_t(RopeArgs& a, bool inplace, cudaStream_t s) {
  const int hp = a.r.rot / 2;
  if (HALF)
    a.units = hp / E + (inplace ? 0 : (a.dim - a.r.rot) / E);
  else
    a.units = inplace ? (a.r.rot + E - 1) / E : a.dim / E;
  const int heads = APPEND ? 2 * a.heads : a.heads;
  // one batch of heads per thread and row; calls of few rows spread a row
  // over all threads of a CTA
  const int few = 2 * sm_count();
  const int lanes = a.rows < few ? heads : (heads + kRopeBatch<HALF> - 1) / kRopeBatch<HALF>;
  a.head_lanes = std::max(1, std::min(lanes, kRopeThreads / a.units));
  const int at_once = kRopeThreads / (a.units * a.head_lanes);
  // rows of a CTA: four rounds of its threads (a rotation of 36384 rows of 16
  // heads: 48 us; eight rounds: 50, one: 58; an append of as many bytes: 51
  // us, eight rounds: 53, sixteen: 60), fewer while that would leave SMs
  // idle, and no more than the (cos, sin) room
  int64_t rpc = static_cast<int64_t>(at_once) * 4;
  rpc = std::min<int64_t>(rpc, a.rows / few);
  if (hp > 0) rpc = std::min<int64_t>(rpc, kRopeMaxCs / hp);
  a.rpc = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rpc, kRopeMaxRows)));
  const unsigned grid = static_cast<unsigned>((a.rows + static_cast<int64_t>(a.rpc) - 1) / a.rpc);
  a.cs_floats = (a.rpc * hp * 2 + 3) & ~3;
  constexpr bool RING = VECT && sizeof(T) * E == 16;
  constexpr int ring = RING ? kRopeStages * (HALF ? 2 : 1) * kRopeBatch<HALF> * kRopeThreads * 16 : 0;
  if (RING) {
    static PerDevice<cudaError_t> once;
    const cudaError_t* attr = once.get([] {
      return cudaFuncSetAttribute(rope_kernel<T, HALF, E, VECT, APPEND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  ring + kRopeMaxCs * 8);
    });
    if (attr == nullptr) return cudaErrorNoDevice;
    if (*attr != cudaSuccess) return *attr;
  }
  return launch_early(rope_kernel<T, HALF, E, VECT, APPEND>, grid, kRopeThreads, a.cs_floats * sizeof(float) + ring, s, 1, a);
}

// The widest piece that the layout and the alignment allow: 16 bytes, a
// pair, or single values. `bits` has every pointer and every stride in bytes
// or-ed together.
template <typename T, bool APPEND>
static cudaError_t launch_e(RopeArgs& a, bool half, bool inplace, uint64_t bits, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int hp = a.r.rot / 2;
  if (half && hp > 0) {
    if (bits % 16 == 0 && hp % V == 0 && a.dim % V == 0) return launch_t<T, true, V, true, APPEND>(a, inplace, s);
    if (bits % (2 * sizeof(T)) == 0 && hp % 2 == 0) return launch_t<T, true, 2, true, APPEND>(a, inplace, s);
    return launch_t<T, true, 1, true, APPEND>(a, inplace, s);
  }
  if (bits % 16 == 0 && a.dim % V == 0) return launch_t<T, false, V, true, APPEND>(a, inplace, s);
  if (bits % (2 * sizeof(T)) == 0) return launch_t<T, false, 2, true, APPEND>(a, inplace, s);
  return launch_t<T, false, 2, false, APPEND>(a, inplace, s);
}

template <typename T>
static cudaError_t launch_rope_t(RopeArgs& a, bool half, cudaStream_t s) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                        (static_cast<uint64_t>(a.ldx | a.ldo) * sizeof(T));
  return launch_e<T, false>(a, half, a.x == a.out, bits, s);
}

cudaError_t launch_rope(const RopeDev& r, bool half, int elem, int rows, int heads, int dim, const void* x,
                        int64_t ldx, void* out, int64_t ldo, const int64_t* pos, bool grad, cudaStream_t s) {
  RopeArgs a{};
  a.r = r;
  a.x = x;
  a.out = out;
  a.ldx = ldx;
  a.ldo = ldo;
  a.pos = pos;
  a.rows = rows;
  a.heads = heads;
  a.dim = dim;
  a.sgn = grad ? -1.f : 1.f;
  if (elem == 2) return launch_rope_t<__half>(a, half, s);
  if (elem == 3) return launch_rope_t<__nv_bfloat16>(a, half, s);
  return launch_rope_t<float>(a, half, s);
}

cudaError_t launch_kv_append(const PagedArgs& p, const RopeDev& r, bool half, int rows, const void* k, int64_t ldk,
                             const void* v, int64_t ldv, const int64_t* pos, cudaStream_t s) {
  RopeArgs a{};
  a.r = r;
  a.x = k;
  a.out = p.pool;
  a.v = v;
  a.ldx = ldk;
  a.ldo = 2 * static_cast<int64_t>(p.kv_heads) * p.dim;
  a.ldv = ldv;
  a.pos = pos;
  a.rows = rows;
  a.heads = p.kv_heads;
  a.dim = p.dim;
  a.sgn = 1.f;
  a.p = p;
  const uint64_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                        reinterpret_cast<uintptr_t>(p.pool) | (static_cast<uint64_t>(ldk | ldv) * 2);
  if (p.dt == DT_BF16) return launch_e<__nv_bfloat16, true>(a, half, false, bits, s);
  return launch_e<__half, true>(a, half, false, bits, s);
}

}  // namespace qi21
