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
constexpr int kRopeBatch = 4;        // units in flight per thread
constexpr int kRopeMaxCs = 4096;     // (cos, sin) pairs of a CTA: 32 KB
constexpr int kRopeMaxRows = 64;     // rows of a CTA

// Division by an invariant d < 2^20 of n < 2^20: n * ceil(2^40 / d) >> 40
// (the multiplier is over by less than 1, so the quotient by less than
// n / 2^40 < 1 / d: exact).
struct FastDiv {
  uint64_t m;
  uint32_t d;
};
static FastDiv fast_div(uint32_t d) { return FastDiv{((1ull << 40) + d - 1) / d, d}; }
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return static_cast<uint32_t>((n * f.m) >> 40);
}

struct RopeArgs {
  RopeDev r;
  const void* x;  // keys, in an append
  void* out;
  const void* v;  // append only
  int64_t ldx, ldo, ldv;
  const int64_t* pos;
  int rows, heads, dim, rpc;  // rpc: rows of a CTA
  int head_units, v_units;    // units of a head of x, 16-byte (or smaller) pieces of a head of v
  float sgn;                  // -1 for the gradient
  FastDiv by_row, by_head;
  PagedArgs p;  // append only
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

// A CTA takes rpc rows; a thread walks units of them, kRopeBatch at a time
// with the loads of a batch ahead of its arithmetic (the first batch's ahead
// of the angles too). A unit is one piece of E values of a head, or in the
// HALF layout of the turned part the two pieces whose values pair up. The
// rows' (cos, sin) are made once per row and shared by its heads.
// What bounds it: the bytes of x and out; the angles cost rot / 2 of about
// 40 instructions per row.
template <typename T, bool HALF, int E, bool VECT, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];  // [rpc][rot / 2]
  __shared__ int64_t s_dst[kRopeMaxRows];  // append: row of the pool, or -1
  __shared__ int64_t s_pos[kRopeMaxRows];  // append without positions: the row's
  const int tid = threadIdx.x;
  const int row0 = static_cast<int>(blockIdx.x) * a.rpc;
  const int nrow = min(a.rpc, a.rows - row0);
  const int hp = a.r.rot >> 1;
  const uint32_t per_row = a.by_row.d;  // units of a row (x, then v)
  const uint32_t total = static_cast<uint32_t>(nrow) * per_row;
  const uint32_t xu = static_cast<uint32_t>(a.heads) * a.head_units;  // units of x in a row
  const int turn_units = HALF ? hp / E : (a.r.rot + E - 1) / E;       // those of a head that turn

  using P = Piece<T, E, VECT>;
  struct Where {
    int row, col, kind;  // kind 0: turned, 1: copied, 2: v copied
    int c;               // first column within the head
  };
  auto locate = [&](uint32_t u) {
    Where w;
    w.row = static_cast<int>(div_by(u, a.by_row));
    const uint32_t q = u - static_cast<uint32_t>(w.row) * per_row;
    if (!APPEND || q < xu) {
      const uint32_t h = div_by(q, a.by_head);
      const int i = static_cast<int>(q - h * a.head_units);
      if (i < turn_units) {
        w.kind = 0;
        w.c = i * E;
      } else {
        w.kind = 1;
        w.c = HALF ? a.r.rot + (i - turn_units) * E : i * E;
      }
      w.col = static_cast<int>(h) * a.dim + w.c;
    } else {
      const uint32_t q2 = q - xu;
      w.kind = 2;
      w.c = 0;
      w.col = static_cast<int>(q2) * E;
    }
    return w;
  };
  auto load = [&](const Where& w, P& p0, P& p1) {
    const T* src = w.kind == 2 ? static_cast<const T*>(a.v) + (row0 + w.row) * a.ldv + w.col
                               : static_cast<const T*>(a.x) + (row0 + w.row) * a.ldx + w.col;
    p0.load(src);
    if (HALF && w.kind == 0) p1.load(src + hp);
  };

  P b0[kRopeBatch], b1[kRopeBatch];
  Where at[kRopeBatch];
#pragma unroll
  for (int i = 0; i < kRopeBatch; ++i) {
    const uint32_t u = tid + i * kRopeThreads;
    if (u < total) {
      at[i] = locate(u);
      load(at[i], b0[i], b1[i]);
    }
  }

  if (APPEND) {
    const int warp = tid >> 5, lane = tid & 31;
    for (int r = warp; r < nrow; r += kRopeThreads / 32) {
      const int t = row0 + r;
      const int b = warp_find_seq(a.p.cu, a.p.nseq, t, lane);
      if (lane == 0) {
        int64_t dst = -1;
        int own = 0;
        if (b < a.p.nseq) {
          own = __ldg(a.p.lens + b) - (__ldg(a.p.cu + b + 1) - t);
          dst = paged_row(a.p, b, own, &s_rope_status);
        }
        s_dst[r] = dst;
        s_pos[r] = static_cast<int64_t>(a.p.prefix_len) + own;
      }
    }
    if (a.pos == nullptr) __syncthreads();
  }
  for (int i = tid; i < nrow * hp; i += kRopeThreads) {
    const int r = i / hp, j = i - r * hp;
    const int64_t ps = APPEND && a.pos == nullptr
                           ? s_pos[r]
                           : __ldg(reinterpret_cast<const long long*>(a.pos) +
                                   static_cast<int64_t>(row0 + r) * a.r.naxes + a.r.axis[j]);
    const float2 z = cos_sin_turns(static_cast<uint64_t>(ps) * a.r.turns[j]);
    cs[i] = make_float2(z.x * a.r.scale, z.y * a.r.scale * a.sgn);
  }
  __syncthreads();

  for (uint32_t u0 = tid; u0 < total; u0 += kRopeBatch * kRopeThreads) {
    if (u0 != static_cast<uint32_t>(tid)) {
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i) {
        const uint32_t u = u0 + i * kRopeThreads;
        if (u < total) {
          at[i] = locate(u);
          load(at[i], b0[i], b1[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (u0 + i * kRopeThreads >= total) break;
      const Where& w = at[i];
      T* dst;
      if (APPEND) {
        const int64_t row = s_dst[w.row];
        if (row < 0) continue;
        dst = static_cast<T*>(a.out) + row * a.ldo + (w.kind == 2 ? a.heads * a.dim : 0) + w.col;
      } else {
        dst = static_cast<T*>(a.out) + (row0 + w.row) * a.ldo + w.col;
      }
      if (w.kind == 0) {
        const float2* z = cs + w.row * hp + (HALF ? w.c : w.c / 2);
        if constexpr (HALF) {
          P o0, o1;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float p = widen(b0[i].e[e]), q = widen(b1[i].e[e]);
            const float2 g = z[e];
            o0.e[e] = narrow<T>(p * g.x - q * g.y);
            o1.e[e] = narrow<T>(p * g.y + q * g.x);
          }
          o0.store(dst);
          o1.store(dst + hp);
        } else {
          P o = b0[i];
          const int live = a.r.rot - w.c;  // the rest of the piece does not turn
#pragma unroll
          for (int e = 0; e + 1 < E; e += 2) {
            if (e < live) {
              const float p = widen(b0[i].e[e]), q = widen(b0[i].e[e + 1]);
              const float2 g = z[e / 2];
              o.e[e] = narrow<T>(p * g.x - q * g.y);
              o.e[e + 1] = narrow<T>(p * g.y + q * g.x);
            }
          }
          o.store(dst);
        }
      } else {
        b0[i].store(dst);
      }
    }
  }
}

template <typename T, bool HALF, int E, bool VECT, bool APPEND>
static cudaError_t launch_t(RopeArgs& a, bool inplace, cudaStream_t s) {
  const int hp = a.r.rot / 2;
  if (HALF)
    a.head_units = hp / E + (inplace ? 0 : (a.dim - a.r.rot) / E);
  else
    a.head_units = inplace ? (a.r.rot + E - 1) / E : a.dim / E;
  a.v_units = APPEND ? a.dim / E : 0;
  const int64_t per_row = static_cast<int64_t>(a.heads) * (a.head_units + a.v_units);
  a.by_row = fast_div(static_cast<uint32_t>(per_row));
  a.by_head = fast_div(static_cast<uint32_t>(a.head_units));
  // rows of a CTA: about two batches of units per thread, fewer while that
  // would leave SMs without a CTA, and no more than the (cos, sin) room
  int64_t rpc = 2 * kRopeBatch * kRopeThreads / per_row;
  rpc = std::min<int64_t>(rpc, a.rows / (2 * sm_count()));
  if (hp > 0) rpc = std::min<int64_t>(rpc, kRopeMaxCs / hp);
  a.rpc = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rpc, kRopeMaxRows)));
  const unsigned grid = static_cast<unsigned>((a.rows + static_cast<int64_t>(a.rpc) - 1) / a.rpc);
  rope_kernel<T, HALF, E, VECT, APPEND>
      <<<grid, kRopeThreads, static_cast<size_t>(a.rpc) * hp * sizeof(float2), s>>>(a);
  return cudaGetLastError();
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
