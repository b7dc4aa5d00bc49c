// Attention over a paged cache for tiles of many rows, on the 5th-generation
// tensor cores. A tile is 128 (row, head) pairs of one key head: whole
// tokens, their query heads next to each other, so a TMA box of the q tensor
// is a tile of Q and the heads of a group share every key block. The tile's
// rows come from one sequence and walk [prefix, own keys] (WIDE_JOINT), or
// they are the rows of all sequences and walk the prefix (WIDE_PREFIX); its
// key blocks may be split over CTAs, whose parts are joined later.
//
// 12 warps, as in the attention over one contiguous prefix, with a second
// loading warp:
//   warps 0,11 TMA: Q and 128-key blocks of K, and of V, into rings, each as
//              boxes of neighbouring rows of one page (as many as the page
//              size and 64 allow). Boxes behind the end are zeros. The rows
//              of a V box behind the end within a page are whatever the page
//              held (0 times a NaN is a NaN, so a weight of 0 does not take
//              them out): that one box is copied by the warp with zeros in
//              their place.
//   warp 1     S_j = Q K_j^T into one of three TMEM buffers
//   warp 10    O += P_j V_j, P read from TMEM
//   warps 2-9  softmax, 16 TMEM lanes (rows) each
// With PAIR a cluster of two CTAs takes two tiles through the pair MMA
// (M 256), each CTA holding half of every key block, so a block crosses from
// L2 into each SM once per 256 rows; that pays when there are rows for two
// tiles. A single CTA (M 128) takes all rows of a block itself. Bound by the
// tensor cores and the softmax between them when the rows are many, by the
// bytes of K and V when one tile holds them all. Every wait is bounded.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn.cuh"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace qi21 {

static __device__ unsigned int s_wide_status = 0;

unsigned int wide_status_read_clear() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, s_wide_status, sizeof v);
  cudaMemcpyToSymbol(s_wide_status, &z, sizeof z);
  return v;
}

constexpr int kWK = 128;                 // keys per block
constexpr int kWBoxShift = 6;            // log2 of the rows per K / V box at most
constexpr int kWThreads = 384;            // 12 warps
constexpr int kWNS = 3;                  // S / P buffers in TMEM

template <int D, bool PAIR>
struct Wide {
  static constexpr int kCols = D / 64;                     // 64-column pieces of a head
  static constexpr int kQ = kCols * 128 * 128;             // bytes of a Q tile
  static constexpr int kKeysK = PAIR ? 64 : 128;           // keys of a block in this CTA's K
  static constexpr int kColsV = PAIR ? 1 : kCols;          // column pieces in this CTA's V
  static constexpr int kK = kKeysK * D * 2;
  static constexpr int kV = 128 * 128 * kColsV;
  static constexpr int kStages = kK + kV > 32768 ? 3 : 6;  // of either ring
  static constexpr int kOffK = kQ;
  static constexpr int kOffV = kOffK + kStages * kK;
  static constexpr int kOffBar = kOffV + kStages * kV;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static_assert((3 + 4 * kStages + 3 * kWNS) * 8 + 16 <= 512, "barrier area");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct WideArgs {
  PagedAttnArgs a;
  CUtensorMap qmap;   // q [rows][heads][dim], box tokens x group x 64 columns
  CUtensorMap kvmap;  // pool [npages * page_rows][2 * kv_heads * dim], box br x 64
  int tokens;         // of a CTA's tile
  int br_shift;       // log2 of the rows of a K / V box
  int joint, splits, tiles;
};

// Transposes the 4 x 4 words of four neighbouring threads (thread j: row j),
// in two rounds of exchanged halves.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int j) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {  // 2 x 2 blocks: words i and i + 1 with thread j ^ 1
    const uint32_t give = j & 1 ? w[i] : w[i + 1];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
    if (j & 1)
      w[i] = got;
    else
      w[i + 1] = got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // the blocks: words i and i + 2 with thread j ^ 2
    const uint32_t give = j & 2 ? w[i] : w[i + 2];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 2);
    if (j & 2)
      w[i] = got;
    else
      w[i + 2] = got;
  }
}

template <bool BF, int D, bool PAIR>
__global__ void __launch_bounds__(kWThreads, 1) attn_paged_wide(const __grid_constant__ WideArgs p) {
  using W = Wide<D, PAIR>;
  constexpr int NK = W::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const PagedAttnArgs& a = p.a;
  const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y;
  constexpr int CT = PAIR ? 2 : 1;  // CTAs (tiles) of an item
  const int item = static_cast<int>(blockIdx.x) / CT;
  // a sequence's last tiles see the most keys: they start first, so that the
  // last wave of CTAs is of short ones
  const int tile = p.tiles - 1 - item % p.tiles, split = item / p.tiles;
  const int P = a.kv.prefix_len;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W::kOffBar);
  uint64_t* qfull = bars;             // even CTA: both Q tiles landed
  uint64_t* vtail = qfull + 1;        // [2] even CTA: the odd CTA's copied V boxes, at most two
  uint64_t* kfull = vtail + 2;        // [NK] even CTA
  uint64_t* vfull = kfull + NK;       // [NK] even CTA
  uint64_t* kempty = vfull + NK;      // [NK] both CTAs: stage's Q K^T done
  uint64_t* vempty = kempty + NK;     // [NK] both CTAs: stage's P V done
  uint64_t* sfull = vempty + NK;      // [kWNS] both CTAs: S_b written
  uint64_t* pfull = sfull + kWNS;     // [kWNS] even CTA: P_b of every CTA written
  uint64_t* pvdone = pfull + kWNS;    // [kWNS] both CTAs: P V of buffer b done
  uint32_t* tslot = reinterpret_cast<uint32_t*>(pvdone + kWNS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);

  if (threadIdx.x == 2 * 32) {
    mbar_init(qfull, 1);
    mbar_init(&vtail[0], 1);
    mbar_init(&vtail[1], 1);
    for (int i = 0; i < NK; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&vfull[i], 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < kWNS; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 8 * CT);  // softmax warps
      mbar_init(&pvdone[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.qmap);
    tma_prefetch_desc(&p.kvmap);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tslot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tslot, 512);
      tmem_relinquish();
    }
  }
  // what came before the call is done from here on; the call's next kernel
  // may start. The item is found by every warp while the barriers and the
  // tensor memory are set up
  grid_wait();
  grid_release();
  // the item: tokens [tok0, tok_end) of this CTA's tile and the keys that its
  // (and its pair's) rows see at most
  int tok0 = 0, tok_end = 0, len = 0, nrows = 0, seq0 = 0;
  const int32_t* own_pages = nullptr;
  if (p.joint) {
    const SeqTile q = warp_find_tile(a, tile, 1, CT * p.tokens, lane);
    seq0 = q.row0;  // no such tile: no rows
    nrows = q.rows;
    tok0 = seq0 + q.at * CT * p.tokens;
    tok_end = seq0 + nrows;
    own_pages = a.kv.table + static_cast<int64_t>(q.b) * a.kv.table_stride;
    len = q.len;
    if (nrows > 0 && (len < nrows || len > a.kv.table_rows) && threadIdx.x == 0)
      atomicOr(&s_wide_status, kStatusPage);
    len = min(max(len, 0), a.kv.table_rows);
  } else {
    tok0 = tile * CT * p.tokens;
    tok_end = min(max(__ldg(a.kv.cu + a.kv.nseq), 0), a.rows);
  }
  // keys of [prefix, own] that token t sees
  const int total = P + len;
  auto limit = [&](int t) {
    int n = total;
    if (a.vis)
      n = static_cast<int>(min(__ldg(a.vis + t), static_cast<uint32_t>(total)));
    else if (a.causal && p.joint)
      n = P + min(max(len - nrows + (t - seq0) + 1, 0), len);
    return n;
  };
  const int item_end = min(tok_end, tok0 + CT * p.tokens);
  int most = 0, least = 0;
  if (a.vis) {
    least = 0x7fffffff;
    for (int t = tok0 + lane; t < item_end; t += 32) {
      most = max(most, limit(t));
      least = min(least, limit(t));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
  } else if (tok0 < item_end) {
    most = limit(item_end - 1);
    least = limit(tok0);
  }
  tok0 += rank * p.tokens;
  // key blocks: the prefix's, then the own keys'; this split's are [j0, j1)
  const int np = min(most, P), no = max(most - P, 0);
  const int npb = (np + kWK - 1) / kWK;
  const int nb = npb + (no + kWK - 1) / kWK;
  const int j0 = static_cast<int>(static_cast<int64_t>(nb) * split / p.splits);
  const int j1 = static_cast<int>(static_cast<int64_t>(nb) * (split + 1) / p.splits);
  const int n = j1 - j0;

  // the loading warps (below) start on their first page ids here
  const bool is_k = warp == 0;
  const int brs = p.br_shift;
  const int keys = is_k ? W::kKeysK : kWK;              // of a block, in this CTA
  const int boxes = keys >> brs;                        // per column piece: 1, 2, 4 or 8
  const int bxs = (is_k && PAIR ? 6 : 7) - brs;         // log2
  const int run = 32 >> bxs;                            // blocks of a run
  const int koff = (is_k ? rank * W::kKeysK : 0) + ((lane & (boxes - 1)) << brs);
  const int none = a.kv.npages * a.kv.page_rows;        // a row behind the pool: zeros
  // this lane's box of the run from block i on: its key (-1: behind the
  // end) and its page id
  int key = -1, id = 0;
  auto ids = [&](int i) {
    const int j = j0 + i + (lane >> bxs);
    const bool pre = j < npb;
    key = (pre ? j : j - npb) * kWK + koff;
    if (i + (lane >> bxs) >= n || key >= (pre ? np : no)) key = -1;
    if (key >= 0) id = __ldg((pre ? a.kv.prefix_pages : own_pages) + key / a.kv.page_rows);
  };
  auto row_of = [&]() {
    if (key < 0) return none;
    if (id < 0 || id >= a.kv.npages) {
      atomicOr(&s_wide_status, kStatusPage);
      return none;
    }
    return id * a.kv.page_rows + key % a.kv.page_rows;
  };
  if (warp == 0 || warp == 11) ids(0);
  tc_fence_before();
  if (PAIR)
    cluster_sync();  // both CTAs' barriers and TMEM ready before any remote use
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tS = tmem;        // S buffers at columns [0, 384)
  const uint32_t tO = tmem + 384;  // O at columns [384, 384 + D)
  const uint32_t tP = tS;          // P_b (16-bit pairs, 64 columns) over the first columns of S_b

  // does block j have a V box that the end cuts (see the producer)?
  auto cut = [&](int j) {
    const bool pre = j < npb;
    const int left = (pre ? np : no) - (pre ? j : j - npb) * kWK;
    return left < kWK && (left & ((1 << p.br_shift) - 1)) != 0;
  };

  // a wait by a whole warp: every lane leaves with the same answer
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &s_wide_status));
  };

  if (warp == 0 || warp == 11) {
    // the two loading warps: Q and the K blocks, and the V blocks. A lane
    // holds the pool row of one box of a run of blocks, the ids of the next
    // run's pages are under way meanwhile, and lane 0 issues the boxes: a
    // block must not wait for its page ids, nor K for V's stage
    if (n > 0) {
      if (is_k && lane == 0) {
        const uint32_t bytes = static_cast<uint32_t>(W::kCols) * p.tokens * a.group * 128;
        if (leader) mbar_arrive_expect_tx(qfull, CT * bytes);
        for (int c = 0; c < W::kCols; ++c) {
          if (PAIR)
            tma_load_3d_pair(smem + c * 16384, &p.qmap, mapa_rank(qfull, 0), c * 64, hk * a.group, tok0);
          else
            tma_load_3d(smem + c * 16384, &p.qmap, qfull, c * 64, hk * a.group, tok0);
        }
      }
      uint64_t* full = is_k ? kfull : vfull;
      uint64_t* empty = is_k ? kempty : vempty;
      const int stage = is_k ? W::kK : W::kV;
      const int cols = is_k ? W::kCols : W::kColsV;
      const int piece = keys * 128;                         // bytes of a column piece
      const int col0 = is_k ? hk * D : a.kv.kv_heads * D + hk * D + (PAIR ? rank * 64 : 0);
      uint8_t* ring = smem + (is_k ? W::kOffK : W::kOffV);
      bool ok = true;
      int rows = none, tails = 0;
      for (int i = 0; i < n && ok; ++i) {
        if ((i & (run - 1)) == 0) {
          rows = row_of();
          ids(i + run);
        }
        const int st = i % NK;
        if (!wait_all(&empty[st], ((i / NK) & 1) ^ 1u)) {
          ok = false;
          break;
        }
        uint8_t* base = ring + st * stage;
        const int at = (i & (run - 1)) << bxs;  // the lane with the block's first box
        int skip = -1;
        if (!is_k && cut(j0 + i)) {
          // the V box that the end cuts, rows behind it zero
          const int j = j0 + i;
          const bool pre = j < npb;
          const int left = (pre ? np : no) - (pre ? j : j - npb) * kWK;
          skip = left >> brs;
          const int live = left - (skip << brs);  // its rows before the end
          const int r0 = __shfl_sync(0xffffffffu, rows, at + skip);
          const uint16_t* src = static_cast<const uint16_t*>(a.kv.pool) +
                                static_cast<int64_t>(r0 == none ? 0 : r0) * (2 * a.kv.kv_heads * D) + col0;
          for (int c = 0; c < cols; ++c) {
            uint8_t* d = base + c * piece + (skip << (brs + 7));
            for (int u0 = lane; u0 < 8 << brs; u0 += 128) {
              uint4 v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = (u0 + 32 * k) >> 3, ch = u0 & 7;
                v[k] = make_uint4(0, 0, 0, 0);
                if (r < live && r0 != none)
                  v[k] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r) * (2 * a.kv.kv_heads * D) +
                                                         c * 64 + ch * 8);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = (u0 + 32 * k) >> 3, ch = u0 & 7;
                *reinterpret_cast<uint4*>(d + r * 128 + ((ch ^ (r & 7)) << 4)) = v[k];
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (PAIR && !leader && lane == 0) mbar_arrive_cluster(mapa_rank(&vtail[tails & 1], 0));
          ++tails;
        }
        if (lane == 0 && leader)
          mbar_arrive_expect_tx(&full[st], CT * (stage - (skip >= 0 ? cols << (brs + 7) : 0)));
        const uint32_t fb = PAIR ? mapa_rank(&full[st], 0) : 0u;
        for (int b = 0; b < boxes; ++b) {
          const int row = __shfl_sync(0xffffffffu, rows, at + b);
          if (lane == 0 && b != skip) {
            uint8_t* d = base + (b << (brs + 7));
            for (int c = 0; c < cols; ++c) {
              if (PAIR)
                tma_load_2d_pair(d + c * piece, &p.kvmap, fb, col0 + c * 64, row);
              else
                tma_load_2d(d + c * piece, &p.kvmap, &full[st], col0 + c * 64, row);
            }
          }
        }
      }
      if (!ok) {
        // gave up: the copies under way land within microseconds, leave
        // them a millisecond before this CTA's memory is given back
        const unsigned long long g0 = globaltimer();
        while (globaltimer() - g0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1 || warp == 10) {
    if (lane == 0 && leader && n > 0) {
      if (warp == 1) {
        constexpr uint32_t idesc = idesc_f16(128 * CT, kWK, false, BF);
        const uint32_t sQ = smem_u32(smem);
        bool ok = mbar_wait(qfull, 0, abort_flag, &s_wide_status);
        for (int i = 0; i < n && ok; ++i) {
          const int b = i % kWNS, st = i % NK;
          // S_b is free once the P V that read P_{i-3} from it is done
          if (i >= kWNS && !mbar_wait(&pvdone[b], ((i - kWNS) / kWNS) & 1, abort_flag, &s_wide_status)) break;
          if (!mbar_wait(&kfull[st], (i / NK) & 1, abort_flag, &s_wide_status)) break;
          tc_fence_after();
          const uint32_t sK = smem_u32(smem + W::kOffK + st * W::kK);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t ad = sdesc_sw128(sQ + (k >> 2) * 16384) + 2 * (k & 3);
            const uint64_t bd = sdesc_sw128(sK + (k >> 2) * (W::kKeysK * 128)) + 2 * (k & 3);
            if (PAIR)
              tc_mma_f16_pair(tS + b * kWK, ad, bd, idesc, k > 0 ? 1u : 0u);
            else
              tc_mma_f16(tS + b * kWK, ad, bd, idesc, k > 0 ? 1u : 0u);
          }
          if (PAIR) {
            tc_commit_pair(&kempty[st], 0x3);
            tc_commit_pair(&sfull[b], 0x3);
          } else {
            tc_commit(&kempty[st]);
            tc_commit(&sfull[b]);
          }
        }
      } else {
        constexpr uint32_t idesc = idesc_f16(128 * CT, D, true, BF);  // V: MN-major
        uint32_t tails = 0;
        for (int i = 0; i < n; ++i) {
          const int b = i % kWNS, st = i % NK;
          if (!mbar_wait(&pfull[b], (i / kWNS) & 1, abort_flag, &s_wide_status)) break;
          if (!mbar_wait(&vfull[st], (i / NK) & 1, abort_flag, &s_wide_status)) break;
          if (PAIR && cut(j0 + i) && !mbar_wait_cluster(&vtail[tails++ & 1], 0, abort_flag, &s_wide_status)) break;
          tc_fence_after();
          const uint32_t sV = smem_u32(smem + W::kOffV + st * W::kV);
#pragma unroll
          for (int k = 0; k < kWK / 16; ++k) {
            // A = P in TMEM (16 keys: 8 columns of pairs); B = V: 16 key rows
            // of 128 bytes, column pieces 16 KB apart, 8-row groups 1 KB
            const uint64_t bd = sdesc(sV + k * 2048, 16384, 1024, 2);
            if (PAIR)
              tc_mma_f16_ts_pair(tO, tP + b * kWK + k * 8, bd, idesc, (i > 0 || k > 0) ? 1u : 0u);
            else
              tc_mma_f16_ts(tO, tP + b * kWK + k * 8, bd, idesc, (i > 0 || k > 0) ? 1u : 0u);
          }
          if (PAIR) {
            tc_commit_pair(&vempty[st], 0x3);
            tc_commit_pair(&pvdone[b], 0x3);
          } else {
            tc_commit(&vempty[st]);
            tc_commit(&pvdone[b]);
          }
        }
      }
    }
  } else {
    // softmax: warps 2-9, two per TMEM lane quadrant, 16 lanes (rows) each;
    // thread t holds rows r0 = base + t/4 and r1 = r0 + 8, columns 8k +
    // 2(t%4) and + 1 of each 8-column group k of a block's scores
    const int q = warp & 3;
    const int hh = (warp - 2) >> 2;
    const int lbase = q * 32 + hh * 16;
    const int tq = lane >> 2, tj = lane & 3;
    const int r0 = lbase + tq, r1 = r0 + 8;
    const int i0 = r0 / a.group, i1 = r1 / a.group;
    const int t0 = tok0 + i0, t1 = tok0 + i1;
    const bool live0 = i0 < p.tokens && t0 < tok_end, live1 = i1 < p.tokens && t1 < tok_end;
    const bool dead = !__any_sync(0xffffffffu, live0 || live1);  // no row of this warp
    const int lim0 = live0 ? limit(t0) : most;
    const int lim1 = live1 ? limit(t1) : most;
    const uint32_t lane_off = static_cast<uint32_t>(lbase) << 16;
    const float c = a.scale_log2;
    const uint64_t c2 = f2(c, c);
    const uint32_t pf_remote = PAIR && !leader ? mapa_rank(pfull, 0) : 0u;
    float m0 = -INFINITY, m1 = -INFINITY;
    uint64_t lacc = 0ull;  // (row r0, row r1) partial sums of this thread's columns
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int b = i % kWNS;
      if (!wait_all(&sfull[b], (i / kWNS) & 1)) {
        ok = false;
        break;
      }
      if (!dead) {
        tc_fence_after();
        uint32_t s[2][32];  // [half of the 128 columns][8 groups x (r0 c, r0 c+1, r1 c, r1 c+1)]
        tmem_ld16x256_x8(tS + b * kWK + lane_off, s[0]);
        tmem_ld16x256_x8(tS + b * kWK + 64 + lane_off, s[1]);
        tmem_ld_wait(s[0]);
        tmem_ld_wait(s[1]);
        // what the rows see of this block: its first e0, e1 keys
        const int j = j0 + i;
        const bool pre = j < npb;
        const int first = pre ? j * kWK : P + (j - npb) * kWK;
        const int e0 = (pre ? min(lim0, P) : lim0) - first, e1 = (pre ? min(lim1, P) : lim1) - first;
        if (min(e0, e1) < kWK) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int g = 0; g < 8; ++g)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int col = hf * 64 + 8 * g + 2 * tj + (e & 1);
                if (col >= ((e & 2) ? e1 : e0)) s[hf][4 * g + e] = __float_as_uint(-INFINITY);
              }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY, my0 = -INFINITY, my1 = -INFINITY;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int g = 0; g < 8; g += 2) {
            mx0 = max3(mx0, __uint_as_float(s[hf][4 * g + 0]), __uint_as_float(s[hf][4 * g + 1]));
            mx1 = max3(mx1, __uint_as_float(s[hf][4 * g + 2]), __uint_as_float(s[hf][4 * g + 3]));
            my0 = max3(my0, __uint_as_float(s[hf][4 * g + 4]), __uint_as_float(s[hf][4 * g + 5]));
            my1 = max3(my1, __uint_as_float(s[hf][4 * g + 6]), __uint_as_float(s[hf][4 * g + 7]));
          }
        mx0 = fmaxf(mx0, my0);
        mx1 = fmaxf(mx1, my1);
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        const float mb0 = mx0 * c, mb1 = mx1 * c;
        // raise each row's running max only past the threshold (O and l share
        // the stale max; p <= 2^threshold stays in f16 range)
        float al0 = 1.f, al1 = 1.f;
        const bool need0 = mb0 > m0 + kPagedRescale, need1 = mb1 > m1 + kPagedRescale;
        if (need0) {
          al0 = ex2(m0 - mb0);
          m0 = mb0;
        }
        if (need1) {
          al1 = ex2(m1 - mb1);
          m1 = mb1;
        }
        {
          float la, lb;
          unf2(lacc, la, lb);
          lacc = f2(la * al0, lb * al1);
        }
        const bool warp_rescale = __any_sync(0xffffffffu, (need0 || need1) && i > 0);
        // a row that has seen no key yet keeps its maximum at -inf and has
        // weights 2^(-inf - 0) = 0. P is rounded to the values' type (half a
        // step of a weight, of either sign); l sums the f32 weights
        const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
        const uint64_t nm0 = f2(n0, n0), nm1 = f2(n1, n1);
        uint32_t pk[32];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            float x0, x1, y0, y1;
            unf2(ffma2(f2(__uint_as_float(s[hf][4 * g + 0]), __uint_as_float(s[hf][4 * g + 1])), c2, nm0), x0, x1);
            unf2(ffma2(f2(__uint_as_float(s[hf][4 * g + 2]), __uint_as_float(s[hf][4 * g + 3])), c2, nm1), y0, y1);
            const float p00 = ex2(x0), p01 = ex2(x1), p10 = ex2(y0), p11 = ex2(y1);
            lacc = fadd2(lacc, f2(p00 + p01, p10 + p11));
            pk[2 * (8 * hf + g)] = pack2<BF>(p00, p01);
            pk[2 * (8 * hf + g) + 1] = pack2<BF>(p10, p11);
          }
        tmem_st16x128_x16(tP + b * kWK + lane_off, pk);
        if (warp_rescale) {
          // O is stable once the P V of block i - 1 is done
          if (!wait_all(&pvdone[(i - 1) % kWNS], ((i - 1) / kWNS) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int hf = 0; hf < W::kCols; ++hf) {
            uint32_t o[32];
            tmem_ld16x256_x8(tO + hf * 64 + lane_off, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              o[4 * g + 0] = __float_as_uint(__uint_as_float(o[4 * g + 0]) * al0);
              o[4 * g + 1] = __float_as_uint(__uint_as_float(o[4 * g + 1]) * al0);
              o[4 * g + 2] = __float_as_uint(__uint_as_float(o[4 * g + 2]) * al1);
              o[4 * g + 3] = __float_as_uint(__uint_as_float(o[4 * g + 3]) * al1);
            }
            tmem_st16x256_x8(tO + hf * 64 + lane_off, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&pfull[b]);
        else
          mbar_arrive_cluster_relaxed(pf_remote + static_cast<uint32_t>(b * 8));
      }
    }
    float l0, l1;
    unf2(lacc, l0, l1);
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (ok && n > 0)
      ok = wait_all(&pvdone[(n - 1) % kWNS], ((n - 1) / kWNS) & 1);
    if (ok && !dead) {
      tc_fence_after();
      const int h0 = hk * a.group + r0 - i0 * a.group, h1 = hk * a.group + r1 - i1 * a.group;
      float odd0 = 0.f, odd1 = 0.f;  // NaN once a sum is not finite
      if (a.slots == 1) {
        const float inv0 = l0 > 0.f || l0 != l0 ? 1.f / l0 : 0.f;  // a row that sees no key is 0
        const float inv1 = l1 > 0.f || l1 != l1 ? 1.f / l1 : 0.f;
        uint16_t* o0 = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(t0) * a.ldo + h0 * D;
        uint16_t* o1 = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(t1) * a.ldo + h1 * D;
#pragma unroll 1
        for (int hf = 0; hf < W::kCols; ++hf) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld16x256_x8(tO + hf * 64 + lane_off, o);
            tmem_ld_wait(o);
          } else {
#pragma unroll
            for (int g = 0; g < 32; ++g) o[g] = 0u;
          }
          // a row's 64 columns sit in four threads as one pair of each group
          // of 8; exchanged, a thread has all of groups tj and tj + 4 and
          // stores 16 bytes at once (the single pairs' stores took 1.2 us)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float x0 = __uint_as_float(o[16 * half + 4 * g + 0]), x1 = __uint_as_float(o[16 * half + 4 * g + 1]);
              const float y0 = __uint_as_float(o[16 * half + 4 * g + 2]), y1 = __uint_as_float(o[16 * half + 4 * g + 3]);
              odd0 = fmaf(0.f, x0 + x1, odd0);
              odd1 = fmaf(0.f, y0 + y1, odd1);
              w0[g] = pack2<BF>(x0 * inv0, x1 * inv0);
              w1[g] = pack2<BF>(y0 * inv1, y1 * inv1);
            }
            quad_transpose(w0, tj);
            quad_transpose(w1, tj);
            const int col = hf * 64 + 32 * half + 8 * tj;
            if (live0) *reinterpret_cast<uint4*>(o0 + col) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
            if (live1) *reinterpret_cast<uint4*>(o1 + col) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
          }
        }
      } else {
        const int64_t at0 = (static_cast<int64_t>(split) * a.rows + t0) * a.heads + h0;
        const int64_t at1 = (static_cast<int64_t>(split) * a.rows + t1) * a.heads + h1;
        if (tj == 0 && live0) a.part_ml[at0] = make_float2(m0, l0);
        if (tj == 0 && live1) a.part_ml[at1] = make_float2(m1, l1);
        if (n > 0) {  // a part without keys has weight 0: its sums are not read
#pragma unroll 1
          for (int hf = 0; hf < W::kCols; ++hf) {
            uint32_t o[32];
            tmem_ld16x256_x8(tO + hf * 64 + lane_off, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const int col = hf * 64 + 8 * g + 2 * tj;
              odd0 = fmaf(0.f, __uint_as_float(o[4 * g + 0]) + __uint_as_float(o[4 * g + 1]), odd0);
              odd1 = fmaf(0.f, __uint_as_float(o[4 * g + 2]) + __uint_as_float(o[4 * g + 3]), odd1);
              if (live0)
                *reinterpret_cast<uint2*>(a.part_o + at0 * D + col) = make_uint2(o[4 * g + 0], o[4 * g + 1]);
              if (live1)
                *reinterpret_cast<uint2*>(a.part_o + at1 * D + col) = make_uint2(o[4 * g + 2], o[4 * g + 3]);
            }
          }
        }
      }
      // A key that some rows of the tile see and others do not has weight 0 in
      // those, but 0 times a value that is not finite is a NaN. Rows with such
      // a sum are done again over the keys that they see alone, if one of the
      // keys between the tile's limits has such a value
      const bool fix0 = live0 && odd0 != odd0 && least < most, fix1 = live1 && odd1 != odd1 && least < most;
      if (__any_sync(0xffffffffu, fix0 || fix1) && n > 0 &&
          odd_values<BF, D>(a, own_pages, hk, least, most, lane)) {
        __syncwarp();  // after the stores above, some of which are replaced
        const int k0 = j0 < npb ? j0 * kWK : P + (j0 - npb) * kWK;             // this split's keys
        const int k1 = j1 <= npb ? min(j1 * kWK, np) : P + min((j1 - npb) * kWK, no);
        for (int e = 0; e < 2; ++e)
          for (unsigned left = __ballot_sync(0xffffffffu, e ? fix1 : fix0); left;) {
            const int l = __ffs(left) - 1;  // a lane of the row's four
            left &= ~(0xfu << (l & ~3));
            const int t = __shfl_sync(0xffffffffu, e ? t1 : t0, l), h = __shfl_sync(0xffffffffu, e ? h1 : h0, l);
            const float mx = __shfl_sync(0xffffffffu, e ? m1 : m0, l), sum = __shfl_sync(0xffffffffu, e ? l1 : l0, l);
            float v[D / 32];
            redo_row<BF, D>(a, own_pages, hk, t, h, k0, min(k1, __shfl_sync(0xffffffffu, e ? lim1 : lim0, l)), mx, lane, v);
            if (a.slots == 1) {
              uint16_t* dst = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(t) * a.ldo + h * D + lane * (D / 32);
              const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
              for (int i = 0; i < D / 32; i += 2)
                *reinterpret_cast<uint32_t*>(dst + i) = pack2<BF>(v[i] * inv, v[i + 1] * inv);
            } else {
              float* dst = a.part_o + ((static_cast<int64_t>(split) * a.rows + t) * a.heads + h) * D + lane * (D / 32);
#pragma unroll
              for (int i = 0; i < D / 32; ++i) dst[i] = v[i];
            }
          }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (PAIR)
    cluster_sync();  // neither CTA leaves while the pair's MMAs may use its memory
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------- host --

template <bool BF, int D, bool PAIR>
static cudaError_t launch_wide_t(const WideArgs& w, cudaStream_t s) {
  using W = Wide<D, PAIR>;
  static PerDevice<cudaError_t> once;
  const cudaError_t* attr = once.get([] {
    return cudaFuncSetAttribute(attn_paged_wide<BF, D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
  });
  if (attr == nullptr) return cudaErrorNoDevice;
  if (*attr != cudaSuccess) return *attr;
  const int64_t gx = static_cast<int64_t>(w.tiles) * w.splits * (PAIR ? 2 : 1);
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), w.a.kv.kv_heads);
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = W::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = PAIR ? 2 : 1;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attn_paged_wide<BF, D, PAIR>, w);
}

cudaError_t launch_attn_wide(const PagedAttnArgs& a, WideMode mode, bool pair, int tiles, int splits, cudaStream_t s) {
  WideArgs w;
  memset(&w, 0, sizeof w);
  w.a = a;
  w.tokens = wide_tokens(a.group);
  w.br_shift = kWBoxShift;
  while (a.kv.page_rows & ((1 << w.br_shift) - 1)) --w.br_shift;  // page_rows is a multiple of 16
  w.joint = mode == WIDE_JOINT;
  w.tiles = tiles;
  w.splits = splits;
  const int D = a.kv.dim;
  const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.heads), static_cast<uint64_t>(a.rows)};
  const uint64_t qs[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.ldq) * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(w.tokens)};
  cudaError_t e = encode_map(&w.qmap, a.kv.dt, 3, a.q, qd, qs, qb);
  if (e != cudaSuccess) return e;
  const uint64_t kd[2] = {2 * static_cast<uint64_t>(a.kv.kv_heads) * D,
                          static_cast<uint64_t>(a.kv.npages) * a.kv.page_rows};
  const uint64_t ks[1] = {kd[0] * 2};
  const uint32_t kb[2] = {64, 1u << w.br_shift};
  e = encode_map(&w.kvmap, a.kv.dt, 2, a.kv.pool, kd, ks, kb);
  if (e != cudaSuccess) return e;
  const bool bf = a.kv.dt == DT_BF16;
  if (D == 64) return bf ? launch_wide_t<true, 64, false>(w, s) : launch_wide_t<false, 64, false>(w, s);
  if (pair) return bf ? launch_wide_t<true, 128, true>(w, s) : launch_wide_t<false, 128, true>(w, s);
  return bf ? launch_wide_t<true, 128, false>(w, s) : launch_wide_t<false, 128, false>(w, s);
}

}  // namespace qi21
