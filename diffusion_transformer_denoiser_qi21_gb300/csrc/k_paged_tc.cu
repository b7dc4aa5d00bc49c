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
// L2 into each SM once per 256 rows. A single CTA (M 128) takes all rows of a
// block itself.
//
// A CTA takes items (tile, key head, split) in turn. The K warp finds them and
// hands them to the other roles through a short list in shared memory, so
// that the loads and the score MMAs of an item run while the softmax warps
// still divide and store the one before: of a first item 3.6 us pass before
// its scores and 3.8 after its last ones, a key block takes 0.75. With STAY a
// CTA takes items until none is left; otherwise it has one, as CTAs that
// start together walk their common keys together (the host's rule has the
// figures). Bound by the tensor cores and the softmax between them when the
// rows are many, by the bytes of K and V when one tile holds them all. Every
// wait is bounded.
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
constexpr int kWTails = 8;               // copied V boxes under way at most: more than ring stages

constexpr int kWItems = 4;               // items of the list between the roles

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
  static_assert((3 + kWTails + 4 * kStages + 3 * kWNS + 2 * kWItems) * 8 + 8 <= 512, "barrier area");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct WideArgs {
  PagedAttnArgs a;
  CUtensorMap qmap;   // q [rows][heads][dim], box tokens x group x 64 columns
  CUtensorMap kvmap;  // pool [npages * page_rows][2 * kv_heads * dim], box br x 64
  int tokens;         // of a CTA's tile
  int br_shift;       // log2 of the rows of a K / V box
  int joint, splits, tiles;
  int items;          // tiles * splits * kv_heads
};

// An item as a CTA sees it: its own tile's tokens [tok0, tok_end), and the
// key blocks that it and its pair walk.
struct WideItem {
  int tok0, tok_end, seq0, nrows, len;
  const int32_t* own_pages;
  int hk, split;
  int np, no;   // keys of the prefix, and own ones, that some row sees
  int npb;      // blocks of the prefix's
  int j0, n;    // this split's blocks; n < 0: there are no more items
  int least, most;  // keys that the item's rows see
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

template <bool BF, int D, bool PAIR, bool STAY>
__global__ void __launch_bounds__(kWThreads, 1) attn_paged_wide(const __grid_constant__ WideArgs p) {
  using W = Wide<D, PAIR>;
  constexpr int NK = W::kStages;
  constexpr int CT = PAIR ? 2 : 1;  // CTAs (tiles) of an item
  __shared__ WideItem s_items[kWItems];
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const PagedAttnArgs& a = p.a;
  const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.kv.prefix_len;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W::kOffBar);
  uint64_t* qfull = bars;             // even CTA: both Q tiles landed
  uint64_t* qempty = qfull + 1;       // both CTAs: the item's Q K^T done
  uint64_t* ofree = qempty + 1;       // even CTA: every CTA's O read
  uint64_t* kfull = ofree + 1;        // [NK] even CTA
  uint64_t* vfull = kfull + NK;       // [NK] even CTA
  uint64_t* vtail = vfull + NK;       // [kWTails] even CTA: the odd CTA's copied V boxes
  uint64_t* kempty = vtail + kWTails;      // [NK] both CTAs: stage's Q K^T done
  uint64_t* vempty = kempty + NK;     // [NK] both CTAs: stage's P V done
  uint64_t* sfull = vempty + NK;      // [kWNS] both CTAs: S_b written
  uint64_t* pfull = sfull + kWNS;     // [kWNS] even CTA: P_b of every CTA written
  uint64_t* pvdone = pfull + kWNS;    // [kWNS] both CTAs: P V of buffer b done
  uint64_t* ifull = pvdone + kWNS;    // [kWItems] this CTA: an item is in the list
  uint64_t* iempty = ifull + kWItems; // [kWItems] this CTA: every role has read it
  uint32_t* tslot = reinterpret_cast<uint32_t*>(iempty + kWItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);

  if (threadIdx.x == 2 * 32) {
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int i = 0; i < kWTails; ++i) mbar_init(&vtail[i], 1);
    mbar_init(ofree, 8 * CT);  // softmax warps
    for (int i = 0; i < NK; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&vfull[i], 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < kWNS; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 8 * CT);
      mbar_init(&pvdone[i], 1);
    }
    for (int i = 0; i < kWItems; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], leader ? 11 : 9);  // V and softmax warps, in the even CTA the MMA warps
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
  // what came before the call is done from here on (the set-up above touches
  // none of it); the call's next kernel may start
  grid_wait();
  grid_release();
  // keys of [prefix, own] that token t of an item sees
  auto limit = [&](const WideItem& w, int t) {
    const int total = P + w.len;
    int n = total;
    if (a.vis)
      n = static_cast<int>(min(__ldg(a.vis + t), static_cast<uint32_t>(total)));
    else if (a.causal && p.joint)
      n = P + min(max(w.len - w.nrows + (t - w.seq0) + 1, 0), w.len);
    return n;
  };
  // the r-th item of this cluster, by a whole warp; false: there is none.
  // Rounds run through the clusters to and fro, and a sequence's last tiles,
  // which see the most keys, come first: the clusters' sums stay even
  const int ncl = static_cast<int>(gridDim.x) / CT, cl = static_cast<int>(blockIdx.x) / CT;
  auto item_at = [&](int r, WideItem& w) -> bool {
    const int64_t i = static_cast<int64_t>(r) * ncl + (r & 1 ? ncl - 1 - cl : cl);
    if (static_cast<int64_t>(r) * ncl >= p.items) return false;
    w.tok0 = w.tok_end = w.seq0 = w.nrows = w.len = w.hk = w.split = 0;
    w.np = w.no = w.npb = w.j0 = w.n = w.least = w.most = 0;
    w.own_pages = nullptr;
    if (i >= p.items) return true;  // none in this round
    int x = static_cast<int>(i);
    int tile;
    if (STAY) {  // in order of tiles, the heads of one next to each other
      w.hk = x % a.kv.kv_heads;
      x /= a.kv.kv_heads;
      w.split = x % p.splits;
      tile = p.tiles - 1 - x / p.splits;
    } else {
      tile = p.tiles - 1 - x % p.tiles;
      x /= p.tiles;
      w.split = x % p.splits;
      w.hk = x / p.splits;
    }
    if (p.joint) {
      const SeqTile q = warp_find_tile(a, tile, 1, CT * p.tokens, lane);
      w.seq0 = q.row0;  // no such tile: no rows
      w.nrows = q.rows;
      w.tok0 = w.seq0 + q.at * CT * p.tokens;
      w.tok_end = w.seq0 + w.nrows;
      w.own_pages = a.kv.table + static_cast<int64_t>(q.b) * a.kv.table_stride;
      w.len = q.len;
      if (w.nrows > 0 && (w.len < w.nrows || w.len > a.kv.table_rows) && threadIdx.x == 0)
        atomicOr(&s_wide_status, kStatusPage);
      w.len = min(max(w.len, 0), a.kv.table_rows);
    } else {
      w.tok0 = tile * CT * p.tokens;
      w.tok_end = min(max(__ldg(a.kv.cu + a.kv.nseq), 0), a.rows);
    }
    const int end = min(w.tok_end, w.tok0 + CT * p.tokens);
    if (a.vis) {
      w.least = 0x7fffffff;
      for (int t = w.tok0 + lane; t < end; t += 32) {
        w.most = max(w.most, limit(w, t));
        w.least = min(w.least, limit(w, t));
      }
      w.most = __reduce_max_sync(0xffffffffu, w.most);
      w.least = __reduce_min_sync(0xffffffffu, w.least);
    } else if (w.tok0 < end) {
      w.most = limit(w, end - 1);
      w.least = limit(w, w.tok0);
    }
    w.tok0 += rank * p.tokens;
    w.np = min(w.most, P);
    w.no = max(w.most - P, 0);
    w.npb = (w.np + kWK - 1) / kWK;
    const int nb = w.npb + (w.no + kWK - 1) / kWK;
    w.j0 = static_cast<int>(static_cast<int64_t>(nb) * w.split / p.splits);
    w.n = static_cast<int>(static_cast<int64_t>(nb) * (w.split + 1) / p.splits) - w.j0;
    return true;
  };
  // does block j have a V box that the end cuts (see the V loads)?
  auto cut = [&](const WideItem& w, int j) {
    const bool pre = j < w.npb;
    const int left = (pre ? w.np : w.no) - (pre ? j : j - w.npb) * kWK;
    return left < kWK && (left & ((1 << p.br_shift) - 1)) != 0;
  };
  // a wait by a whole warp: every lane leaves with the same answer
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &s_wide_status));
  };

  WideItem w;
  if (!STAY) item_at(0, w);  // its waits for memory run beside the set-up
  // the loading warps' (below): of a CTA's only item they start on the first
  // page ids here
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
    const int j = w.j0 + i + (lane >> bxs);
    const bool pre = j < w.npb;
    key = (pre ? j : j - w.npb) * kWK + koff;
    if (i + (lane >> bxs) >= w.n || key >= (pre ? w.np : w.no)) key = -1;
    if (key >= 0) id = __ldg((pre ? a.kv.prefix_pages : w.own_pages) + key / a.kv.page_rows);
  };
  if (!STAY && (warp == 0 || warp == 11)) ids(0);
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

  // the next item of the list, for the roles that do not find it
  int seen = 0;
  auto next_item = [&](WideItem& w) -> bool {
    const int slot = seen % kWItems;
    if (!wait_all(&ifull[slot], (seen / kWItems) & 1)) return false;
    w = s_items[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&iempty[slot]);
    ++seen;
    return w.n >= 0;
  };

  int done = 0;  // items with keys so far (Q, O)
  int tails = 0;  // copied V boxes so far
  int blk = 0;   // key blocks so far (ring stages, S buffers)
  bool ok = true;
  if (warp == 0 || warp == 11) {
    // the two loading warps: Q and the K blocks, and the V blocks. A lane
    // holds the pool row of one box of a run of blocks, the ids of the next
    // run's pages are under way meanwhile, and lane 0 issues the boxes: a
    // block must not wait for its page ids, nor K for V's stage
    auto row_of = [&]() {
      if (key < 0) return none;
      if (id < 0 || id >= a.kv.npages) {
        atomicOr(&s_wide_status, kStatusPage);
        return none;
      }
      return id * a.kv.page_rows + key % a.kv.page_rows;
    };
    uint64_t* full = is_k ? kfull : vfull;
    uint64_t* empty = is_k ? kempty : vempty;
    const int stage = is_k ? W::kK : W::kV;
    const int cols = is_k ? W::kCols : W::kColsV;
    const int piece = keys * 128;                         // bytes of a column piece
    uint8_t* ring = smem + (is_k ? W::kOffK : W::kOffV);
    // the list: the K warp's next item to every other role
    auto find_item = [&](int r) -> bool {
      const bool has = item_at(r, w);
      if (!has) w.n = -1;
      const int slot = r % kWItems;
      if (!wait_all(&iempty[slot], ((r / kWItems) & 1) ^ 1u)) {
        ok = false;
        return false;
      }
      if (lane == 0) {
        s_items[slot] = w;
        mbar_arrive(&ifull[slot]);
      }
      __syncwarp();
      return has;
    };
    for (int r = 0; ok && (!STAY ? r == 0 : is_k ? find_item(r) : next_item(w)); ++r) {
      if (w.n == 0) continue;
      if (STAY) ids(0);
      // Q goes after the first two K blocks: its place is free only when the
      // scores of the item before are done
      auto load_q = [&]() -> bool {
        if (STAY && !wait_all(qempty, (done & 1) ^ 1u)) return false;
        if (lane == 0) {
          const uint32_t bytes = static_cast<uint32_t>(W::kCols) * p.tokens * a.group * 128;
          if (leader) mbar_arrive_expect_tx(qfull, CT * bytes);
          for (int c = 0; c < W::kCols; ++c) {
            uint8_t* d = smem + c * 16384;
            if (PAIR)
              tma_load_3d_pair(d, &p.qmap, mapa_rank(qfull, 0), c * 64, w.hk * a.group, w.tok0);
            else
              tma_load_3d(d, &p.qmap, qfull, c * 64, w.hk * a.group, w.tok0);
          }
        }
        ++done;
        return true;
      };
      const int q_at = !STAY || done == 0 ? -1 : min(1, w.n - 1);
      if (is_k && q_at < 0 && !(ok = load_q())) break;
      const int col0 = (is_k ? 0 : a.kv.kv_heads * D + (PAIR ? rank * 64 : 0)) + w.hk * D;
      int rows = none;
      for (int i = 0; i < w.n; ++i, ++blk) {
        if ((i & (run - 1)) == 0) {
          rows = row_of();
          ids(i + run);
        }
        const int st = blk % NK;
        if (!(ok = wait_all(&empty[st], ((blk / NK) & 1) ^ 1u))) break;
        uint8_t* base = ring + st * stage;
        const int at = (i & (run - 1)) << bxs;  // the lane with the block's first box
        int skip = -1;
        if (!is_k) {
          const int j = w.j0 + i;
          if (cut(w, j)) {
            // the V box that the end cuts, rows behind it zero
            const bool pre = j < w.npb;
            const int left = (pre ? w.np : w.no) - (pre ? j : j - w.npb) * kWK;
            skip = left >> brs;
            const int live = left - (skip << brs);  // its rows before the end
            const int r0 = __shfl_sync(0xffffffffu, rows, at + skip);
            const uint16_t* src = static_cast<const uint16_t*>(a.kv.pool) +
                                  static_cast<int64_t>(r0 == none ? 0 : r0) * (2 * a.kv.kv_heads * D) + col0;
            for (int c = 0; c < cols; ++c) {
              uint8_t* d = base + c * piece + (skip << (brs + 7));
              // a lane's pieces all loaded before the first is stored: the
              // box is one wait for memory
              uint4 v[8 << (kWBoxShift - 5)];
              const int r1 = lane >> 3, ch = lane & 7;
#pragma unroll
              for (int k = 0; k < 8 << (kWBoxShift - 5); ++k) {
                v[k] = make_uint4(0, 0, 0, 0);
                if (r1 + 4 * k < live && r0 != none)
                  v[k] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r1 + 4 * k) * (2 * a.kv.kv_heads * D) +
                                                         c * 64 + ch * 8);
              }
#pragma unroll
              for (int k = 0; k < 8 << (kWBoxShift - 5); ++k) {
                const int rr = r1 + 4 * k;
                if (rr < 1 << brs) *reinterpret_cast<uint4*>(d + rr * 128 + ((ch ^ (rr & 7)) << 4)) = v[k];
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            // the even CTA's P V waits for the odd one's copy
            if (PAIR && !leader && lane == 0) mbar_arrive_cluster(mapa_rank(&vtail[tails % kWTails], 0));
            ++tails;
          }
        }
        if (lane == 0 && leader)
          mbar_arrive_expect_tx(&full[st], CT * (stage - (skip >= 0 ? cols << (brs + 7) : 0)));
        const uint32_t fb = PAIR ? mapa_rank(&full[st], 0) : 0u;
        // every row first, then the boxes one after the other: an exchange
        // between two boxes held the next one up (16-row boxes: 67 us against
        // 61 for three sequences of 200 rows behind 2000 + 700)
        int row[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) row[b] = __shfl_sync(0xffffffffu, rows, at + b);
        if (lane == 0) {
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            if (b >= boxes) break;
            if (b == skip) continue;
            uint8_t* d = base + (b << (brs + 7));
            for (int c = 0; c < cols; ++c) {
              if (PAIR)
                tma_load_2d_pair(d + c * piece, &p.kvmap, fb, col0 + c * 64, row[b]);
              else
                tma_load_2d(d + c * piece, &p.kvmap, &full[st], col0 + c * 64, row[b]);
            }
          }
        }
        if (is_k && i == q_at && !(ok = load_q())) break;
      }
    }
    if (!ok) {
      // gave up: the copies under way land within microseconds, leave them a
      // millisecond before this CTA's memory is given back
      const unsigned long long g0 = globaltimer();
      while (globaltimer() - g0 < 1000000ull) __nanosleep(1000);
    }
  } else if (warp == 1 && leader) {
    constexpr uint32_t idesc = idesc_f16(128 * CT, kWK, false, BF);
    for (int r = 0; ok && (STAY ? next_item(w) : r == 0); ++r) {
      if (w.n == 0) continue;
      if (lane == 0) {
        const uint32_t sQ = smem_u32(smem);
        ok = mbar_wait(qfull, done & 1, abort_flag, &s_wide_status);
        for (int i = 0; i < w.n && ok; ++i) {
          const int g = blk + i;
          const int b = g % kWNS, st = g % NK;
          // S_b is free once the P V that read P_{g-3} from it is done
          if (g >= kWNS && !(ok = mbar_wait(&pvdone[b], ((g - kWNS) / kWNS) & 1, abort_flag, &s_wide_status))) break;
          if (!(ok = mbar_wait(&kfull[st], (g / NK) & 1, abort_flag, &s_wide_status))) break;
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
        if (ok) {
          if (PAIR)
            tc_commit_pair(qempty, 0x3);
          else
            tc_commit(qempty);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      blk += w.n;
      ++done;
    }
  } else if (warp == 10 && leader) {
    constexpr uint32_t idesc = idesc_f16(128 * CT, D, true, BF);  // V: MN-major
    for (int r = 0; ok && (STAY ? next_item(w) : r == 0); ++r) {
      if (w.n == 0) continue;
      if (lane == 0) {
        for (int i = 0; i < w.n; ++i) {
          const int g = blk + i;
          const int b = g % kWNS, st = g % NK;
          if (!(ok = mbar_wait(&pfull[b], (g / kWNS) & 1, abort_flag, &s_wide_status))) break;
          if (!(ok = mbar_wait(&vfull[st], (g / NK) & 1, abort_flag, &s_wide_status))) break;
          if (PAIR && cut(w, w.j0 + i)) {
            if (!(ok = mbar_wait_cluster(&vtail[tails % kWTails], (tails / kWTails) & 1, abort_flag, &s_wide_status)))
              break;
            ++tails;
          }
          // the item before has been read out of O
          if (STAY && i == 0 && done > 0 && !(ok = mbar_wait(ofree, (done - 1) & 1, abort_flag, &s_wide_status))) break;
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
      ok = __shfl_sync(0xffffffffu, ok, 0);
      blk += w.n;
      ++done;
    }
  } else if (warp >= 2 && warp <= 9) {
    // softmax: two warps per TMEM lane quadrant, 16 lanes (rows) each; thread
    // t holds rows r0 = base + t/4 and r1 = r0 + 8, columns 8k + 2(t%4) and
    // + 1 of each 8-column group k of a block's scores
    const int q = warp & 3;
    const int hh = (warp - 2) >> 2;
    const int lbase = q * 32 + hh * 16;
    const int tq = lane >> 2, tj = lane & 3;
    const int r0 = lbase + tq, r1 = r0 + 8;
    const int i0 = r0 / a.group, i1 = r1 / a.group;
    const uint32_t lane_off = static_cast<uint32_t>(lbase) << 16;
    const float c = a.scale_log2;
    const uint64_t c2 = f2(c, c);
    const uint32_t pf_remote = PAIR && !leader ? mapa_rank(pfull, 0) : 0u;
    for (int r = 0; ok && (STAY ? next_item(w) : r == 0); ++r) {
      const int t0 = w.tok0 + i0, t1 = w.tok0 + i1;
      const bool live0 = i0 < p.tokens && t0 < w.tok_end, live1 = i1 < p.tokens && t1 < w.tok_end;
      const bool dead = !__any_sync(0xffffffffu, live0 || live1);  // no row of this warp
      const int lim0 = live0 ? limit(w, t0) : w.most;
      const int lim1 = live1 ? limit(w, t1) : w.most;
      float m0 = -INFINITY, m1 = -INFINITY;
      uint64_t lacc = 0ull;  // (row r0, row r1) partial sums of this thread's columns
      for (int i = 0; i < w.n; ++i, ++blk) {
        const int b = blk % kWNS;
        if (!(ok = wait_all(&sfull[b], (blk / kWNS) & 1))) break;
        if (!dead) {
          tc_fence_after();
          uint32_t s[2][32];  // [half of the 128 columns][8 groups x (r0 c, r0 c+1, r1 c, r1 c+1)]
          tmem_ld16x256_x8(tS + b * kWK + lane_off, s[0]);
          tmem_ld16x256_x8(tS + b * kWK + 64 + lane_off, s[1]);
          tmem_ld_wait(s[0]);
          tmem_ld_wait(s[1]);
          // what the rows see of this block: its first e0, e1 keys
          const int j = w.j0 + i;
          const bool pre = j < w.npb;
          const int first = pre ? j * kWK : P + (j - w.npb) * kWK;
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
          // raise each row's running max only past the threshold (O and l
          // share the stale max; p <= 2^threshold stays in f16 range)
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
          // weights 2^(-inf - 0) = 0. P is rounded to the values' type (half
          // a step of a weight, of either sign); l sums the f32 weights
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
            // O is stable once the P V of the block before is done
            const int g = blk - 1;
            if (!(ok = wait_all(&pvdone[g % kWNS], (g / kWNS) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int hf = 0; hf < W::kCols; ++hf) {
              uint32_t o[32];
              tmem_ld16x256_x8(tO + hf * 64 + lane_off, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                o[4 * k + 0] = __float_as_uint(__uint_as_float(o[4 * k + 0]) * al0);
                o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * al0);
                o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * al1);
                o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * al1);
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
      if (!ok) break;
      uint32_t o[W::kCols][32];
#pragma unroll
      for (int hf = 0; hf < W::kCols; ++hf)
#pragma unroll
        for (int k = 0; k < 32; ++k) o[hf][k] = 0u;
      if (w.n > 0) {
        // the item's sums into registers; O is then free for the next item
        const int g = blk - 1;
        if (!(ok = wait_all(&pvdone[g % kWNS], (g / kWNS) & 1))) break;
        if (!dead) {
          tc_fence_after();
#pragma unroll
          for (int hf = 0; hf < W::kCols; ++hf) tmem_ld16x256_x8(tO + hf * 64 + lane_off, o[hf]);
#pragma unroll
          for (int hf = 0; hf < W::kCols; ++hf) tmem_ld_wait(o[hf]);
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive(ofree);
          else
            mbar_arrive_cluster_relaxed(mapa_rank(ofree, 0));
        }
      }
      if (dead) continue;
      float l0, l1;
      unf2(lacc, l0, l1);
#pragma unroll
      for (int k = 1; k <= 2; k <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, k);
        l1 += __shfl_xor_sync(0xffffffffu, l1, k);
      }
      const int h0 = w.hk * a.group + r0 - i0 * a.group, h1 = w.hk * a.group + r1 - i1 * a.group;
      float odd0 = 0.f, odd1 = 0.f;  // NaN once a sum is not finite
      if (a.slots == 1) {
        const float inv0 = l0 > 0.f || l0 != l0 ? 1.f / l0 : 0.f;  // a row that sees no key is 0
        const float inv1 = l1 > 0.f || l1 != l1 ? 1.f / l1 : 0.f;
        uint16_t* o0 = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(t0) * a.ldo + h0 * D + 8 * tj;
        uint16_t* o1 = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(t1) * a.ldo + h1 * D + 8 * tj;
        // a row's 64 columns sit in four threads as one pair of each group of
        // 8; exchanged, a thread has all of groups tj and tj + 4 and stores 16
        // bytes at once (the single pairs' stores took 1.2 us)
#pragma unroll
        for (int hf = 0; hf < W::kCols; ++hf)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float x0 = __uint_as_float(o[hf][16 * half + 4 * g + 0]), x1 = __uint_as_float(o[hf][16 * half + 4 * g + 1]);
              const float y0 = __uint_as_float(o[hf][16 * half + 4 * g + 2]), y1 = __uint_as_float(o[hf][16 * half + 4 * g + 3]);
              odd0 = fmaf(0.f, x0 + x1, odd0);
              odd1 = fmaf(0.f, y0 + y1, odd1);
              w0[g] = pack2<BF>(x0 * inv0, x1 * inv0);
              w1[g] = pack2<BF>(y0 * inv1, y1 * inv1);
            }
            quad_transpose(w0, tj);
            quad_transpose(w1, tj);
            const int col = hf * 64 + 32 * half;
            if (live0) *reinterpret_cast<uint4*>(o0 + col) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
            if (live1) *reinterpret_cast<uint4*>(o1 + col) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
          }
      } else {
        const int64_t at0 = (static_cast<int64_t>(w.split) * a.rows + t0) * a.heads + h0;
        const int64_t at1 = (static_cast<int64_t>(w.split) * a.rows + t1) * a.heads + h1;
        if (tj == 0 && live0) a.part_ml[at0] = make_float2(m0, l0);
        if (tj == 0 && live1) a.part_ml[at1] = make_float2(m1, l1);
        if (w.n > 0) {  // a part without keys has weight 0: its sums are not read
#pragma unroll
          for (int hf = 0; hf < W::kCols; ++hf)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int col = hf * 64 + 8 * k + 2 * tj;
              odd0 = fmaf(0.f, __uint_as_float(o[hf][4 * k + 0]) + __uint_as_float(o[hf][4 * k + 1]), odd0);
              odd1 = fmaf(0.f, __uint_as_float(o[hf][4 * k + 2]) + __uint_as_float(o[hf][4 * k + 3]), odd1);
              if (live0)
                *reinterpret_cast<uint2*>(a.part_o + at0 * D + col) = make_uint2(o[hf][4 * k + 0], o[hf][4 * k + 1]);
              if (live1)
                *reinterpret_cast<uint2*>(a.part_o + at1 * D + col) = make_uint2(o[hf][4 * k + 2], o[hf][4 * k + 3]);
            }
        }
      }
      // A key that some rows of the tile see and others do not has weight 0 in
      // those, but 0 times a value that is not finite is a NaN. Rows with such
      // a sum are done again over the keys that they see alone, if one of the
      // keys between the tile's limits has such a value
      const bool fix0 = live0 && odd0 != odd0 && w.least < w.most, fix1 = live1 && odd1 != odd1 && w.least < w.most;
      if (__any_sync(0xffffffffu, fix0 || fix1) && w.n > 0 &&
          odd_values<BF, D>(a, w.own_pages, w.hk, w.least, w.most, lane)) {
        __syncwarp();  // after the stores above, some of which are replaced
        const int j1 = w.j0 + w.n;
        const int k0 = w.j0 < w.npb ? w.j0 * kWK : P + (w.j0 - w.npb) * kWK;           // this split's keys
        const int k1 = j1 <= w.npb ? min(j1 * kWK, w.np) : P + min((j1 - w.npb) * kWK, w.no);
        for (int e = 0; e < 2; ++e)
          for (unsigned left = __ballot_sync(0xffffffffu, e ? fix1 : fix0); left;) {
            const int l = __ffs(left) - 1;  // a lane of the row's four
            left &= ~(0xfu << (l & ~3));
            const int t = __shfl_sync(0xffffffffu, e ? t1 : t0, l), h = __shfl_sync(0xffffffffu, e ? h1 : h0, l);
            const float mx = __shfl_sync(0xffffffffu, e ? m1 : m0, l), sum = __shfl_sync(0xffffffffu, e ? l1 : l0, l);
            float v[D / 32];
            redo_row<BF, D>(a, w.own_pages, w.hk, t, h, k0, min(k1, __shfl_sync(0xffffffffu, e ? lim1 : lim0, l)), mx,
                            lane, v);
            if (a.slots == 1) {
              uint16_t* dst = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(t) * a.ldo + h * D + lane * (D / 32);
              const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
              for (int i = 0; i < D / 32; i += 2)
                *reinterpret_cast<uint32_t*>(dst + i) = pack2<BF>(v[i] * inv, v[i + 1] * inv);
            } else {
              float* dst = a.part_o + ((static_cast<int64_t>(w.split) * a.rows + t) * a.heads + h) * D + lane * (D / 32);
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

template <bool BF, int D, bool PAIR, bool STAY>
static cudaError_t launch_wide_s(const WideArgs& w, cudaStream_t s) {
  using W = Wide<D, PAIR>;
  auto config = [](cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, unsigned grid, cudaStream_t s) {
    cfg->gridDim = dim3(grid);
    cfg->blockDim = dim3(kWThreads);
    cfg->dynamicSmemBytes = W::kSmem;
    cfg->stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = PAIR ? 2 : 1;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = at;
    cfg->numAttrs = 2;
  };
  // the shared-memory opt-in and the clusters that run at once, per device
  struct Init {
    cudaError_t e;
    int clusters;
  };
  static PerDevice<Init> once;
  const Init* init = once.get([&] {
    Init r{cudaFuncSetAttribute(attn_paged_wide<BF, D, PAIR, STAY>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem),
           sm_count()};
    if (r.e == cudaSuccess && PAIR) {
      cudaLaunchConfig_t cfg{};
      cudaLaunchAttribute at[2];
      config(&cfg, at, 2 * static_cast<unsigned>(sm_count()), nullptr);
      cfg.numAttrs = 1;
      r.clusters = 0;
      r.e = cudaOccupancyMaxActiveClusters(&r.clusters, attn_paged_wide<BF, D, PAIR, STAY>, &cfg);
    }
    r.clusters = std::max(1, r.clusters);
    return r;
  });
  if (init == nullptr) return cudaErrorNoDevice;
  if (init->e != cudaSuccess) return init->e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  config(&cfg, at, static_cast<unsigned>((STAY ? std::min(w.items, init->clusters) : w.items) * (PAIR ? 2 : 1)), s);
  return cudaLaunchKernelEx(&cfg, attn_paged_wide<BF, D, PAIR, STAY>, w);
}

template <bool BF, int D, bool PAIR>
static cudaError_t launch_wide_t(const WideArgs& w, bool stay, cudaStream_t s) {
  return stay ? launch_wide_s<BF, D, PAIR, true>(w, s) : launch_wide_s<BF, D, PAIR, false>(w, s);
}

cudaError_t launch_attn_wide(const PagedAttnArgs& a, WideMode mode, bool pair, int tiles, int splits, cudaStream_t s) {
  WideArgs w;
  memset(&w, 0, sizeof w);
  w.a = a;
  w.tokens = wide_tokens(a.group);
  w.br_shift = kWBoxShift;
  while (a.kv.page_rows & ((1 << w.br_shift) - 1)) --w.br_shift;  // page_rows is a multiple of 16
  w.joint = mode != WIDE_PREFIX;
  w.tiles = tiles;
  w.splits = splits;
  const int64_t items = static_cast<int64_t>(tiles) * splits * a.kv.kv_heads;
  if (items > 0x3fffffff) return cudaErrorInvalidValue;
  w.items = static_cast<int>(items);
  const bool stay = mode == WIDE_STAY;
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
  if (D == 64) return bf ? launch_wide_t<true, 64, false>(w, stay, s) : launch_wide_t<false, 64, false>(w, stay, s);
  if (pair) return bf ? launch_wide_t<true, 128, true>(w, stay, s) : launch_wide_t<false, 128, true>(w, stay, s);
  return bf ? launch_wide_t<true, 128, false>(w, stay, s) : launch_wide_t<false, 128, false>(w, stay, s);
}

}  // namespace qi21
