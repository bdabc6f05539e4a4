// blocks.cuh -- what the kernels of the block-selected attention share: the
// shape as the device sees it, the limit of a query row, the walk over a tile
// of queries' selected blocks, row gathers into swizzled shared memory.
//
// Rows. A key head is shared by G = H / Hkv query heads, which select the same
// blocks. A row is one (query, head of the group) pair; a 128-row MMA tile
// holds tpt = 128 / G consecutive queries, query-major (row = query * G +
// head), so that the rows of a warp belong to few queries and a warp often has
// nothing to do for a block that only other queries selected.
//
// Keys come in tiles of 64 (kKeyTile); a block is a run of `nsub` tiles.
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace svoo {

constexpr int kRowTile = 128;
constexpr int kKeyTile = 64;
constexpr int kMaxSel = 256;      // slots of a query
constexpr int kMaxBlocks = 16384;  // blocks of a sequence
constexpr size_t kMaxSmem = 232448;  // dynamic shared memory of one CTA

struct BlockDims {
  int B, H, Hkv, G;
  int Nq, Nk, cap;  // queries, keys, key rows from one head to the next
  int nb, block, nsub, n_sel;
  int sink, local, causal, q_start;
  int tpt;      // queries of a row tile
  int inv_g;    // ceil(2^16 / G): r / G = r * inv_g >> 16 for r < 128
};

inline bool block_shape_ok(const svoo_block_shape* s) {
  if (!s) return false;
  if (s->B < 1 || s->H < 1 || s->Hkv < 1 || s->H % s->Hkv || s->H / s->Hkv > kRowTile) return false;
  if (s->Nq < 0 || s->Nk < 1 || s->cap < s->Nk || s->cap > (1 << 20) || s->Nq > (1 << 20)) return false;
  if (s->d != 64 && s->d != 128) return false;
  if (s->block < kKeyTile || s->block % kKeyTile || s->block > 1024) return false;
  if (s->n_sel < 1 || s->n_sel > kMaxSel) return false;
  if (s->causal != 0 && s->causal != 1) return false;
  if (s->sink < 0 || s->local < 0 || s->sink > s->n_sel || s->local > s->n_sel || s->sink + s->local > s->n_sel)
    return false;
  if (s->causal ? s->local < 1 : s->local != 0) return false;
  if (s->q_start < -1 || s->q_start > (1 << 20)) return false;
  if (static_cast<long long>(s->B) * s->H > 65535) return false;  // grid.y limit
  // rows of q and of k, v: TMA row coordinates and row indices are int32
  if (static_cast<long long>(s->B) * s->H * (s->Nq > 1 ? s->Nq : 1) >= (1LL << 31) - 256) return false;
  if (static_cast<long long>(s->B) * s->Hkv * s->cap >= (1LL << 31) - 256) return false;
  return true;
}

inline BlockDims block_dims(const svoo_block_shape* s) {
  BlockDims p;
  p.B = s->B;
  p.H = s->H;
  p.Hkv = s->Hkv;
  p.G = s->H / s->Hkv;
  p.Nq = s->Nq;
  p.Nk = s->Nk;
  p.cap = s->cap;
  p.block = s->block;
  p.nsub = s->block / kKeyTile;
  p.nb = (s->Nk + s->block - 1) / s->block;
  p.n_sel = s->n_sel;
  p.sink = s->sink;
  p.local = s->local;
  p.causal = s->causal;
  p.q_start = s->q_start;
  p.tpt = kRowTile / p.G;
  p.inv_g = (65536 + p.G - 1) / p.G;
  return p;
}

// Rows of a tensor map over keys or values: up to the last key of the last head.
// A view may begin inside its buffer, whose end is then less than cap rows from
// there, and a whole tile is loaded where the sequence ends inside one: what the
// map does not cover arrives as zeros and is not read.
inline uint64_t mapped_key_rows(const BlockDims& p) {
  return (static_cast<uint64_t>(p.B) * p.Hkv - 1) * p.cap + p.Nk;
}

inline bool scale_ok(float scale) { return scale > 0.f && scale < INFINITY; }

#ifdef __CUDACC__

// keys of sequence b, clamped to what the buffers hold
__device__ __forceinline__ int seq_len(const BlockDims& p, const int32_t* lengths, int b) {
  return lengths ? max(0, min(p.Nk, lengths[b])) : p.Nk;
}

__device__ __forceinline__ int query_pos(const BlockDims& p, int len, int i) {
  return p.q_start >= 0 ? p.q_start + i : len - p.Nq + i;
}

// Query i attends to keys below this: its own position + 1 (nothing for a
// query outside its sequence), or the whole sequence when not causal.
__device__ __forceinline__ int query_limit(const BlockDims& p, int len, int i) {
  if (!p.causal) return len;
  const int pos = query_pos(p, len, i);
  return pos >= 0 && pos < len ? pos + 1 : 0;
}

// A query's slots hold ascending block ids, then -1. The list ends at the first
// entry that is out of range or not above the one before it; *bad is raised
// when that entry is not -1. A warp calls it together; f(block) is called by
// the lane that holds the block. Returns the list's length.
template <class F>
__device__ __forceinline__ int walk_slots(const int32_t* slots, int n, int nb, bool* bad, F f) {
  const int lane = threadIdx.x & 31;
  int count = 0, carry = -1;
  for (int s0 = 0; s0 < n; s0 += 32) {
    const int s = s0 + lane;
    const int v = s < n ? slots[s] : -1;
    int prev = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) prev = carry;
    const bool ok = v >= 0 && v < nb && v > prev;
    const unsigned bal = __ballot_sync(0xffffffffu, ok);
    const int pre = bal == 0xffffffffu ? 32 : __ffs(~bal) - 1;
    if (lane < pre) f(v);
    count += pre;
    if (pre < 32) {
      if (__shfl_sync(0xffffffffu, v, pre) != -1) *bad = true;
      break;
    }
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
  return count;
}

// The same for at most 32 slots, one a lane: the lane's block, or -1 behind the
// list's end.
__device__ __forceinline__ int counted_slot(int v, int nb, bool* bad) {
  const int lane = threadIdx.x & 31;
  int prev = __shfl_up_sync(0xffffffffu, v, 1);
  if (lane == 0) prev = -1;
  const unsigned bal = __ballot_sync(0xffffffffu, v >= 0 && v < nb && v > prev);
  const int pre = bal == 0xffffffffu ? 32 : __ffs(~bal) - 1;
  if (__any_sync(0xffffffffu, lane == pre && v != -1)) *bad = true;
  return lane < pre ? v : -1;
}

// What a row tile has to visit: the key tiles of the union of its queries'
// blocks, ascending, and for every block of the union a bit per query. Walking
// the blocks' bitmap and every query's slots step by step instead cost the
// forward kernel a third of its time.
//   list  tile | ordinal of its block in the union << 16
//   mask  [block of the union][words] bits of the queries that selected it
struct TileList {
  uint32_t* list;
  uint32_t* mask;
  uint32_t* bits;   // a bit per block
  uint16_t* rank;   // union blocks before each word of `bits`
  int words;        // ceil(tpt / 32)
};

// blocks of the union, at most
inline size_t union_cap(const BlockDims& p) {
  const size_t chosen = static_cast<size_t>(p.tpt) * p.n_sel;
  return static_cast<size_t>(p.nb) < chosen ? p.nb : chosen;
}
inline size_t tile_list_bytes(const BlockDims& p) {
  const size_t words = (p.nb + 31) / 32;
  return 4 * (union_cap(p) * (p.nsub + (p.tpt + 31) / 32) + words + (words + 1) / 2);
}
// Queries of a row tile, at most: as many as keep its list within `room` bytes of
// shared memory (long sequences of few heads a group name more blocks than fit
// beside the tiles; the rows behind the last query then work for nothing). One
// query's 256 slots of blocks of 1024 keys are 20 KB.
inline BlockDims fit_tile(BlockDims p, size_t room) {
  while (p.tpt > 1 && tile_list_bytes(p) > room) --p.tpt;
  return p;
}

__device__ __forceinline__ TileList tile_list(const BlockDims& p, int cap, void* at) {
  TileList t;
  const int w = (p.nb + 31) / 32;
  t.words = (p.tpt + 31) / 32;
  t.list = static_cast<uint32_t*>(at);
  t.mask = t.list + cap * p.nsub;
  t.bits = t.mask + cap * t.words;
  t.rank = reinterpret_cast<uint16_t*>(t.bits + w);
  return t;
}

// Fills a CTA's list (all its threads; limits[] of the tile's queries are
// written too). Returns the number of key tiles. `shared_max`, `shared_tiles`:
// ints in shared memory.
template <int kThreads>
__device__ __forceinline__ int make_tile_list(const BlockDims& p, const TileList& t, const int32_t* slots, int t0,
                                              int nt, int len, int* limits, int* shared_max, int* shared_tiles,
                                              int* err) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int w_all = (p.nb + 31) / 32;
  for (int i = tid; i < w_all; i += kThreads) t.bits[i] = 0;
  if (tid == 0) *shared_max = 0;
  // A warp's queries, all loads in flight at once; a lane holds a slot (where
  // they are at most 32), -1 if it does not count
  constexpr int kMine = (kRowTile + kThreads / 32 - 1) / (kThreads / 32);
  const bool few = p.n_sel <= 32;
  int held[kMine];
  if (few) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int ti = warp + i * (kThreads / 32);
      held[i] = ti < nt && lane < p.n_sel ? slots[static_cast<size_t>(ti) * p.n_sel + lane] : -1;
    }
  }
  __syncthreads();
  bool bad = false;
  int most = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int ti = warp + i * (kThreads / 32);
    if (ti >= nt) break;
    const int lim = query_limit(p, len, t0 + ti);
    auto add = [&](int blk) {
      if (blk * p.block < lim) atomicOr(&t.bits[blk >> 5], 1u << (blk & 31));
    };
    if (few) {
      held[i] = counted_slot(held[i], p.nb, &bad);
      if (held[i] >= 0 && held[i] * p.block >= lim) held[i] = -1;
      if (held[i] >= 0) add(held[i]);
    } else {
      walk_slots(slots + static_cast<size_t>(ti) * p.n_sel, p.n_sel, p.nb, &bad, add);
    }
    if (lane == 0) limits[ti] = lim;
    most = max(most, lim);
  }
  if (lane == 0) atomicMax(shared_max, most);
  if (bad && lane == 0) report_error(err, kErrBadPlan);
  __syncthreads();
  const int tiles = (*shared_max + kKeyTile - 1) / kKeyTile;
  if (warp == 0) {
    int blocks = 0, n_tiles = 0;
    for (int w0 = 0; w0 < w_all; w0 += 32) {
      const int w = w0 + lane;
      uint32_t word = w < w_all ? t.bits[w] : 0u;
      const int n = __popc(word);
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      int ord = blocks + inc - n;
      if (w < w_all) t.rank[w] = static_cast<uint16_t>(ord);
      // only the last block of all can reach behind the last tile, and only in part
      while (word) {
        const int blk = w * 32 + __ffs(word) - 1;
        word &= word - 1;
        for (int s = 0; s < p.nsub && blk * p.nsub + s < tiles; ++s) {
          t.list[ord * p.nsub + s] = static_cast<uint32_t>(blk * p.nsub + s) | static_cast<uint32_t>(ord) << 16;
          n_tiles = ord * p.nsub + s + 1;
        }
        ++ord;
      }
      blocks += __shfl_sync(0xffffffffu, inc, 31);
    }
    n_tiles = __reduce_max_sync(0xffffffffu, n_tiles);
    for (int i = lane; i < blocks * t.words; i += 32) t.mask[i] = 0;
    if (lane == 0) *shared_tiles = n_tiles;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int ti = warp + i * (kThreads / 32);
    if (ti >= nt) break;
    auto mark = [&](int blk) {
      const int ord = t.rank[blk >> 5] + __popc(t.bits[blk >> 5] & ((1u << (blk & 31)) - 1u));
      atomicOr(&t.mask[ord * t.words + (ti >> 5)], 1u << (ti & 31));
    };
    if (few) {
      if (held[i] >= 0) mark(held[i]);
    } else {
      const int lim = limits[ti];
      walk_slots(slots + static_cast<size_t>(ti) * p.n_sel, p.n_sel, p.nb, &bad, [&](int blk) {
        if (blk * p.block < lim) mark(blk);
      });
    }
  }
  return *shared_tiles;
}

// 64 key rows from `row0` of a [rows, D] bf16 matrix into a swizzled tile of
// `kRows` rows, rows from `valid` on as zeros (what lies behind a sequence may
// hold anything, and 0 * NaN would reach every row). `lanes` threads take part.
template <int D, int kRows = kKeyTile>
__device__ __forceinline__ void load_key_rows(uint8_t* dst, const uint16_t* src, size_t row0, int valid, int tid,
                                              int lanes) {
  constexpr int kChunks = D / 8;
#pragma unroll 8
  for (int c = tid; c < kKeyTile * kChunks; c += lanes) {
    const int r = c / kChunks, ch = c - r * kChunks;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < valid) x = *reinterpret_cast<const uint4*>(src + (row0 + r) * D + ch * 8);
    *reinterpret_cast<uint4*>(dst + sw128_offset(r, ch * 8, kRows)) = x;
  }
}

// The two 64-key tiles of a step (first keys key[0], key[1]; below 0: none,
// zeros) into one swizzled 128-row tile, completing on `bar` (one arrival). A
// tile that the sequence ends in goes through plain loads, zeros behind its end.
// One warp.
template <int D>
__device__ __forceinline__ void load_key_pair(const CUtensorMap* map, const uint16_t* src, uint8_t* dst, uint32_t bar,
                                              size_t row0, int len, const int (&key)[2]) {
  constexpr int kRows = 2 * kKeyTile;
  const int lane = threadIdx.x & 31;
  uint32_t bytes = 0;
  bool slow = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (key[h] >= 0 && len - key[h] >= kKeyTile) {
      bytes += kKeyTile * D * 2;
    } else {
      load_key_rows<D, kRows>(dst + h * kKeyTile * 128, src, row0 + max(key[h], 0), key[h] < 0 ? 0 : len - key[h], lane,
                              32);
      slow = true;
    }
  }
  if (slow) {
    fence_proxy_async_smem();
    __syncwarp();
  }
  if (lane != 0) return;
  if (bytes == 0) {
    mbar_arrive(bar);
    return;
  }
  mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (key[h] >= 0 && len - key[h] >= kKeyTile)
      for (int s = 0; s < D / 64; ++s)
        tma_load_2d(map, smem_u32(dst) + s * kRows * 128 + h * kKeyTile * 128, bar, s * 64,
                    static_cast<int>(row0 + key[h]));
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One thread: the rows of a row tile (query-major, see above) of a [B, H, Nq, D]
// bf16 tensor (mapped by encode_token_major) into a swizzled 128-row tile,
// completing on `bar`, which expects tpt * G * D * 2 bytes of it. Queries behind
// the last arrive as zeros; rows from tpt * G on keep what was there, and rows of
// queries outside their sequence may hold anything: a row's products reach that
// row alone, and what such rows yield is not written.
template <int D>
__device__ __forceinline__ void load_query_rows(const CUtensorMap* map, uint8_t* dst, uint32_t bar, int head0, int t0,
                                                int b) {
  for (int s = 0; s < D / 64; ++s)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst) + s * kRowTile * 128),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(s * 64), "r"(head0), "r"(t0), "r"(b)
        : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// what `at` (shared memory) holds in CTA `rank` of the cluster
__device__ __forceinline__ float2 cluster_read2(uint32_t at, int rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_read4(uint32_t at, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T, kind::f16, A read from tensor memory.
__device__ __forceinline__ void umma_f16_a_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

#endif  // __CUDACC__

}  // namespace svoo
