// block_lists.cuh -- for every block the list of the queries that selected it,
// in a fixed order (no atomics decide a place), and the work items of kernels
// that go by key tiles: a key tile with a piece of its block's list.
#pragma once

#include "blocks.cuh"

#ifdef __CUDACC__

namespace svoo {

namespace {

// A warp takes `chunk` queries of one (sequence, key head) in order, 32 at a
// time and slot by slot; lanes with the same block are ranked by lane. Both
// passes walk the same way, so a place depends on the selection alone.
// kSelCount: the chunk's count per block; kSelList: the lists; kSelPlaces: and
// for every slot its place in them (-1: in none).
enum SelPass { kSelCount, kSelList, kSelPlaces };

template <SelPass kPass>
__global__ void __launch_bounds__(32)
    sel_walk_kernel(BlockDims p, const int32_t* __restrict__ idx, const int32_t* __restrict__ lengths, int chunk,
                    int nchunk, int32_t* __restrict__ hist, const int32_t* __restrict__ start,
                    int32_t* __restrict__ list, int32_t* __restrict__ places) {
  extern __shared__ int cnt[];
  const int lane = threadIdx.x, c = blockIdx.x, bh = blockIdx.y;
  const int len = seq_len(p, lengths, bh / p.Hkv);
  int32_t* h = hist + (static_cast<size_t>(bh) * nchunk + c) * p.nb;
  for (int i = lane; i < p.nb; i += 32) cnt[i] = kPass != kSelCount ? start[static_cast<size_t>(bh) * p.nb + i] + h[i] : 0;
  __syncwarp();
  const int t1 = min(p.Nq, (c + 1) * chunk);
  for (int t0 = c * chunk; t0 < t1; t0 += 32) {
    const int t = t0 + lane;
    const int lim = t < t1 ? query_limit(p, len, t) : 0;
    const int32_t* mine = idx + (static_cast<size_t>(bh) * p.Nq + (t < t1 ? t : 0)) * p.n_sel;
    int prev = -1;
    bool go = t < t1;
    for (int s = 0; s < p.n_sel; ++s) {
      const int blk = go ? mine[s] : -1;
      go = go && blk > prev && blk < p.nb;
      prev = blk;
      if (kPass != kSelPlaces && !__any_sync(0xffffffffu, go)) break;
      const bool take = go && blk * p.block < lim;
      const unsigned same = __match_any_sync(0xffffffffu, take ? blk : -1 - lane);
      int place = -1;
      if (kPass != kSelCount && take) {
        place = cnt[blk] + __popc(same & ((1u << lane) - 1u));
        list[static_cast<size_t>(bh) * p.Nq * p.n_sel + place] = t;
      }
      if (kPass == kSelPlaces && t < t1) places[(static_cast<size_t>(bh) * p.Nq + t) * p.n_sel + s] = place;
      __syncwarp();
      if (take && (same & ((1u << lane) - 1u)) == 0) cnt[blk] += __popc(same);
      __syncwarp();
    }
  }
  if (kPass == kSelCount)
    for (int i = lane; i < p.nb; i += 32) h[i] = cnt[i];
}

// per block: running sums of the chunks' counts (in place) and the total; a CTA
// takes 32 blocks, its eight warps an eighth of the chunks each
__global__ void __launch_bounds__(256)
    sel_scan_kernel(BlockDims p, int nchunk, int32_t* __restrict__ hist, int32_t* __restrict__ total) {
  __shared__ int part[8][32];
  const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5, blk = blockIdx.x * 32 + lane, bh = blockIdx.y;
  const int per = (nchunk + 7) / 8, c0 = min(nchunk, seg * per), c1 = min(nchunk, c0 + per);
  const bool there = blk < p.nb;
  int32_t* h = hist + static_cast<size_t>(bh) * nchunk * p.nb + (there ? blk : 0);
  int a = 0;
  if (there) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) a += h[static_cast<size_t>(c) * p.nb];
  }
  part[seg][lane] = a;
  __syncthreads();
  a = 0;
  for (int s = 0; s < seg; ++s) a += part[s][lane];
  if (!there) return;
#pragma unroll 8
  for (int c = c0; c < c1; ++c) {
    const int x = h[static_cast<size_t>(c) * p.nb];
    h[static_cast<size_t>(c) * p.nb] = a;
    a += x;
  }
  if (seg == 7) total[static_cast<size_t>(bh) * p.nb + blk] = a;
}

// Exclusive sums over a block of 1024 threads, each with its own value.
__device__ __forceinline__ int block_exclusive(int x, int* warp_sums, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *all = warp_sums[31];
  const int r = inc - x + (warp ? warp_sums[warp - 1] : 0);
  __syncthreads();
  return r;
}

// Where each block's list starts (per (sequence, key head)), and the work
// items: every key tile's list in pieces of at most `piece` rows (one piece
// where there are none). items: tile, piece, pieces, slot of the piece's part
// (-1 where it is the only one). One block of 1024 threads.
__global__ void __launch_bounds__(1024)
    sel_items_kernel(BlockDims p, int ktiles, int piece, const int32_t* __restrict__ total, int32_t* __restrict__ start,
                     int4* __restrict__ items, int32_t* __restrict__ counts) {
  __shared__ int sums[32];
  const int BH = p.B * p.Hkv;
  for (int bh = 0; bh < BH; ++bh) {
    int base = 0;
    for (int i0 = 0; i0 < p.nb; i0 += 1024) {
      const int i = i0 + threadIdx.x;
      int all;
      const int x = block_exclusive(i < p.nb ? total[static_cast<size_t>(bh) * p.nb + i] : 0, sums, &all);
      if (i < p.nb) start[static_cast<size_t>(bh) * p.nb + i] = base + x;
      base += all;
    }
  }
  int n_items = 0, n_slots = 0;
  const int tiles = BH * ktiles;
  for (int i0 = 0; i0 < tiles; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    int pieces = 0;
    if (i < tiles) {
      const int bh = i / ktiles, kt = i - bh * ktiles;
      const long long rows = static_cast<long long>(total[static_cast<size_t>(bh) * p.nb + kt / p.nsub]) * p.G;
      pieces = max(1, static_cast<int>((rows + piece - 1) / piece));
    }
    int all, all_slots;
    int at = block_exclusive(pieces, sums, &all) + n_items;
    const int slot = block_exclusive(pieces > 1 ? pieces : 0, sums, &all_slots) + n_slots;
    for (int c = 0; c < pieces; ++c) items[at + c] = make_int4(i, c, pieces, pieces > 1 ? slot + c : -1);
    n_items += all;
    n_slots += all_slots;
  }
  if (threadIdx.x == 0) {
    counts[0] = n_items;
    counts[1] = n_slots;
  }
}

// barrier of the loader warps, with a vote
template <int kThreads>
__device__ __forceinline__ bool loaders_agree(bool ok) {
  uint32_t r;
  __syncwarp();  // bar takes a warp's threads together
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(kThreads)
      : "memory");
  return r != 0;
}

// Queries of a chunk, which one warp counts: many chunks, while their counts
// stay below four per query.
inline int sel_chunk(const BlockDims& p) { return p.nb > 256 ? (p.nb / 4 + 31) / 32 * 32 : 64; }

}  // namespace

}  // namespace svoo

#endif  // __CUDACC__
