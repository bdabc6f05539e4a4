// cache.cu -- attention of one token per sequence over a cache, with each
// slot's softmax weight added to a running sum, and eviction by those sums.
//
//   o = softmax(scale q K^T) V over the sequence's slots (or those of the
//   blocks that the query selected);  weight[slot] += sum over the group's
//   heads of the slot's softmax weight
//
// cache_attn_kernel   A CTA takes one key head and a run of 64-slot tiles, so
//                     every key and value row is read once for all G heads of
//                     its group. A producer warp streams the tiles by TMA
//                     through a ring; four warps take 16 slots of each tile
//                     with heads as the 16 rows of mma.sync m16n8k16 (G <= 16
//                     heads are far from filling a tcgen05 tile, and the kernel
//                     is bound by the cache's bytes), each with its own running
//                     maximum, sum and output, joined once at the end.
//                     Up to eight runs are a cluster and join through each
//                     other's shared memory. 75 us at 48 sequences, 40/8 heads,
//                     d = 128, 32 blocks of 64 slots each (403 MB: 5.4 TB/s).
// cache_join_kernel   joins more runs, and turns the kept scores into weights
//                     (not while a timeout bit is set).
// evict_select_kernel the slots that stay, one CTA per (sequence, key head): 21 us
//                     for 128 of them with 8192 slots (barriers of its passes).
// evict_move_kernel   moves kept rows from behind `keep` into the holes: 49 us
//                     for 8192 -> 4096 slots of the same (the rows' bytes).
#include "blocks.cuh"

namespace svoo {

namespace {

constexpr int kCacheWarps = 4;                        // 16 slots of a tile each
constexpr int kCacheThreads = 32 * (kCacheWarps + 1);  // and the producer
constexpr int kCacheStages = 3;
constexpr int kHeadRows = 16;  // heads of one CTA
constexpr int kMaxJoined = 8;  // CTAs of a cluster
constexpr int kMaxRuns = 256;

struct CacheSmem {
  uint64_t full[kCacheStages], empty[kCacheStages];
#ifdef SVOO_TEST_STALL
  uint64_t stall;  // test-only: a barrier that nothing completes
#endif
  int abort;
  float m[kCacheWarps][kHeadRows], l[kCacheWarps][kHeadRows];
  float2 ml[kHeadRows];  // of the CTA, for its cluster
};

template <int D>
constexpr size_t cache_smem_bytes() {
  return 1024 + kCacheStages * 2 * static_cast<size_t>(kKeyTile) * D * 2 + sizeof(CacheSmem);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Grid (runs, B * Hkv, ceil(G / 16)). Partial results of run x: o (fp32
// [runs][B*H][D]) and (m in log2 units, l) per head; with one run, or where the
// runs are a cluster (joined), the output itself. scores (may be NULL): fp32 [B*H][cap], scale * q.k * log2 e.
template <int D>
__global__ void __launch_bounds__(kCacheThreads)
    cache_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, BlockDims p,
                      const uint16_t* __restrict__ q, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ lengths, float scale_log2, int joined, float* __restrict__ scores,
                      float* __restrict__ part_o, float2* __restrict__ part_ml, uint16_t* __restrict__ o,
                      float* __restrict__ lse, int* __restrict__ err) {
  constexpr int kSub = D / 64;
  constexpr int kTileBytes = kKeyTile * D * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CacheSmem* S = reinterpret_cast<CacheSmem*>(base + kCacheStages * 2 * kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.y, b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int h0 = blockIdx.z * kHeadRows, heads = min(kHeadRows, p.G - h0);
  const int len = seq_len(p, lengths, b);
  const int32_t* slots = idx ? idx + static_cast<size_t>(bh) * p.n_sel : nullptr;
  // a CTA of a cluster stays to its end: the others read its shared memory
  const bool skip = __syncthreads_or(timed_out_before(err) ? 1 : 0) != 0;
  if (skip && !joined) return;
  if (tid == 0) {
    S->abort = 0;
    for (int s = 0; s < kCacheStages; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), kCacheWarps);
    }
#ifdef SVOO_TEST_STALL
    mbar_init(smem_u32(&S->stall), 1);
#endif
    fence_mbar_init();
  }
  // tiles of this run: [i0, i1) of the sequence's, or of its selected blocks'
  int tiles = (len + kKeyTile - 1) / kKeyTile;
  if (slots) {
    bool bad = false;
    tiles = walk_slots(slots, p.n_sel, p.nb, &bad, [](int) {}) * p.nsub;
    if (bad && tid == 0 && blockIdx.x == 0) report_error(err, kErrBadPlan);
  }
  if (skip) tiles = 0;
  const int per = (tiles + gridDim.x - 1) / gridDim.x;
  const int i0 = min(tiles, static_cast<int>(blockIdx.x) * per), i1 = min(tiles, i0 + per);
  auto tile_key = [&](int i) { return (slots ? slots[i / p.nsub] * p.nsub + i % p.nsub : i) * kKeyTile; };
  __syncthreads();
  volatile int* abort = &S->abort;
  const uint32_t ring = smem_u32(base);

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
  int armed = -1;

  if (warp == kCacheWarps) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
      const int row0 = bh * p.cap;
      int j = 0;
      bool go = true;
#ifdef SVOO_TEST_STALL
      go = mbar_wait(smem_u32(&S->stall), 0, abort);  // nothing completes it
#endif
      for (int i = i0; i < i1 && go; ++i) {
        const int key0 = tile_key(i);
        if (key0 >= len) continue;
        const int st = j % kCacheStages;
        if (j >= kCacheStages && !mbar_wait(smem_u32(&S->empty[st]), (j / kCacheStages - 1) & 1, abort)) break;
        const uint32_t bar = smem_u32(&S->full[st]), dst = ring + st * 2 * kTileBytes;
        mbar_arrive_expect_tx(bar, 2 * kTileBytes);
        for (int s = 0; s < kSub; ++s) {
          tma_load_2d(&kmap, dst + s * kKeyTile * 128, bar, s * 64, row0 + key0);
          tma_load_2d(&vmap, dst + kTileBytes + s * kKeyTile * 128, bar, s * 64, row0 + key0);
        }
        armed = j++;
      }
    }
  } else {
    // ---------------------------------------------------------------- 16 slots of every tile
    const int hr = lane >> 2, c2 = (lane & 3) * 2;  // fragment: head rows hr, hr + 8; columns c2, c2 + 1
    uint32_t qa[D / 16][4];
    {
      const uint16_t* q0 = q + (static_cast<size_t>(b) * p.H + hk * p.G + h0) * D;
      const bool r0 = hr < heads, r1 = hr + 8 < heads;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint16_t* a = q0 + hr * D + kk * 16 + c2;
        qa[kk][0] = r0 ? *reinterpret_cast<const uint32_t*>(a) : 0u;
        qa[kk][1] = r1 ? *reinterpret_cast<const uint32_t*>(a + 8 * D) : 0u;
        qa[kk][2] = r0 ? *reinterpret_cast<const uint32_t*>(a + 8) : 0u;
        qa[kk][3] = r1 ? *reinterpret_cast<const uint32_t*>(a + 8 * D + 8) : 0u;
      }
    }
    const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix, row
    int j = 0;
    for (int i = i0; i < i1; ++i) {
      const int key0 = tile_key(i);
      if (key0 >= len) continue;
      const int st = j % kCacheStages;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&S->full[st]), (j / kCacheStages) & 1, abort))) break;
      const uint32_t ks = ring + st * 2 * kTileBytes, vs = ks + kTileBytes;
      const int first = key0 + warp * 16, valid = min(16, len - first);
      if (valid > 0) {
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
          const int row = warp * 16 + n * 8 + mr;
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {  // 32 columns at a time
            const int ch = kk * 4 + mi;
            uint32_t r[4];
            ldsm4(ks + (ch >> 3) * kKeyTile * 128 + row * 128 + (((ch & 7) ^ mr) << 4), r);
            mma_16x8x16(s[n], qa[2 * kk][0], qa[2 * kk][1], qa[2 * kk][2], qa[2 * kk][3], r[0], r[1]);
            mma_16x8x16(s[n], qa[2 * kk + 1][0], qa[2 * kk + 1][1], qa[2 * kk + 1][2], qa[2 * kk + 1][3], r[2], r[3]);
          }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = n * 8 + c2 + (c & 1);
            s[n][c] = key < valid ? s[n][c] * scale_log2 : -INFINITY;
            mx[c >> 1] = fmaxf(mx[c >> 1], s[n][c]);
          }
        if (scores) {
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            if (hr + 8 * rr >= heads) continue;
            float* out = scores + (static_cast<size_t>(b) * p.H + hk * p.G + h0 + hr + 8 * rr) * p.cap + first;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (n * 8 + c2 + c < valid) out[n * 8 + c2 + c] = s[n][rr * 2 + c];
          }
        }
        uint32_t pa[4];
        float al[2];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 1));
          mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 2));
          const float mn = fmaxf(m[rr], mx[rr]);  // finite: valid > 0
          al[rr] = ex2_approx(m[rr] - mn);
          m[rr] = mn;
          const float p0 = ex2_approx(s[0][rr * 2] - mn), p1 = ex2_approx(s[0][rr * 2 + 1] - mn);
          const float p2 = ex2_approx(s[1][rr * 2] - mn), p3 = ex2_approx(s[1][rr * 2 + 1] - mn);
          l[rr] = l[rr] * al[rr] + ((p0 + p1) + (p2 + p3));  // this lane's columns, in 32 bits
          pa[rr] = pack_bf16x2(p0, p1);                       // bf16 for the second product
          pa[rr + 2] = pack_bf16x2(p2, p3);
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            acc[d][0] *= al[0];
            acc[d][1] *= al[0];
            acc[d][2] *= al[1];
            acc[d][3] *= al[1];
          }
        }
        if (valid < 16) {
          // what lies behind the sequence may be NaN, and 0 * NaN is NaN
          for (int c = lane; c < (16 - valid) * (D / 8); c += 32) {
            const int row = warp * 16 + valid + c / (D / 8), ch = c % (D / 8);
            *reinterpret_cast<uint4*>(base + (vs - ring) + (ch >> 3) * kKeyTile * 128 + row * 128 + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const int row = warp * 16 + (mi & 1) * 8 + mr;
#pragma unroll
        for (int dd = 0; dd < D / 16; ++dd) {
          const int ch = dd * 2 + (mi >> 1);
          uint32_t r[4];
          ldsm4_t(vs + (ch >> 3) * kKeyTile * 128 + row * 128 + (((ch & 7) ^ mr) << 4), r);
          mma_16x8x16(acc[2 * dd], pa[0], pa[1], pa[2], pa[3], r[0], r[1]);
          mma_16x8x16(acc[2 * dd + 1], pa[0], pa[1], pa[2], pa[3], r[2], r[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->empty[st]));
      ++j;
    }
    // per-row sums over the quad's columns
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
      l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
      if ((lane & 3) == 0) {
        S->m[warp][hr + 8 * rr] = m[rr];
        S->l[warp][hr + 8 * rr] = l[rr];
      }
    }
  }
  __syncthreads();
  const bool failed = *abort != 0;
  if (failed) {
    if (tid == 0) report_error(err, kErrTimeoutAttn);
    if (warp == kCacheWarps && lane == 0)  // copies in flight land before the shared memory goes away
      for (int j = max(0, armed - kCacheStages + 1); j <= armed; ++j)
        mbar_wait_cleanup(smem_u32(&S->full[j % kCacheStages]), (j / kCacheStages) & 1);
  }
  // join the four warps: every tile has been consumed, the ring is free
  float* os = reinterpret_cast<float*>(base);  // [warp][16][D]
  if (warp < kCacheWarps && !failed) {
    const int hr = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
      *reinterpret_cast<float2*>(os + (warp * kHeadRows + hr) * D + d * 8 + c2) = make_float2(acc[d][0], acc[d][1]);
      *reinterpret_cast<float2*>(os + (warp * kHeadRows + hr + 8) * D + d * 8 + c2) =
          make_float2(acc[d][2], acc[d][3]);
    }
  }
  __syncthreads();
  if (failed && !joined) return;
  if (failed)
    for (int h = tid; h < heads; h += kCacheThreads) S->ml[h] = make_float2(-INFINITY, 0.f);
  for (int i = tid; i < heads * (D / 2) && !failed; i += kCacheThreads) {
    // (one thread has all of a column's four values)
    const int h = i / (D / 2), c = (i - h * (D / 2)) * 2;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kCacheWarps; ++w) mm = fmaxf(mm, S->m[w][h]);
    float ll = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kCacheWarps; ++w) {
      const float f = S->m[w][h] == -INFINITY ? 0.f : ex2_approx(S->m[w][h] - mm);
      const float2 v = *reinterpret_cast<const float2*>(os + (w * kHeadRows + h) * D + c);
      ll = fmaf(S->l[w][h], f, ll);
      x = fmaf(v.x, f, x);
      y = fmaf(v.y, f, y);
    }
    const size_t row = static_cast<size_t>(b) * p.H + hk * p.G + h0 + h;
    if (gridDim.x == 1) {
      const float inv = ll > 0.f ? 1.f / ll : 0.f;
      *reinterpret_cast<uint32_t*>(o + row * D + c) = pack_bf16x2(x * inv, y * inv);
      if (c == 0) lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    } else if (joined) {
      *reinterpret_cast<float2*>(os + h * D + c) = make_float2(x, y);
      if (c == 0) S->ml[h] = make_float2(mm, ll);
    } else {
      const size_t at = static_cast<size_t>(blockIdx.x) * p.B * p.H + row;
      *reinterpret_cast<float2*>(part_o + at * D + c) = make_float2(x, y);
      if (c == 0) part_ml[at] = make_float2(mm, ll);
    }
  }
  if (!joined) return;
  // a share of the columns each, over all CTAs of the cluster
  cluster_sync();
  const int runs = gridDim.x;
  for (int i = blockIdx.x * kCacheThreads + tid; i < heads * (D / 2); i += runs * kCacheThreads) {
    const int h = i / (D / 2), c = (i - h * (D / 2)) * 2;
    float2 ml[kMaxJoined], v[kMaxJoined];
    float mm = -INFINITY;
#pragma unroll
    for (int x = 0; x < kMaxJoined; ++x) {
      ml[x] = x < runs ? cluster_read2(smem_u32(&S->ml[h]), x) : make_float2(-INFINITY, 0.f);
      v[x] = x < runs ? cluster_read2(smem_u32(os + h * D + c), x) : make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int x = 0; x < kMaxJoined; ++x) mm = fmaxf(mm, ml[x].x);
    float ll = 0.f, a = 0.f, e = 0.f;
#pragma unroll
    for (int x = 0; x < kMaxJoined; ++x) {
      if (ml[x].x == -INFINITY) continue;  // an empty run's columns may be anything
      const float f = ex2_approx(ml[x].x - mm);
      ll = fmaf(ml[x].y, f, ll);
      a = fmaf(v[x].x, f, a);
      e = fmaf(v[x].y, f, e);
    }
    const size_t row = static_cast<size_t>(b) * p.H + hk * p.G + h0 + h;
    const float inv = ll > 0.f ? 1.f / ll : 0.f;
    *reinterpret_cast<uint32_t*>(o + row * D + c) = pack_bf16x2(a * inv, e * inv);
    if (c == 0) lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
  }
  cluster_sync();  // nobody leaves while its shared memory is read
}

// Grid (1 + chunks of 1024 slots where weights are kept, B * Hkv). Block 0
// joins the runs of the group's heads (when there are several), the others add
// the slots' weights, unless a wait has run out: a run that gave up left its
// scores unwritten, and the weights are the caller's for good. Dynamic shared
// memory: a factor per (head, run).
template <int D>
__global__ void __launch_bounds__(256)
    cache_join_kernel(BlockDims p, int runs, const int32_t* __restrict__ lengths, const float* __restrict__ part_o,
                      const float2* __restrict__ part_ml, const float* __restrict__ scores, uint16_t* __restrict__ o,
                      float* __restrict__ lse, float* __restrict__ weight, const int* __restrict__ err) {
  extern __shared__ float factor[];
  __shared__ float lse2[kRowTile];
  if (__syncthreads_or(timed_out_before(err) ? 1 : 0)) return;
  const int bh = blockIdx.y, b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const size_t row0 = static_cast<size_t>(b) * p.H + hk * p.G, rows = static_cast<size_t>(p.B) * p.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int g = warp; g < p.G; g += 8) {
    float l2;
    if (runs > 1) {
      // lanes over the runs (at most kMaxRuns: eight a lane)
      float2 v[8];
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = i * 32 + lane;
        v[i] = x < runs ? part_ml[x * rows + row0 + g] : make_float2(-INFINITY, 0.f);
        mm = fmaxf(mm, v[i].x);
      }
#pragma unroll
      for (int s = 16; s; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (v[i].y > 0.f) ll = fmaf(v[i].y, ex2_approx(v[i].x - mm), ll);
#pragma unroll
      for (int s = 16; s; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
      l2 = ll > 0.f ? mm + log2f(ll) : -INFINITY;
      if (blockIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 32 + lane < runs) factor[g * runs + i * 32 + lane] = v[i].y > 0.f ? ex2_approx(v[i].x - l2) : 0.f;
      }
    } else {
      l2 = lse[row0 + g] * 1.4426950408889634f;
    }
    if (lane == 0) lse2[g] = l2;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (runs == 1) return;
    for (int i = tid; i < p.G * (D / 2); i += 256) {
      const int g = i / (D / 2), c = (i - g * (D / 2)) * 2;
      const float* f = factor + g * runs;
      const float* src = part_o + (row0 + g) * D + c;
      float a = 0.f, e = 0.f;
#pragma unroll 8
      for (int x = 0; x < runs; ++x) {
        const float2 v = *reinterpret_cast<const float2*>(src + x * rows * D);
        a = fmaf(v.x, f[x], a);
        e = fmaf(v.y, f[x], e);
      }
      *reinterpret_cast<uint32_t*>(o + (row0 + g) * D + c) = pack_bf16x2(a, e);
      if (c == 0) lse[row0 + g] = lse2[g] * 0.6931471805599453f;
    }
    return;
  }
  const int len = seq_len(p, lengths, b);
  const int k0 = (blockIdx.x - 1) * 1024 + tid;
  if (k0 - tid >= len) return;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int g = 0; g < p.G; ++g) {
    const float* src = scores + (row0 + g) * p.cap;
    const float l2 = lse2[g];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i * 256 < len) a[i] += ex2_approx(src[k0 + i * 256] - l2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (k0 + i * 256 < len) weight[static_cast<size_t>(bh) * p.cap + k0 + i * 256] += a[i];
}

// Runs per (sequence, key head): enough CTAs to fill the card four times over
// (two fit an SM), so that the last ones do not run alone, with at least 8
// tiles each; below that, as few tiles as it takes to reach every SM.
inline int cache_runs(const BlockDims& p, bool selected) {
  const int tiles = selected ? p.n_sel * p.nsub : (p.Nk + kKeyTile - 1) / kKeyTile;
  const long long ctas = static_cast<long long>(p.B) * p.Hkv * ((p.G + kHeadRows - 1) / kHeadRows);
  const long long most = (4 * 2 * 148 + ctas - 1) / ctas;
  long long runs = tiles / 8 < most ? tiles / 8 : most;
  const long long few = (148 + ctas - 1) / ctas;
  if (runs < few) runs = few < tiles ? few : tiles;
  if (runs > kMaxRuns) runs = kMaxRuns;
  return runs < 1 ? 1 : static_cast<int>(runs);
}

// Up to eight runs are a cluster where all CTAs run at once, and need no kernel
// (5 us and its launch) to join them. (In several waves a cluster waits for its
// slowest run with all its places: 48 sequences, 40/8 heads, 32 blocks of 64:
// 88 us against 75 + 8.) More runs become eight where that leaves at most four
// tiles to a run: a tile takes a run about 1 us.
inline int cache_runs(const BlockDims& p, bool selected, bool* joined) {
  const int tiles = selected ? p.n_sel * p.nsub : (p.Nk + kKeyTile - 1) / kKeyTile;
  int runs = cache_runs(p, selected);
  if (runs > kMaxJoined && tiles <= 4 * kMaxJoined) runs = kMaxJoined;
  const long long ctas = static_cast<long long>(runs) * p.B * p.Hkv * ((p.G + kHeadRows - 1) / kHeadRows);
  *joined = runs > 1 && runs <= kMaxJoined && ctas <= 2 * 148;
  return runs;
}

struct CachePlan {
  int runs;
  bool joined;
  float *part_o, *scores;
  float2* part_ml;
  size_t bytes;
};
CachePlan cache_plan(const BlockDims& p, int d, bool selected, bool weights, void* ws) {
  CachePlan c;
  c.runs = cache_runs(p, selected, &c.joined);
  Carver w(ws);
  const size_t rows = static_cast<size_t>(p.B) * p.H;
  const size_t parts = c.runs > 1 && !c.joined ? c.runs * rows : 0;
  c.part_o = w.take<float>(parts * d);
  c.part_ml = w.take<float2>(parts);
  c.scores = w.take<float>(weights ? rows * p.cap : 0);
  c.bytes = (w.used + 255) / 256 * 256;
  return c;
}

template <int D>
svoo_status launch_cache_attn(const BlockDims& p, const void* q, const void* k, const void* v, const int32_t* lengths,
                              const int32_t* idx, float scale, float* weight, void* o, float* lse, void* ws,
                              int32_t* dev_err, cudaStream_t st) {
  const CachePlan c = cache_plan(p, D, idx != nullptr, weight != nullptr, ws);
  CUtensorMap km, vm;
  const uint64_t rows = mapped_key_rows(p);
  if (encode_tiled_2d(&km, k, rows, D, kKeyTile, 64) != CUDA_SUCCESS ||
      encode_tiled_2d(&vm, v, rows, D, kKeyTile, 64) != CUDA_SUCCESS)
    return SVOO_ERR_CUDA;
  const size_t smem = cache_smem_bytes<D>();
  if (!allow_smem(cache_attn_kernel<D>, smem)) return SVOO_ERR_CUDA;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.runs, p.B * p.Hkv, (p.G + kHeadRows - 1) / kHeadRows);
  cfg.blockDim = dim3(kCacheThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = c.runs;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = c.joined ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, cache_attn_kernel<D>, km, vm, p, static_cast<const uint16_t*>(q), idx, lengths,
                         scale_log2, c.joined ? 1 : 0, weight ? c.scores : nullptr, c.part_o, c.part_ml,
                         static_cast<uint16_t*>(o), lse, static_cast<int*>(dev_err)) != cudaSuccess)
    return launch_status();
  const int runs = c.joined ? 1 : c.runs;  // still to join
  const size_t factors = runs > 1 ? static_cast<size_t>(p.G) * runs * 4 : 0;
  // (48 KB need no leave, the kernel's own half KB among them)
  if (factors > 32 * 1024 && !allow_smem(cache_join_kernel<D>, kRowTile * kMaxRuns * 4)) return SVOO_ERR_CUDA;
  if (runs > 1 || weight)
    cache_join_kernel<D><<<dim3(1 + (weight ? (p.Nk + 1023) / 1024 : 0), p.B * p.Hkv), 256, factors, st>>>(
        p, runs, lengths, c.part_o, c.part_ml, c.scores, static_cast<uint16_t*>(o), lse, weight, dev_err);
  return launch_status();
}

// ------------------------------------------------------------------ eviction

constexpr int kEvictThreads = 1024;

struct EvictDims {
  int B, Hkv, cap, keep, sink, recent;
};

// Order of a slot: protected ones first, then by weight (NaN last), as an
// unsigned key; larger stays.
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int sink, int newest, int recent) {
  if (pos < sink || pos > newest - recent) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w);
  const uint32_t k = (u << 1) == 0 ? 0x80000000u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);  // -0 as 0
  return (u & 0x7fffffffu) > 0x7f800000u ? 0u : min(k, 0xfffffffeu);
}

// Sums before each warp of a round, in place: n counts (one per warp and round,
// in slot order) by the first warp. Returns nothing until the caller's barrier.
__device__ __forceinline__ void evict_scan(int* counts, int n) {
  const int lane = threadIdx.x;  // of the first warp
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int x = i0 + lane < n ? counts[i0 + lane] : 0;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (i0 + lane < n) counts[i0 + lane] = base + inc - x;
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) counts[n] = base;
}

// One CTA per (sequence, key head). Finds the keep-th largest key by radix
// selection (four passes of 8 bits), then walks the slots in order: equal keys
// stay from the lowest slot up; evicted slots below `keep` are holes, kept ones
// from `keep` on are sources. moves: the i-th hole and the i-th source. R keys a
// thread stay in registers; R = 0 reads the weights anew in every pass.
template <int R>
__global__ void __launch_bounds__(kEvictThreads)
    evict_select_kernel(EvictDims p, const float* __restrict__ weight, const int32_t* __restrict__ pos,
                        const int32_t* __restrict__ lengths, int m_cap, int2* __restrict__ moves,
                        int32_t* __restrict__ n_moves) {
  constexpr int kCounts = (R ? R : 1) * (kEvictThreads / 32);
  __shared__ int hist[4][256];  // four, since weights share their leading bits
  __shared__ int counts[2][kCounts + 1];
  __shared__ int newest_s, digit_s, left_s;
  const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x;
  const int len = max(0, min(p.cap, lengths[b]));
  if (len <= p.keep) {
    if (tid == 0) n_moves[bh] = 0;
    return;
  }
  const float* w = weight + static_cast<size_t>(bh) * p.cap;
  const int32_t* ps = pos + static_cast<size_t>(bh) * p.cap;
  if (tid == 0) newest_s = -1;
  hist[tid >> 8][tid & 255] = 0;
  static_assert(kEvictThreads == 4 * 256, "one thread per counter");
  const int warp = tid >> 5, lane = tid & 31;
  uint32_t held[R ? R : 1];
  int place[R ? R : 1];
  int newest = -1;
  if (R) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * kEvictThreads + tid;
      held[r] = i < len ? __float_as_uint(w[i]) : 0u;
      place[r] = i < len ? ps[i] : -1;
      newest = max(newest, place[r]);
    }
  } else {
    for (int i = tid; i < len; i += kEvictThreads) newest = max(newest, ps[i]);
  }
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, newest);
  if ((tid & 31) == 0) atomicMax(&newest_s, newest);
  __syncthreads();
  newest = newest_s;
  if (R) {
#pragma unroll
    for (int r = 0; r < R; ++r) held[r] = evict_key(__uint_as_float(held[r]), place[r], p.sink, newest, p.recent);
  }
  const int rounds = (len + kEvictThreads - 1) / kEvictThreads;
  // f(round, slot, key) for every slot, a round of threads at a time
  auto each = [&](auto f) {
    if (R) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rounds) f(r, r * kEvictThreads + tid, held[r]);
    } else {
      for (int r = 0; r < rounds; ++r) {
        const int i = r * kEvictThreads + tid;
        f(r, i, i < len ? evict_key(w[i], ps[i], p.sink, newest, p.recent) : 0u);
      }
    }
  };
  uint32_t prefix = 0, mask = 0;
  int want = p.keep;  // the want-th largest of those that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    each([&](int r, int i, uint32_t k) {
      if (i < len && (k & mask) == prefix) atomicAdd(&hist[warp & 3][(k >> shift) & 255], 1);
    });
    __syncthreads();
    if (tid < 32) {
      // from the top: lane l holds digits 255 - 8 l ... 248 - 8 l
      int c[8], s = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          c[i] += hist[h][255 - tid * 8 - i];
          hist[h][255 - tid * 8 - i] = 0;
        }
        s += c[i];
      }
      int inc = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= o) inc += y;
      }
      int above = inc - s;
      if (above < want && inc >= want) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < want && above + c[i] >= want) {
            digit_s = 255 - tid * 8 - i;
            left_s = want - above;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(digit_s) << shift;
    mask |= 255u << shift;
    want = left_s;
  }
  // Kept: keys above `prefix`, and the first `want` equal to it. A slot's place
  // among its like: ballots within a warp, sums over the warps before it. Both
  // lists of moves have at most m_cap entries.
  const unsigned below = (1u << lane) - 1u;
  constexpr int kWarps = kEvictThreads / 32;
  int2* out = moves + static_cast<size_t>(bh) * m_cap;
  auto kept = [&](int i, uint32_t k, int equal_before, unsigned eq) {
    return i < len && (k > prefix || (k == prefix && equal_before + __popc(eq & below) < want));
  };
  if (R) {
    each([&](int r, int i, uint32_t k) {
      const unsigned eq = __ballot_sync(0xffffffffu, i < len && k == prefix);
      if (lane == 0) counts[0][r * kWarps + warp] = __popc(eq);
    });
    __syncthreads();
    if (warp == 0) evict_scan(counts[0], rounds * kWarps);
    __syncthreads();
    unsigned keeps[R ? R : 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * kEvictThreads + tid;
      const unsigned eq = __ballot_sync(0xffffffffu, r < rounds && i < len && held[r] == prefix);
      keeps[r] = __ballot_sync(0xffffffffu, r < rounds && kept(i, held[r], r < rounds ? counts[0][r * kWarps + warp] : 0, eq));
    }
    __syncthreads();
    // holes lie below `keep`, sources from there on: one count per warp for both
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * kEvictThreads + tid;
      const bool keep = (keeps[r] >> lane) & 1u;
      const unsigned hole = __ballot_sync(0xffffffffu, i < p.keep && i < len && !keep);
      const unsigned src = __ballot_sync(0xffffffffu, i >= p.keep && keep);
      if (lane == 0 && r < rounds) {
        counts[0][r * kWarps + warp] = __popc(hole);
        counts[1][r * kWarps + warp] = __popc(src);
      }
    }
    __syncthreads();
    if (warp == 0) {
      evict_scan(counts[0], rounds * kWarps);
      evict_scan(counts[1], rounds * kWarps);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * kEvictThreads + tid;
      const bool keep = (keeps[r] >> lane) & 1u;
      const unsigned hole = __ballot_sync(0xffffffffu, i < p.keep && i < len && !keep);
      const unsigned src = __ballot_sync(0xffffffffu, i >= p.keep && keep);
      if (r < rounds) {
        if ((hole >> lane) & 1u) out[counts[0][r * kWarps + warp] + __popc(hole & below)].x = i;
        if ((src >> lane) & 1u) out[counts[1][r * kWarps + warp] + __popc(src & below)].y = i;
      }
    }
    if (tid == 0) n_moves[bh] = counts[1][rounds * kWarps];
  } else {
    int equal = 0, holes = 0, srcs = 0;
    each([&](int r, int i, uint32_t k) {
      const unsigned eq = __ballot_sync(0xffffffffu, i < len && k == prefix);
      if (lane == 0) counts[0][warp] = __popc(eq);
      __syncthreads();
      if (warp == 0) evict_scan(counts[0], kWarps);
      __syncthreads();
      const bool keep = kept(i, k, equal + counts[0][warp], eq);
      equal += counts[0][kWarps];
      __syncthreads();
      const unsigned hole = __ballot_sync(0xffffffffu, i < p.keep && i < len && !keep);
      const unsigned src = __ballot_sync(0xffffffffu, i >= p.keep && keep);
      if (lane == 0) {
        counts[0][warp] = __popc(hole);
        counts[1][warp] = __popc(src);
      }
      __syncthreads();
      if (warp == 0) {
        evict_scan(counts[0], kWarps);
        evict_scan(counts[1], kWarps);
      }
      __syncthreads();
      if ((hole >> lane) & 1u) out[holes + counts[0][warp] + __popc(hole & below)].x = i;
      if ((src >> lane) & 1u) out[srcs + counts[1][warp] + __popc(src & below)].y = i;
      holes += counts[0][kWarps];
      srcs += counts[1][kWarps];
      __syncthreads();
    });
    if (tid == 0) n_moves[bh] = srcs;
  }
}

// Grid (chunks, B * Hkv): the lanes of a move carry both its rows, 16 bytes
// each, four moves in flight; weight and position with them. Sources lie at or
// behind `keep`, holes before it: no order needed.
template <int D>
__global__ void __launch_bounds__(256)
    evict_move_kernel(EvictDims p, int m_cap, const int2* __restrict__ moves, const int32_t* __restrict__ n_moves,
                      uint16_t* __restrict__ k, uint16_t* __restrict__ v, float* __restrict__ weight,
                      int32_t* __restrict__ pos, int32_t* __restrict__ lengths) {
  constexpr int kLanes = D / 8;  // 16-byte pieces of a row
  constexpr int kSide = 256 / (2 * kLanes);  // moves side by side in a CTA
  constexpr int kDeep = 4;
  const int bh = blockIdx.y, n = n_moves[bh];
  const int in = threadIdx.x % (2 * kLanes), side = threadIdx.x / (2 * kLanes);
  const size_t base = static_cast<size_t>(bh) * p.cap;
  uint16_t* x = (in < kLanes ? k : v) + base * D + (in % kLanes) * 8;
  const int2* mine = moves + static_cast<size_t>(bh) * m_cap;
  for (int i0 = blockIdx.x * kSide * kDeep + side; i0 < n; i0 += gridDim.x * kSide * kDeep) {
    int2 mv[kDeep];
    uint4 row[kDeep];
    float w[kDeep];
    int32_t ps[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int i = i0 + j * kSide;
      mv[j] = i < n ? mine[i] : make_int2(-1, -1);
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      if (mv[j].y < 0) continue;
      row[j] = *reinterpret_cast<const uint4*>(x + static_cast<size_t>(mv[j].y) * D);
      if (in == 0) w[j] = weight[base + mv[j].y];
      if (in == 1) ps[j] = pos[base + mv[j].y];
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      if (mv[j].y < 0) continue;
      *reinterpret_cast<uint4*>(x + static_cast<size_t>(mv[j].x) * D) = row[j];
      if (in == 0) weight[base + mv[j].x] = w[j];
      if (in == 1) pos[base + mv[j].x] = ps[j];
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && bh % p.Hkv == 0) {
    const int b = bh / p.Hkv;
    if (lengths[b] > p.keep) lengths[b] = p.keep;
  }
}

inline bool evict_ok(int B, int Hkv, int cap, int d, int keep, int sink, int recent) {
  if (B < 1 || Hkv < 1 || cap < 1 || cap > (1 << 20) || (d != 64 && d != 128)) return false;
  if (keep < 1 || sink < 0 || recent < 0 || sink > keep || recent > keep - sink) return false;
  if (static_cast<long long>(B) * Hkv > 65535) return false;
  return static_cast<long long>(B) * Hkv * cap < (1LL << 31) - 256;
}

inline int evict_move_cap(int cap, int keep) { return keep >= cap ? 0 : (keep < cap - keep ? keep : cap - keep); }

}  // namespace

}  // namespace svoo

using namespace svoo;

extern "C" size_t svoo_cache_attn_workspace_size(const svoo_block_shape* shape, int selected, int weights) {
  if (!block_shape_ok(shape) || shape->Nq != 1) return 0;
  return cache_plan(block_dims(shape), shape->d, selected != 0, weights != 0, nullptr).bytes;
}

extern "C" svoo_status svoo_cache_attn(const svoo_block_shape* shape, const void* q, const void* k, const void* v,
                                       const int32_t* lengths, const int32_t* idx, float scale, float* weight, void* o,
                                       float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                       void* stream) {
  if (!block_shape_ok(shape) || shape->Nq != 1 || !q || !k || !v || !o || !lse || !scale_ok(scale))
    return SVOO_ERR_INVALID_ARG;
  if (idx && weight) return SVOO_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(lengths, 4) || !aligned(idx, 4) || !aligned(weight, 4) || !aligned(dev_err, 4) ||
      !aligned(workspace, 256))
    return SVOO_ERR_INVALID_ARG;
  const BlockDims p = block_dims(shape);
  const size_t need = cache_plan(p, shape->d, idx != nullptr, weight != nullptr, nullptr).bytes;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SVOO_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128)
    return launch_cache_attn<128>(p, q, k, v, lengths, idx, scale, weight, o, lse, workspace, dev_err, st);
  return launch_cache_attn<64>(p, q, k, v, lengths, idx, scale, weight, o, lse, workspace, dev_err, st);
}

extern "C" size_t svoo_cache_evict_workspace_size(int B, int Hkv, int cap, int keep) {
  if (!evict_ok(B, Hkv, cap, 64, keep, 0, 0)) return 0;
  const size_t rows = static_cast<size_t>(B) * Hkv;
  return (rows * 4 + 255) / 256 * 256 + (rows * evict_move_cap(cap, keep) * 8 + 255) / 256 * 256;
}

extern "C" svoo_status svoo_cache_evict(int B, int Hkv, int cap, int d, int keep, int sink, int recent, void* k,
                                        void* v, float* weight, int32_t* pos, int32_t* lengths, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (!evict_ok(B, Hkv, cap, d, keep, sink, recent) || !k || !v || !weight || !pos || !lengths || !workspace)
    return SVOO_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(weight, 4) || !aligned(pos, 4) || !aligned(lengths, 4) ||
      !aligned(workspace, 256))
    return SVOO_ERR_INVALID_ARG;
  if (workspace_bytes < svoo_cache_evict_workspace_size(B, Hkv, cap, keep)) return SVOO_ERR_WORKSPACE;
  const int m_cap = evict_move_cap(cap, keep);
  if (m_cap == 0) return SVOO_OK;  // nothing can be longer than keep
  const EvictDims p = {B, Hkv, cap, keep, sink, recent};
  const int rows = B * Hkv;
  int32_t* n_moves = static_cast<int32_t*>(workspace);
  int2* moves = reinterpret_cast<int2*>(static_cast<char*>(workspace) + (static_cast<size_t>(rows) * 4 + 255) / 256 * 256);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cap <= 4 * kEvictThreads)
    evict_select_kernel<4><<<rows, kEvictThreads, 0, st>>>(p, weight, pos, lengths, m_cap, moves, n_moves);
  else if (cap <= 16 * kEvictThreads)
    evict_select_kernel<16><<<rows, kEvictThreads, 0, st>>>(p, weight, pos, lengths, m_cap, moves, n_moves);
  else
    evict_select_kernel<0><<<rows, kEvictThreads, 0, st>>>(p, weight, pos, lengths, m_cap, moves, n_moves);
  // 32 moves (64 at d = 64) a CTA and turn; the moves are not known here, their bound is
  const int turn = 4 * 256 / (2 * (d / 8));
  int chunks = (m_cap + turn - 1) / turn;
  if (chunks > 32) chunks = 32;
  if (d == 128)
    evict_move_kernel<128><<<dim3(chunks, rows), 256, 0, st>>>(p, m_cap, moves, n_moves, static_cast<uint16_t*>(k),
                                                               static_cast<uint16_t*>(v), weight, pos, lengths);
  else
    evict_move_kernel<64><<<dim3(chunks, rows), 256, 0, st>>>(p, m_cap, moves, n_moves, static_cast<uint16_t*>(k),
                                                              static_cast<uint16_t*>(v), weight, pos, lengths);
  return launch_status();
}
