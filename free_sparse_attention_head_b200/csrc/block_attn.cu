// block_attn.cu -- attention of every query over the key blocks that it
// selected, forward, sm_100a.
//
//   o = softmax(scale q K_S^T) V_S,  lse = log sum exp(scale q K_S^T),
//   S = the keys below the query's limit in its selected blocks.
//
// One CTA per 128-row tile (tpt consecutive queries x G heads of one key
// head's group). It walks the union of its queries' blocks once, in ascending
// 64-key tiles; a row whose query did not select the tile's block gets P = 0,
// and a warp none of whose queries did skips the exponentials. The union keeps
// the tensor cores on full 128-row products whatever G is, at the price of
// rows that compute for nothing: neighbouring queries mostly agree, and in the
// worst case the union is what dense attention would read. 534 us at 32760
// tokens, 16/2 heads, d = 128, 16 blocks of 64 keys, whose unions are 1.9
// selections: 0.5 PFLOP/s of the selected keys, 0.97 of what it computes. Where
// unions would be near everything, a call goes by key blocks instead (below).
//
// Where there are few row tiles, a tile's list is shared out to several CTAs
// (grid.z), a cluster that puts its parts together from its shared memories.
//
// Two CTAs share an SM (256 tensor-memory columns and half of the shared
// memory each), so one's softmax runs beside the other's products.
// Warps: 0-3 softmax (thread r = row r = TMEM lane r), 4 key/value producer
// (TMA; the tile that crosses the sequence's end by plain loads with zeros
// behind it), 5 MMA issuer, which runs S(j+1) ahead of the softmax of tile j.
// TMEM: S [0,64) and [64,128) alternating, P over the S that it came from,
// O [128,128+D).
#include "block_lists.cuh"

namespace svoo {

namespace {

constexpr int kFwdThreads = 192;
constexpr int kMaxShares = 8;  // CTAs that share a row tile's list: a cluster
// Shared memory of which an SM holds no three CTAs (228 KB, 1 KB of each its own).
// A cluster's CTA keeps its tensor memory, half of the SM's, until the others are
// through; a third on the SM would wait for some, and clusters could wait for each
// other in a ring. (As compiled, 113 registers a thread leave room for two as well.)
constexpr size_t kNoThird = 228 * 1024 / 3 - 1024 + 128;
// The running maximum stays until it is outgrown by 2^32: P (bf16, fp32's range)
// and its sums lose nothing by being large, at most 2^52 here, and the rescaling
// that a smaller bound (2^8) asked for stalled most steps on the last product.
constexpr float kFwdRescaleLog2 = 32.0f;

struct FwdSmem {
  uint64_t q_full, k_full[2], v_full[2], k_empty[2], v_empty[2];
  uint64_t s_full[2], p_full[2], mma_final;
#ifdef SVOO_TEST_STALL
  uint64_t stall;  // test-only: a barrier that nothing completes
#endif
  uint32_t tmem_base;
  int abort;
  int max_limit;
  int tiles;                 // of the list
  int limit[kRowTile];  // per query of the tile
  float2 ml[kRowTile];  // of this share's rows
};

template <int D>
constexpr size_t fwd_tile_bytes() {
  return static_cast<size_t>(kRowTile) * D * 2 + 4 * static_cast<size_t>(kKeyTile) * D * 2;
}

// shared memory before a tile's list
constexpr size_t fwd_smem(int d) {
  return 1024 + (d == 128 ? fwd_tile_bytes<128>() : fwd_tile_bytes<64>()) + sizeof(FwdSmem);
}

// byte of the c4-th 16 bytes of row r of a share's part
template <int D>
__device__ __forceinline__ uint32_t part_at(int r, int c4) {
  return r * (D * 4) + ((c4 ^ (r & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 2)
    block_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, BlockDims p, int cap,
                      const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ lengths, float scale_log2, uint16_t* __restrict__ o,
                      float* __restrict__ lse, int* __restrict__ err) {
  constexpr int kSub = D / 64;
  constexpr int kKvBytes = kKeyTile * D * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = base;
  uint8_t* k_s = q_s + kRowTile * D * 2;  // 2 stages
  uint8_t* v_s = k_s + 2 * kKvBytes;      // 2 stages
  FwdSmem* S = reinterpret_cast<FwdSmem*>(v_s + 2 * kKvBytes);
  TileList tl = tile_list(p, cap, S + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int shares = gridDim.z;
  // a CTA of a cluster stays to its end: the others read its shared memory
  const bool skip = __syncthreads_or(timed_out_before(err) ? 1 : 0) != 0;
  if (skip && shares == 1) return;
  const int b = blockIdx.y / p.Hkv, hk = blockIdx.y - b * p.Hkv;
  const int t0 = blockIdx.x * p.tpt;
  const int nt = min(p.tpt, p.Nq - t0);
  const int len = seq_len(p, lengths, b);
  const int32_t* slots = idx + (static_cast<size_t>(blockIdx.y) * p.Nq + t0) * p.n_sel;

  if (tid == 0) {
    S->abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&S->k_full[s]), 1);
      mbar_init(smem_u32(&S->v_full[s]), 1);
      mbar_init(smem_u32(&S->k_empty[s]), 1);
      mbar_init(smem_u32(&S->v_empty[s]), 1);
      mbar_init(smem_u32(&S->s_full[s]), 1);
      mbar_init(smem_u32(&S->p_full[s]), 4);
    }
    mbar_init(smem_u32(&S->q_full), 1);
    mbar_init(smem_u32(&S->mma_final), 1);
#ifdef SVOO_TEST_STALL
    mbar_init(smem_u32(&S->stall), 1);
#endif
    fence_mbar_init();
    mbar_arrive_expect_tx(smem_u32(&S->q_full), p.tpt * p.G * D * 2);
    load_query_rows<D>(&qmap, q_s, smem_u32(&S->q_full), hk * p.G, t0, b);
  }
  if (warp == 5) {
    __syncwarp();
    tmem_alloc(smem_u32(&S->tmem_base), 256);
    tmem_relinquish();
  }
  int tiles = make_tile_list<kFwdThreads>(p, tl, slots, t0, nt, len, S->limit, &S->max_limit, &S->tiles, err);
  if (skip) tiles = 0;
  if (shares > 1) {  // this CTA's share of the list
    const int per = (tiles + shares - 1) / shares, first = min(tiles, static_cast<int>(blockIdx.z) * per);
    tl.list += first;
    tiles = min(per, tiles - first);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = S->tmem_base;
  volatile int* abort = &S->abort;
  const uint32_t q_u = smem_u32(q_s), k_u = smem_u32(k_s), v_u = smem_u32(v_s);
  int k_armed = -1, v_armed = -1;

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    const size_t row0 = static_cast<size_t>(blockIdx.y) * p.cap;
    auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {
      int okl = 1;
      if (lane == 0) okl = mbar_wait(bar, parity, abort) ? 1 : 0;
      return __shfl_sync(0xffffffffu, okl, 0) != 0;
    };
    auto fill = [&](const CUtensorMap* map, const uint16_t* src, uint8_t* dst, uint32_t bar, int key0) {
      const int valid = len - key0;
      if (valid >= kKeyTile) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, kKvBytes);
          for (int s = 0; s < kSub; ++s)
            tma_load_2d(map, smem_u32(dst) + s * kKeyTile * 128, bar, s * 64, static_cast<int>(row0 + key0));
        }
      } else {
        load_key_rows<D>(dst, src, row0 + key0, valid, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      }
    };
    if (lane == 0) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    for (int j = 0; j < tiles; ++j) {
      const int st = j & 1, key0 = static_cast<int>(tl.list[j] & 0xffffu) * kKeyTile;
      if (j >= 2 && !warp_wait(smem_u32(&S->k_empty[st]), ((j - 2) >> 1) & 1)) break;
      fill(&kmap, k, k_s + st * kKvBytes, smem_u32(&S->k_full[st]), key0);
      k_armed = j;
      if (j >= 2 && !warp_wait(smem_u32(&S->v_empty[st]), ((j - 2) >> 1) & 1)) break;
      fill(&vmap, v, v_s + st * kKvBytes, smem_u32(&S->v_full[st]), key0);
      v_armed = j;
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16_f32(kRowTile, kKeyTile, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(kRowTile, D, false, true);
      auto issue_s = [&](int j) -> bool {
        const int st = j & 1;
        if (!mbar_wait(smem_u32(&S->k_full[st]), (j >> 1) & 1, abort)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t ad = sw128_desc(q_u + (kk >> 2) * kRowTile * 128 + (kk & 3) * 32, 16, 1024);
          const uint64_t bd = sw128_desc(k_u + st * kKvBytes + (kk >> 2) * kKeyTile * 128 + (kk & 3) * 32, 16, 1024);
          umma_f16(tmem + st * 64, ad, bd, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(smem_u32(&S->s_full[st]));
        umma_commit(smem_u32(&S->k_empty[st]));
        return true;
      };
      bool ok = mbar_wait(smem_u32(&S->q_full), 0, abort) && tiles > 0;
#ifdef SVOO_TEST_STALL
      ok = ok && mbar_wait(smem_u32(&S->stall), 0, abort);  // nothing completes it
#endif
      ok = ok && issue_s(0);
      for (int j = 0; j < tiles && ok; ++j) {
        const int st = j & 1;
        // S(j+1) goes where P(j-1) was: its product is ahead in the queue
        if (j + 1 < tiles && !(ok = issue_s(j + 1))) break;
        ok = mbar_wait(smem_u32(&S->p_full[st]), (j >> 1) & 1, abort) &&
             mbar_wait(smem_u32(&S->v_full[st]), (j >> 1) & 1, abort);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kKeyTile / 16; ++kk) {
          const uint64_t bd = sw128_desc(v_u + st * kKvBytes + kk * 16 * 128, kKeyTile * 128, 1024);
          umma_f16_a_tmem(tmem + 128, tmem + st * 64 + kk * 8, bd, idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(smem_u32(&S->v_empty[st]));
      }
      // every MMA of this thread done before the tensor memory goes back
      umma_commit(smem_u32(&S->mma_final));
      mbar_wait_cleanup(smem_u32(&S->mma_final), 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int r = tid;
    const int ti = (r * p.inv_g) >> 16, g = r - ti * p.G;
    const bool live = ti < nt;
    const int lim = live ? S->limit[ti] : 0;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // m: running maximum in log2 units, moved when it is outgrown; l: sum of P in 32 bits, before P is rounded to
    // bf16 for the second product
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const uint32_t* my_word = tl.mask + (live ? ti >> 5 : 0);
    auto visible = [&](int j) {  // keys of tile j that the row sees
      const uint32_t e = tl.list[j];
      const bool sel = live && ((my_word[(e >> 16) * tl.words] >> (ti & 31)) & 1u);
      return sel ? max(0, min(kKeyTile, lim - static_cast<int>(e & 0xffffu) * kKeyTile)) : 0;
    };
    int nv = tiles > 0 ? visible(0) : 0;
    for (int j = 0; j < tiles; ++j) {
      const int st = j & 1;
      const uint32_t s_col = lane_base + st * 64;
      const bool some = __any_sync(0xffffffffu, nv > 0);
      const bool whole = __all_sync(0xffffffffu, nv == kKeyTile || nv == 0);
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->s_full[st]), (j >> 1) & 1, abort));
      if (!ok) break;
      tc_fence_after();
      float alpha = 1.f;
      if (some) {
        float s[kKeyTile];
        tmem_ld32f(s_col, s);
        tmem_ld32f(s_col + 32, s + 32);
        tmem_wait_ld_f(s);
        tmem_wait_ld_f(s + 32);
        if (!whole) {  // a row's own limit falls into this tile
#pragma unroll
          for (int c = 0; c < kKeyTile; ++c)
            if (c >= nv) s[c] = -INFINITY;
        }
        float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kKeyTile; c += 8) {
          m4[0] = fmax3(m4[0], s[c], s[c + 1]);
          m4[1] = fmax3(m4[1], s[c + 2], s[c + 3]);
          if (c + 4 < kKeyTile) {
            m4[2] = fmax3(m4[2], s[c + 4], s[c + 5]);
            m4[3] = fmax3(m4[3], s[c + 6], s[c + 7]);
          }
        }
        const float mx = nv > 0 ? fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * scale_log2 : -INFINITY;
        if (m == -INFINITY) {
          m = mx;  // nothing accumulated yet
        } else if (mx > m + kFwdRescaleLog2) {
          alpha = ex2_approx(m - mx);
          m = mx;
        }
        // a row that does not take part: 2^(s - inf) = 0
        const float nm = nv > 0 ? -m : -INFINITY;
        const uint64_t sc2 = f2pack(scale_log2, scale_log2), nm2 = f2pack(nm, nm);
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float x0, x1;
            f2unpack(f2fma(f2pack(s[h * 32 + 2 * c], s[h * 32 + 2 * c + 1]), sc2, nm2), x0, x1);
            x0 = ex2_approx(x0);
            x1 = ex2_approx(x1);
            pk[c] = pack_bf16x2(x0, x1);
            sum2[c & 1] = f2add(f2pack(x0, x1), sum2[c & 1]);
          }
          tmem_st16(s_col + h * 16, pk);
        }
        float a0, a1, a2, a3;
        f2unpack(sum2[0], a0, a1);
        f2unpack(sum2[1], a2, a3);
        l = l * alpha + ((a0 + a1) + (a2 + a3));
      } else {
        uint32_t z[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) z[c] = 0u;
        tmem_st16(s_col, z);
        tmem_st16(s_col + 16, z);
      }
      // every phase is waited for in turn (v_empty: PV done), or a parity would say too little
      if (j > 1) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->v_empty[st]), ((j - 2) >> 1) & 1, abort));
      if (j > 0 && ok && __any_sync(0xffffffffu, alpha != 1.f)) {
        // O may be touched only between products
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->v_empty[st ^ 1]), ((j - 1) >> 1) & 1, abort));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < D / 16; ++c0) {
          uint32_t x[16];
          tmem_ld16(lane_base + 128 + c0 * 16, x);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * alpha);
          tmem_st16(lane_base + 128 + c0 * 16, x);
        }
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->p_full[st]));
      if (j + 1 < tiles) nv = visible(j + 1);
    }
    // ---------------------------------------------------------------- epilogue
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->mma_final), 0, abort));
    if (!ok) l = 0.f;
    if (shares > 1) S->ml[r] = make_float2(l > 0.f ? m : -INFINITY, l);
    if (ok) {
      tc_fence_after();
      const size_t row = (static_cast<size_t>(b) * p.H + hk * p.G + g) * p.Nq + t0 + ti;
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t x[32];
        if (tiles > 0) {
          tmem_ld32(lane_base + 128 + c0 * 32, x);
          tmem_wait_ld_regs(x);
        }
        if (!live) continue;
        if (shares > 1) {  // where keys and values were; 16-byte pieces of a row in an order that spreads the banks
          if (l > 0.f) {
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4)
              *reinterpret_cast<uint4*>(k_s + part_at<D>(r, c0 * 8 + c4)) =
                  make_uint4(x[c4 * 4], x[c4 * 4 + 1], x[c4 * 4 + 2], x[c4 * 4 + 3]);
          }
          continue;
        }
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
          uint4 pk = make_uint4(0, 0, 0, 0);
          if (l > 0.f) {
            pk.x = pack_bf16x2(__uint_as_float(x[c8 * 8 + 0]) * inv, __uint_as_float(x[c8 * 8 + 1]) * inv);
            pk.y = pack_bf16x2(__uint_as_float(x[c8 * 8 + 2]) * inv, __uint_as_float(x[c8 * 8 + 3]) * inv);
            pk.z = pack_bf16x2(__uint_as_float(x[c8 * 8 + 4]) * inv, __uint_as_float(x[c8 * 8 + 5]) * inv);
            pk.w = pack_bf16x2(__uint_as_float(x[c8 * 8 + 6]) * inv, __uint_as_float(x[c8 * 8 + 7]) * inv);
          }
          reinterpret_cast<uint4*>(o + row * D + c0 * 32)[c8] = pk;
        }
      }
      if (live && shares == 1) lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    if (tid == 0) report_error(err, kErrTimeoutAttn);
    if (warp == 4 && lane == 0) {  // copies still in flight land before the shared memory goes away
      for (int j = max(0, k_armed - 1); j <= k_armed; ++j)
        mbar_wait_cleanup(smem_u32(&S->k_full[j & 1]), (j >> 1) & 1);
      for (int j = max(0, v_armed - 1); j <= v_armed; ++j)
        mbar_wait_cleanup(smem_u32(&S->v_full[j & 1]), (j >> 1) & 1);
      mbar_wait_cleanup(smem_u32(&S->q_full), 0);
    }
    __syncthreads();
  }
  if (shares > 1) {
    // o = sum of the shares' parts, each at its own maximum; a share of the pieces each
    cluster_sync();
    for (int i = blockIdx.z * kFwdThreads + tid; i < nt * p.G * (D / 4); i += shares * kFwdThreads) {
      const int r = i / (D / 4), c4 = i - r * (D / 4), ti = (r * p.inv_g) >> 16, g = r - ti * p.G;
      float2 ml[kMaxShares];
      float4 x[kMaxShares];
      float top = -INFINITY;
#pragma unroll
      for (int z = 0; z < kMaxShares; ++z) {
        ml[z] = z < shares ? cluster_read2(smem_u32(&S->ml[r]), z) : make_float2(-INFINITY, 0.f);
        if (z < shares) x[z] = cluster_read4(smem_u32(k_s + part_at<D>(r, c4)), z);
      }
#pragma unroll
      for (int z = 0; z < kMaxShares; ++z) top = fmaxf(top, ml[z].x);
      float l = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int z = 0; z < kMaxShares; ++z) {
        if (!(ml[z].y > 0.f)) continue;  // the row had nothing there: its part was not written
        const float f = ex2_approx(ml[z].x - top);
        l = fmaf(ml[z].y, f, l);
        a[0] = fmaf(x[z].x, f, a[0]);
        a[1] = fmaf(x[z].y, f, a[1]);
        a[2] = fmaf(x[z].z, f, a[2]);
        a[3] = fmaf(x[z].w, f, a[3]);
      }
      const size_t row = (static_cast<size_t>(b) * p.H + hk * p.G + g) * p.Nq + t0 + ti;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      *reinterpret_cast<uint2*>(o + row * D + c4 * 4) =
          make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
      if (c4 == 0) lse[row] = l > 0.f ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
    cluster_sync();  // nobody leaves while its shared memory is read
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------ by key blocks

// The other way round, for calls whose unions would be nearly all blocks: a CTA
// keeps 128 keys of one block and their values in shared memory and runs through
// the block's list, 128 gathered rows at a time, so that no row works for
// nothing. What a row gets from those keys (a part: O at its own maximum m, and
// m, l) goes to memory in 32 bits, in the list's order; block_parts_kernel finds
// a row's parts by its slots' places in the lists and adds them. The parts' bytes
// bound it (D * 4 per row and 128 keys, written and read), so the way pays only
// where a block has 128 keys or more.
// A row tile's parts lie as [D / 8][rows of the tile][8], so that a warp, whose
// threads have a row each, stores 1 KB at a time: whole rows would be 32 lines a
// store, and kept the load/store unit busy for half of the kernel's time.
// Two CTAs share an SM, each with one row tile in work; stores (32 bytes a clock
// and SM) take as long as the rest, so warps of their own issue them, beside the
// products and the softmax of the next tile. The softmax warps gather the next
// tile's rows (cp.async) as soon as S has been computed.
// Warps: 0-3 gather and softmax (thread = row), 4-7 stores, 8 keys and values
// (TMA), MMA issuer.
// TMEM: S [0,128), P over its first half, O [128,128+D).

constexpr int kListThreads = 288;
constexpr int kListKeys = 2 * kKeyTile;

constexpr int kPartCols = 8;  // columns that a part's rows have together

struct ListSmem {
  uint64_t kv_full[2], full, s_full, p_full, o_full, o_read, mma_final;
#ifdef SVOO_TEST_STALL
  uint64_t stall;  // test-only: a barrier that nothing completes
#endif
  uint32_t tmem_base;
  int abort;
};

template <int D>
constexpr size_t list_tile_bytes() {
  return static_cast<size_t>(2 * kListKeys + kRowTile) * D * 2;
}

__device__ __forceinline__ void st_global_f32x8(float* at, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// Dimensions as the lists' kernels take them here: a key tile is 128 keys.
inline BlockDims list_dims(BlockDims p) {
  p.nsub = p.block / kListKeys;
  return p;
}

// The first part of a block's list for its c-th 128 keys; a list has `rows` rows.
__device__ __forceinline__ size_t list_part(const BlockDims& p, int bh, int start, int rows, int c) {
  return (static_cast<size_t>(bh) * p.Nq * p.n_sel + start) * p.G * p.nsub + static_cast<size_t>(c) * rows;
}

template <int D>
__global__ void __launch_bounds__(kListThreads, 2)
    block_list_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, BlockDims p,
                      int ktiles, int piece, const uint16_t* __restrict__ q, const uint16_t* __restrict__ k,
                      const uint16_t* __restrict__ v, const int32_t* __restrict__ lengths,
                      const int32_t* __restrict__ total, const int32_t* __restrict__ start,
                      const int32_t* __restrict__ list, const int4* __restrict__ items,
                      const int32_t* __restrict__ counts, float scale_log2, float* __restrict__ part_o,
                      float2* __restrict__ part_ml, int* __restrict__ err) {
  constexpr int kKvBytes = kListKeys * D * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* k_s = base;
  uint8_t* v_s = k_s + kKvBytes;
  uint8_t* q_s = v_s + kKvBytes;
  ListSmem* S = reinterpret_cast<ListSmem*>(q_s + kRowTile * D * 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (static_cast<int>(blockIdx.x) >= counts[0]) return;
  if (__syncthreads_or(timed_out_before(err) ? 1 : 0)) return;
  const int4 item = items[blockIdx.x];
  const int bh = item.x / ktiles, kt = item.x - bh * ktiles, key0 = kt * kListKeys;
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int len = seq_len(p, lengths, b);
  const size_t at = static_cast<size_t>(bh) * p.nb + kt / p.nsub;
  const int32_t* toks = list + static_cast<size_t>(bh) * p.Nq * p.n_sel + start[at];
  const long long all_rows = static_cast<long long>(total[at]) * p.G;
  const long long row0 = static_cast<long long>(item.y) * piece;
  const int rows = static_cast<int>(min(static_cast<long long>(piece), all_rows - row0));
  const int nj = (max(rows, 0) + kRowTile - 1) / kRowTile;
  if (nj == 0) return;
  const size_t part0 = list_part(p, bh, start[at], static_cast<int>(all_rows), kt % p.nsub) + row0;

  if (tid == 0) {
    S->abort = 0;
    mbar_init(smem_u32(&S->kv_full[0]), 1);
    mbar_init(smem_u32(&S->kv_full[1]), 1);
    mbar_init(smem_u32(&S->full), 4);  // one arrival per warp
    mbar_init(smem_u32(&S->s_full), 1);
    mbar_init(smem_u32(&S->p_full), 4);
    mbar_init(smem_u32(&S->o_full), 1);
    mbar_init(smem_u32(&S->o_read), 4);
    mbar_init(smem_u32(&S->mma_final), 1);
#ifdef SVOO_TEST_STALL
    mbar_init(smem_u32(&S->stall), 1);
#endif
    fence_mbar_init();
  }
  if (warp == 8) {
    __syncwarp();
    tmem_alloc(smem_u32(&S->tmem_base), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  volatile int* abort = &S->abort;

  if (warp == 8) {
    // ---------------------------------------------------------------- keys, values, MMA issuer
    const size_t krow = static_cast<size_t>(bh) * p.cap;
    const int key[2] = {key0, key0 + kKeyTile < len ? key0 + kKeyTile : -1};
    load_key_pair<D>(&kmap, k, k_s, smem_u32(&S->kv_full[0]), krow, len, key);
    load_key_pair<D>(&vmap, v, v_s, smem_u32(&S->kv_full[1]), krow, len, key);
    __syncwarp();
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16_f32(kRowTile, kListKeys, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(kRowTile, D, false, true);
      const uint32_t k_u = smem_u32(k_s), v_u = smem_u32(v_s), q_u = smem_u32(q_s);
      bool there = mbar_wait(smem_u32(&S->kv_full[0]), 0, abort) && mbar_wait(smem_u32(&S->kv_full[1]), 0, abort);
#ifdef SVOO_TEST_STALL
      there = there && mbar_wait(smem_u32(&S->stall), 0, abort);  // nothing completes it
#endif
      for (int j = 0; j < nj && there; ++j) {
        if (!mbar_wait(smem_u32(&S->full), j & 1, abort)) break;
        tc_fence_after();
        // over P(j-1), whose product is ahead in the queue
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16(tmem, sw128_desc(q_u + (kk >> 2) * kRowTile * 128 + (kk & 3) * 32, 16, 1024),
                   sw128_desc(k_u + (kk >> 2) * kListKeys * 128 + (kk & 3) * 32, 16, 1024), idesc_s, kk > 0 ? 1u : 0u);
        umma_commit(smem_u32(&S->s_full));
        if (!mbar_wait(smem_u32(&S->p_full), j & 1, abort)) break;
        if (j > 0 && !mbar_wait(smem_u32(&S->o_read), (j - 1) & 1, abort)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kListKeys / 16; ++kk)
          umma_f16_a_tmem(tmem + 128, tmem + kk * 8,
                          sw128_desc(v_u + kk * 16 * 128, kListKeys * 128, 1024), idesc_o, kk > 0 ? 1u : 0u);
        umma_commit(smem_u32(&S->o_full));
      }
      umma_commit(smem_u32(&S->mma_final));
      mbar_wait_cleanup(smem_u32(&S->mma_final), 0);
      if (!there) {  // the copies land before the shared memory goes away
        mbar_wait_cleanup(smem_u32(&S->kv_full[0]), 0);
        mbar_wait_cleanup(smem_u32(&S->kv_full[1]), 0);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- stores
    const int r = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128;
    for (int j = 0; j < nj; ++j) {
      const int n = min(kRowTile, rows - j * kRowTile);  // rows of the tile
      float* to = part_o + (part0 + static_cast<size_t>(j) * kRowTile) * D + r * kPartCols;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&S->o_full), j & 1, abort))) break;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t x[2][32];
        tmem_ld32(lane_base + c0, x[0]);
        tmem_ld32(lane_base + c0 + 32, x[1]);
        tmem_wait_ld_regs(x[0]);
        tmem_wait_ld_regs(x[1]);
        if (c0 + 64 == D) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&S->o_read));
        }
        if (r < n) {
#pragma unroll
          for (int c = 0; c < 64; c += 8)
            st_global_f32x8(to + (c0 + c) / kPartCols * n * kPartCols + c % kPartCols, x[c >> 5] + (c & 31));
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- gather, softmax
    const int r = tid;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint64_t sc2 = f2pack(scale_log2, scale_log2);
    const unsigned first_row = static_cast<unsigned>(row0);
    auto entry = [&](int j) {  // the query of this thread's row in tile j, -1 behind the last
      const int f = j * kRowTile + r;
      return f < rows ? toks[(first_row + f) / p.G] : -1;
    };
    auto row_of = [&](int j, int tok) {
      if (tok < 0) return -1;
      return (b * p.H + hk * p.G + static_cast<int>((first_row + j * kRowTile + r) % p.G)) * p.Nq + tok;
    };
    auto keys_of = [&](int tok) {  // that the row sees
      return tok < 0 ? 0 : max(0, min(kListKeys, query_limit(p, len, tok) - key0));
    };
    auto gather = [&](int row) {  // this warp's rows
      constexpr int kChunks = D / 8, kRows = 32 / kChunks;
      const int ch = lane % kChunks, r0 = lane / kChunks;
#pragma unroll
      for (int i = 0; i < 32; i += kRows) {
        const int src = __shfl_sync(0xffffffffu, row, i + r0);
        cp_async16_or_zero(smem_u32(q_s) + sw128_offset(warp * 32 + i + r0, ch * 8, kRowTile),
                           q + static_cast<size_t>(src < 0 ? 0 : src) * D + ch * 8, src >= 0);
      }
    };
    auto landed = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->full));
    };
    int tok = entry(0);
    gather(row_of(0, tok));
    int nv = keys_of(tok);
    tok = entry(1);
    landed();
    for (int j = 0; j < nj; ++j) {
      const bool more = j + 1 < nj;
      const int row = row_of(j + 1, tok), nv_next = keys_of(tok);
      tok = entry(j + 2);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&S->s_full), j & 1, abort))) break;
      tc_fence_after();
      if (more) gather(row);  // S(j) is done with the rows
      const bool whole = __all_sync(0xffffffffu, nv == kListKeys);  // no row's own limit falls into these keys
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float s[32];
        tmem_ld32f(lane_base + h * 32, s);
        tmem_wait_ld_f(s);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (h * 32 + c >= nv) s[c] = -INFINITY;
        }
        float m2[2] = {fmaxf(m, s[0]), s[1]};
#pragma unroll
        for (int c = 2; c < 32; c += 4) {
          m2[0] = fmax3(m2[0], s[c], s[c + 1]);
          if (c + 2 < 32) m2[1] = fmax3(m2[1], s[c + 2], s[c + 3]);
        }
        m = fmaxf(m2[0], m2[1]);
      }
      m *= scale_log2;
      const float nm = m > -INFINITY ? -m : 0.f;  // a row without keys here: P = 2^(-inf - 0) = 0
      const uint64_t nm2 = f2pack(nm, nm);
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // P(h) goes where S(h / 2) was
        float s[32];
        tmem_ld32f(lane_base + h * 32, s);
        tmem_wait_ld_f(s);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (h * 32 + c >= nv) s[c] = -INFINITY;
        }
        uint32_t pk[16];
        uint64_t sum2 = 0ull;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float x0, x1;
          f2unpack(f2fma(f2pack(s[2 * c], s[2 * c + 1]), sc2, nm2), x0, x1);
          x0 = ex2_approx(x0);
          x1 = ex2_approx(x1);
          pk[c] = pack_bf16x2(x0, x1);  // for the second product; l sums them in 32 bits
          sum2 = f2add(f2pack(x0, x1), sum2);
        }
        tmem_st16(lane_base + h * 16, pk);
        float a0, a1;
        f2unpack(sum2, a0, a1);
        l += a0 + a1;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->p_full));
      if (j * kRowTile + r < rows) part_ml[part0 + static_cast<size_t>(j) * kRowTile + r] = make_float2(m, l);
      if (more) landed();
      nv = nv_next;
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort) report_error(err, kErrTimeoutAttn);
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// One warp per row of [B*H*Nq, D], a lane per part: o = sum of the row's parts,
// each at its own maximum.
template <int D>
__global__ void __launch_bounds__(256)
    block_parts_kernel(BlockDims p, const int32_t* __restrict__ idx, const int32_t* __restrict__ lengths,
                       const int32_t* __restrict__ total, const int32_t* __restrict__ start,
                       const int32_t* __restrict__ places, const float* __restrict__ part_o,
                       const float2* __restrict__ part_ml, uint16_t* __restrict__ o, float* __restrict__ lse,
                       int* __restrict__ err) {
  const size_t row = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<size_t>(p.B) * p.H * p.Nq) return;
  constexpr int kE = D / 32, kDeep = 8;
  const int t = static_cast<int>(row % p.Nq), head = static_cast<int>(row / p.Nq);
  const int b = head / p.H, hk = (head - b * p.H) / p.G, g = head % p.G, bh = b * p.Hkv + hk;
  const size_t mine = (static_cast<size_t>(bh) * p.Nq + t) * p.n_sel;
  const int parts = p.n_sel * p.nsub, slot = lane / p.nsub, c = lane % p.nsub;
  // a slot with no place does not count, or lies behind the row's limit, as its
  // later keys may: nobody wrote a part for keys behind the last
  const int lim = query_limit(p, seq_len(p, lengths, b), t);
  const int given = lane < p.n_sel ? idx[mine + lane] : -1;
  const int place = lane < parts ? places[mine + slot] : -1;
  bool bad = false;
  counted_slot(given, p.nb, &bad);
  if (bad && lane == 0) report_error(err, kErrBadPlan);
  const int blk = __shfl_sync(0xffffffffu, given, slot & 31);
  float2 ml = make_float2(-INFINITY, 0.f);
  size_t at = 0;   // of the part's first columns
  int stride = 0;  // from these to the next
  const bool there = place >= 0 && (blk * p.nsub + c) * kListKeys < lim;
  if (there) {
    const size_t cell = static_cast<size_t>(bh) * p.nb + blk;
    const int first = start[cell], rows = total[cell] * p.G, r = (place - first) * p.G + g;
    const int tile = r & ~(kRowTile - 1), n = min(kRowTile, rows - tile);
    const size_t tile0 = list_part(p, bh, first, rows, c) + tile;
    ml = part_ml[tile0 + (r - tile)];
    at = tile0 * D + (r - tile) * kPartCols;
    stride = n * kPartCols;
  }
  float top = ml.x;
#pragma unroll
  for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  const float f = there ? ex2_approx(ml.x - top) : 0.f;
  float l = ml.y * f;
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  float acc[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) acc[e] = 0.f;
  const unsigned all = __ballot_sync(0xffffffffu, there);
  const int c0 = lane * kE / kPartCols, in = lane * kE % kPartCols;  // this lane's columns
  for (int i0 = 0; i0 < parts; i0 += kDeep) {
    float x[kDeep][kE];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const size_t from = __shfl_sync(0xffffffffu, at, (i0 + i) & 31);
      const int by = __shfl_sync(0xffffffffu, stride, (i0 + i) & 31);
      const float* src = part_o + from + static_cast<size_t>(c0 * by + in);
      const bool on = i0 + i < parts && ((all >> ((i0 + i) & 31)) & 1u);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[i][e] = 0.f;
      if (kE == 4) {
        if (on) *reinterpret_cast<float4*>(x[i]) = *reinterpret_cast<const float4*>(src);
      } else {
        if (on) *reinterpret_cast<float2*>(x[i]) = *reinterpret_cast<const float2*>(src);
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, (i0 + i) & 31);
      if (i0 + i < parts)
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = fmaf(x[i][e], fi, acc[e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(o + row * D + lane * kE);
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0) lse[row] = l > 0.f ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// ------------------------------------------------------------------ host side

// Whether a call goes by key blocks. The union of a row tile's selections costs
// time by its size, this way by the selections': it pays from unions of about
// four selections on. A union is as large as that where the queries see more
// than four times the blocks that they select, and the tile's queries are enough
// to name each of them eight times over (neighbouring queries agree). Measured
// (us, union / this, d = 128; neighbours that agree, then independent queries):
//   12 heads, 16380 queries, 16 of 128 blocks   1384 / 840, 1553 / 851
//    8 of 128   846 / 489, 1511 / 480      24 of 128   1495 / 1209, 1554 / 1224
//   causal      892 / 800,  939 / 806      32760 queries, 16 of 256   3058 / 1621
//   16 of 64 blocks, 8192 queries  430 / 452 (not taken: four selections)
//   two heads a group  1005 / 1031, 1574 / 1046   four (not taken)  681 / 1555
// d = 64 (half the parts' bytes): 1430 / 562. Lists and launches cost some 40 us:
// small calls keep to the union. The parts' place stays below 4.3 GB.
inline bool by_blocks(const BlockDims& p) {
  if (p.block % kListKeys || p.n_sel * (p.block / kListKeys) > 32) return false;
  const long long parts = static_cast<long long>(p.B) * p.H * p.Nq * p.n_sel * (p.block / kListKeys);
  if (parts < 1 << 18 || parts > 1 << 23) return false;
  long long seen = p.nb;  // blocks before the middle query
  if (p.causal) {
    const long long middle = (p.q_start >= 0 ? p.q_start : p.Nk - p.Nq) + p.Nq / 2;
    if (middle / p.block + 1 < seen) seen = middle / p.block + 1;
  }
  return seen > 4LL * p.n_sel && static_cast<long long>(p.tpt) * p.n_sel >= 8 * seen;
}

// Shares of a row tile's list: as many as bring two CTAs to every SM, while a
// share may have four key tiles or more (the lists' lengths are not known here,
// their bound is).
inline int block_shares(const BlockDims& p) {
  const long long ctas = static_cast<long long>((p.Nq + p.tpt - 1) / p.tpt) * p.B * p.Hkv;
  if (ctas == 0) return 1;
  const long long longest = static_cast<long long>(union_cap(p)) * p.nsub;
  long long z = 2 * 148 / ctas;
  if (z > longest / 4) z = longest / 4;
  if (z > kMaxShares) z = kMaxShares;
  return z < 1 ? 1 : static_cast<int>(z);
}

// Rows of one piece of a list: an eighth of an SM's share of all, two CTAs an SM.
inline int list_piece(const BlockDims& p) {
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nq * p.n_sel * p.nsub;
  long long piece = (rows / (148 * 8) + kRowTile - 1) / kRowTile * kRowTile;
  return static_cast<int>(piece < 8 * kRowTile ? 8 * kRowTile : piece);
}

struct FwdPlan {
  bool by_blocks;
  BlockDims tile;  // as row tiles take them
  int shares;
  int ktiles, chunk, nchunk, piece;
  long long max_items;
  int32_t *hist, *total, *start, *list, *places, *counts;
  int4* items;
  float* part_o;
  float2* part_ml;
  size_t bytes;
};
FwdPlan fwd_plan(const BlockDims& p, int d, void* ws) {
  FwdPlan f = {};
  f.by_blocks = by_blocks(p);
  f.tile = fit_tile(p, kMaxSmem - fwd_smem(d));
  f.shares = f.by_blocks ? 1 : block_shares(f.tile);
  Carver c(ws);
  size_t parts = 0;
  if (f.by_blocks) {
    const BlockDims lp = list_dims(p);
    const size_t BHk = static_cast<size_t>(p.B) * p.Hkv;
    parts = static_cast<size_t>(p.B) * p.H * p.Nq * p.n_sel * lp.nsub;
    f.ktiles = (p.Nk + kListKeys - 1) / kListKeys;
    f.chunk = sel_chunk(p);
    f.nchunk = (p.Nq + f.chunk - 1) / f.chunk;
    f.piece = list_piece(lp);
    f.max_items = static_cast<long long>(BHk * f.ktiles + parts / f.piece);
    f.hist = c.take<int32_t>(BHk * f.nchunk * p.nb);
    f.total = c.take<int32_t>(BHk * p.nb);
    f.start = c.take<int32_t>(BHk * p.nb);
    f.list = c.take<int32_t>(BHk * p.Nq * p.n_sel);
    f.places = c.take<int32_t>(BHk * p.Nq * p.n_sel);
    f.counts = c.take<int32_t>(2);
    f.items = c.take<int4>(static_cast<size_t>(f.max_items));
  }
  f.part_o = c.take<float>(parts * d);
  f.part_ml = c.take<float2>(parts);
  f.bytes = (c.used + 255) / 256 * 256;
  return f;
}

template <int D>
svoo_status launch_block_lists(const BlockDims& p, const FwdPlan& f, const uint16_t* q, const uint16_t* k,
                               const uint16_t* v, const int32_t* idx, const int32_t* lengths, float scale_log2,
                               uint16_t* o, float* lse, int32_t* dev_err, cudaStream_t st) {
  const BlockDims lp = list_dims(p);
  const int BHk = p.B * p.Hkv;
  CUtensorMap km, vm;
  const uint64_t krows = mapped_key_rows(p);
  if (encode_tiled_2d(&km, k, krows, D, kKeyTile, 64) != CUDA_SUCCESS ||
      encode_tiled_2d(&vm, v, krows, D, kKeyTile, 64) != CUDA_SUCCESS)
    return SVOO_ERR_CUDA;
  const size_t smem = 1024 + list_tile_bytes<D>() + sizeof(ListSmem), cnt = static_cast<size_t>(p.nb) * 4;
  if (!allow_smem(block_list_kernel<D>, smem) || !allow_smem(sel_walk_kernel<kSelCount>, kMaxBlocks * 4) ||
      !allow_smem(sel_walk_kernel<kSelPlaces>, kMaxBlocks * 4))
    return SVOO_ERR_CUDA;
  sel_walk_kernel<kSelCount><<<dim3(f.nchunk, BHk), 32, cnt, st>>>(lp, idx, lengths, f.chunk, f.nchunk, f.hist,
                                                                   nullptr, nullptr, nullptr);
  sel_scan_kernel<<<dim3((p.nb + 31) / 32, BHk), 256, 0, st>>>(lp, f.nchunk, f.hist, f.total);
  sel_items_kernel<<<1, 1024, 0, st>>>(lp, f.ktiles, f.piece, f.total, f.start, f.items, f.counts);
  sel_walk_kernel<kSelPlaces><<<dim3(f.nchunk, BHk), 32, cnt, st>>>(lp, idx, lengths, f.chunk, f.nchunk, f.hist,
                                                                    f.start, f.list, f.places);
  block_list_kernel<D><<<static_cast<unsigned>(f.max_items), kListThreads, smem, st>>>(
      km, vm, lp, f.ktiles, f.piece, q, k, v, lengths, f.total, f.start, f.list, f.items, f.counts, scale_log2, f.part_o,
      f.part_ml, dev_err);
  const size_t rows = static_cast<size_t>(p.B) * p.H * p.Nq;
  block_parts_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(lp, idx, lengths, f.total, f.start,
                                                                               f.places, f.part_o, f.part_ml, o, lse,
                                                                               dev_err);
  return launch_status();
}

template <int D>
svoo_status launch_block_attn(const BlockDims& p, const void* q, const void* k, const void* v, const int32_t* idx,
                              const int32_t* lengths, float scale, void* o, float* lse, void* ws, int32_t* dev_err,
                              cudaStream_t st) {
  const FwdPlan f = fwd_plan(p, D, ws);
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (f.by_blocks)
    return launch_block_lists<D>(p, f, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                                 static_cast<const uint16_t*>(v), idx, lengths, scale_log2, static_cast<uint16_t*>(o),
                                 lse, dev_err, st);
  const BlockDims& t = f.tile;
  CUtensorMap qm, km, vm;
  const uint64_t rows = mapped_key_rows(t);
  if (encode_token_major(&qm, q, t.B, t.H, t.Nq, D, t.G, t.tpt) != CUDA_SUCCESS ||
      encode_tiled_2d(&km, k, rows, D, kKeyTile, 64) != CUDA_SUCCESS ||
      encode_tiled_2d(&vm, v, rows, D, kKeyTile, 64) != CUDA_SUCCESS)
    return SVOO_ERR_CUDA;
  if (!allow_smem(block_attn_kernel<D>, kMaxSmem)) return SVOO_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((t.Nq + t.tpt - 1) / t.tpt, t.B * t.Hkv, f.shares);
  cfg.blockDim = dim3(kFwdThreads);
  cfg.dynamicSmemBytes = fwd_smem(D) + tile_list_bytes(t);
  if (f.shares > 1 && cfg.dynamicSmemBytes < kNoThird) cfg.dynamicSmemBytes = kNoThird;
  cfg.stream = st;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = f.shares;
  cfg.attrs = &cluster;
  cfg.numAttrs = f.shares > 1 ? 1 : 0;
  cudaLaunchKernelEx(&cfg, block_attn_kernel<D>, qm, km, vm, t, static_cast<int>(union_cap(t)),
                     static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), idx, lengths, scale_log2,
                     static_cast<uint16_t*>(o), lse, static_cast<int*>(dev_err));
  return launch_status();
}

}  // namespace

}  // namespace svoo

using namespace svoo;

extern "C" size_t svoo_block_attn_workspace_size(const svoo_block_shape* shape) {
  if (!block_shape_ok(shape)) return 0;
  return fwd_plan(block_dims(shape), shape->d, nullptr).bytes;
}

extern "C" svoo_status svoo_block_attn(const svoo_block_shape* shape, const void* q, const void* k, const void* v,
                                       const int32_t* idx, const int32_t* lengths, float scale, void* o, float* lse,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  if (!block_shape_ok(shape) || !scale_ok(scale)) return SVOO_ERR_INVALID_ARG;
  if (shape->Nq == 0) return SVOO_OK;  // empty tensors have no address
  if (!q || !k || !v || !idx || !o || !lse) return SVOO_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(idx, 4) ||
      !aligned(lse, 4) || !aligned(lengths, 4) || !aligned(dev_err, 4) || !aligned(workspace, 256))
    return SVOO_ERR_INVALID_ARG;
  const BlockDims p = block_dims(shape);
  const size_t need = fwd_plan(p, shape->d, nullptr).bytes;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SVOO_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128) return launch_block_attn<128>(p, q, k, v, idx, lengths, scale, o, lse, workspace, dev_err, st);
  return launch_block_attn<64>(p, q, k, v, idx, lengths, scale, o, lse, workspace, dev_err, st);
}
