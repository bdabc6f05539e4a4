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
// worst case the union is what dense attention would read.
//
// Where there are few row tiles, a tile's list is shared out to several CTAs
// (grid.z), whose parts block_join_kernel puts together.
//
// Two CTAs share an SM (256 tensor-memory columns and half of the shared
// memory each), so one's softmax runs beside the other's products.
// Warps: 0-3 softmax (thread r = row r = TMEM lane r), 4 key/value producer
// (TMA; the tile that crosses the sequence's end by plain loads with zeros
// behind it), 5 MMA issuer, which runs S(j+1) ahead of the softmax of tile j.
// TMEM: S [0,64) and [64,128) alternating, P over the S that it came from,
// O [128,128+D).
#include "blocks.cuh"

namespace svoo {

namespace {

constexpr int kFwdThreads = 192;
constexpr int kMaxShares = 16;  // CTAs that share a row tile's list
// The running maximum stays until it is outgrown by 2^32: P (bf16, fp32's range)
// and its sums lose nothing by being large, at most 2^52 here, and the rescaling
// that a smaller bound (2^8) asked for stalled most steps on the last product.
constexpr float kFwdRescaleLog2 = 32.0f;

struct FwdSmem {
  uint64_t q_full, k_full[2], v_full[2], k_empty[2], v_empty[2];
  uint64_t s_full[2], p_full[2], mma_final;
  uint32_t tmem_base;
  int abort;
  int max_limit;
  int tiles;                 // of the list
  int limit[kRowTile];  // per query of the tile
};

template <int D>
constexpr size_t fwd_tile_bytes() {
  return static_cast<size_t>(kRowTile) * D * 2 + 4 * static_cast<size_t>(kKeyTile) * D * 2;
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 2)
    block_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, BlockDims p, int cap,
                      const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ lengths, float scale_log2, uint16_t* __restrict__ o,
                      float* __restrict__ lse, float* __restrict__ part_o, float2* __restrict__ part_ml,
                      int* __restrict__ err) {
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
  if (__syncthreads_or(timed_out_before(err) ? 1 : 0)) return;
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
  if (gridDim.z > 1) {  // this CTA's share of the list
    const int per = (tiles + gridDim.z - 1) / gridDim.z, first = min(tiles, static_cast<int>(blockIdx.z) * per);
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
      bool ok = mbar_wait(smem_u32(&S->q_full), 0, abort) && tiles > 0 && issue_s(0);
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
    if (ok) {
      tc_fence_after();
      const size_t row = (static_cast<size_t>(b) * p.H + hk * p.G + g) * p.Nq + t0 + ti;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const bool part = gridDim.z > 1;
      const size_t at = blockIdx.z * (static_cast<size_t>(p.B) * p.H * p.Nq) + row;  // of a part
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t x[32];
        if (tiles > 0) {
          tmem_ld32(lane_base + 128 + c0 * 32, x);
          tmem_wait_ld_regs(x);
        }
        if (!live) continue;
        if (part) {
          if (l > 0.f) {
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4)
              *reinterpret_cast<uint4*>(part_o + at * D + c0 * 32 + c4 * 4) =
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
      if (live && part) part_ml[at] = make_float2(m, l);
      if (live && !part) lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
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
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// One warp per row of [B*H*Nq, D]: o = sum of the shares' parts, each at its own
// maximum. A share that the row had nothing in (l = 0) wrote no part.
template <int D>
__global__ void __launch_bounds__(256)
    block_join_kernel(size_t rows, int shares, const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                      uint16_t* __restrict__ o, float* __restrict__ lse) {
  const size_t row = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  constexpr int kE = D / 32;
  float2 ml[kMaxShares];
  float top = -INFINITY, l = 0.f, acc[kE];
#pragma unroll
  for (int z = 0; z < kMaxShares; ++z) {
    ml[z] = z < shares ? part_ml[z * rows + row] : make_float2(-INFINITY, 0.f);
    if (ml[z].y > 0.f) top = fmaxf(top, ml[z].x);
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) acc[e] = 0.f;
#pragma unroll
  for (int z = 0; z < kMaxShares; ++z) {
    if (!(ml[z].y > 0.f)) continue;
    const float f = ex2_approx(ml[z].x - top);
    l = fmaf(ml[z].y, f, l);
    const float2* src = reinterpret_cast<const float2*>(part_o + (z * rows + row) * D + lane * kE);
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) {
      const float2 x = src[e];
      acc[2 * e] = fmaf(x.x, f, acc[2 * e]);
      acc[2 * e + 1] = fmaf(x.y, f, acc[2 * e + 1]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(o + row * D + lane * kE);
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0) lse[row] = l > 0.f ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY;
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

struct FwdPlan {
  int shares;
  float* part_o;
  float2* part_ml;
  size_t bytes;
};
FwdPlan fwd_plan(const BlockDims& p, int d, void* ws) {
  FwdPlan f;
  f.shares = block_shares(p);
  const size_t rows = f.shares > 1 ? static_cast<size_t>(f.shares) * p.B * p.H * p.Nq : 0;
  Carver c(ws);
  f.part_o = c.take<float>(rows * d);
  f.part_ml = c.take<float2>(rows);
  f.bytes = (c.used + 255) / 256 * 256;
  return f;
}

template <int D>
svoo_status launch_block_attn(const BlockDims& p, const void* q, const void* k, const void* v, const int32_t* idx,
                              const int32_t* lengths, float scale, void* o, float* lse, void* ws, int32_t* dev_err,
                              cudaStream_t st) {
  const FwdPlan f = fwd_plan(p, D, ws);
  CUtensorMap qm, km, vm;
  const uint64_t rows = static_cast<uint64_t>(p.B) * p.Hkv * p.cap;
  if (encode_token_major(&qm, q, p.B, p.H, p.Nq, D, p.G, p.tpt) != CUDA_SUCCESS ||
      encode_tiled_2d(&km, k, rows, D, kKeyTile, 64) != CUDA_SUCCESS ||
      encode_tiled_2d(&vm, v, rows, D, kKeyTile, 64) != CUDA_SUCCESS)
    return SVOO_ERR_CUDA;
  const size_t smem = 1024 + fwd_tile_bytes<D>() + sizeof(FwdSmem) + tile_list_bytes(p);
  if (cudaFuncSetAttribute(block_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return SVOO_ERR_CUDA;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  block_attn_kernel<D><<<dim3((p.Nq + p.tpt - 1) / p.tpt, p.B * p.Hkv, f.shares), kFwdThreads, smem, st>>>(
      qm, km, vm, p, static_cast<int>(union_cap(p)), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), idx, lengths, scale_log2, static_cast<uint16_t*>(o), lse, f.part_o, f.part_ml,
      dev_err);
  if (f.shares > 1) {
    const size_t qrows = static_cast<size_t>(p.B) * p.H * p.Nq;
    block_join_kernel<D><<<static_cast<unsigned>((qrows + 7) / 8), 256, 0, st>>>(qrows, f.shares, f.part_o, f.part_ml,
                                                                                static_cast<uint16_t*>(o), lse);
  }
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
      !aligned(lse, 4) || !aligned(lengths, 4) || !aligned(workspace, 256))
    return SVOO_ERR_INVALID_ARG;
  const BlockDims p = block_dims(shape);
  const size_t need = fwd_plan(p, shape->d, nullptr).bytes;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SVOO_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128) return launch_block_attn<128>(p, q, k, v, idx, lengths, scale, o, lse, workspace, dev_err, st);
  return launch_block_attn<64>(p, q, k, v, idx, lengths, scale, o, lse, workspace, dev_err, st);
}
