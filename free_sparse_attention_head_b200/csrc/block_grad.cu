// block_grad.cu -- gradient of the block-selected attention, sm_100a. The
// selection is a constant of the gradient.
//
//   P = exp(scale q K^T - lse), delta = rowsum(do * o), dS = P * (do V^T - delta)
//   dq = scale dS K,   dk = scale dS^T q,   dv = P^T do
//
// P is computed again from lse in both kernels rather than kept: two products
// of 64 keys cost less than its bytes.
//
//   block_dq_kernel      delta, and dq: row tiles against the union of their
//                        blocks, as the forward kernel walks it
//   sel_walk / sel_scan / sel_items (block_lists.cuh)
//                        for every block the list of the queries that selected
//                        it, in a fixed order (no atomics decide a place)
//   block_dkv_kernel     dk, dv: one key tile against its list's rows, gathered
//                        128 at a time, so no row computes for nothing
//   block_dkv_sum_kernel long lists (a block that every query keeps) are cut
//                        into pieces; their parts are added in order
//
// Every sum runs in a fixed order: two calls give the same bits.
#include "block_lists.cuh"

namespace svoo {

namespace {

// ------------------------------------------------------------------ dq

// Row tiles as in the forward kernel, in steps of two 64-key tiles; P needs no
// maximum here, so the two tiles of a step are two groups of warps that never
// meet. One CTA per SM. Q and dO are the products' first operand from tensor
// memory: from shared memory, each product would read its 32 KB anew, and the
// step was bound by shared memory's bandwidth (2400 cycles, for 1540 of the
// tensor core). dS goes over dP, so that S(j+1) can follow as soon as S(j) has
// been read, under the work on dS(j); dQ(j) and dP(j+1) follow that.
// dS goes into its product as two bf16 parts, 16 bits of it: rows of dS sum to
// zero, so that one part's rounding is as large in dq as that of the output
// (relative to the formula in 64 bits 2.9e-3 in all, with two parts 2.2e-3,
// for 632 -> 784 us at 16,384 tokens with 16/4 heads).
// Warps: 0-3, 4-7 dS of a step's first / second tile (thread = row), 8 key and
// value producer, 9 MMA issuer.
// TMEM: S [0,128); dP [128,256), the parts of dS over each tile's half of it;
// dQ [256,256+D); Q [384,384+D/2), dO [448,448+D/2).

constexpr int kDqThreads = 320;
constexpr int kDqPair = 2 * kKeyTile;
constexpr int kDqK = 3;  // stages of K: dQ(j) still reads one while S(j+1) reads the next
constexpr int kDqV = 2;  // stages of V, where Q and dO pass through first

struct DqSmem {
  uint64_t k_full[kDqK], k_empty[kDqK], v_full[kDqV], v_empty[kDqV];
  uint64_t q_full, s_full, s_read, dp_full, ds_full, mma_final;
#ifdef SVOO_TEST_STALL
  uint64_t stall;  // test-only: a barrier that nothing completes
#endif
  uint32_t tmem_base;
  int abort;
  int max_limit;
  int tiles;
  int limit[kRowTile];
  float delta[kRowTile];
};

// shared memory before a tile's list
template <int D>
constexpr size_t dq_smem() {
  return static_cast<size_t>(kDqK + kDqV) * kDqPair * D * 2 + sizeof(DqSmem);
}

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
    block_dq_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap gmap,
                    const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, BlockDims p, int cap, const uint16_t* __restrict__ k,
                    const uint16_t* __restrict__ v, const float* __restrict__ lse, float* __restrict__ delta, const int32_t* __restrict__ idx,
                    const int32_t* __restrict__ lengths, float scale, float scale_log2, uint16_t* __restrict__ dq,
                    int* __restrict__ err) {
  constexpr int kSub = D / 64;
  constexpr int kHalfBytes = kKeyTile * D * 2;
  constexpr int kPairBytes = 2 * kHalfBytes;
  constexpr int kRowBytes = kRowTile * D * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // no room to round up in: the declared alignment has to hold
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) report_error(err, kErrBadPlan);
    return;
  }
  uint8_t* k_s = smem_raw;
  uint8_t* v_s = k_s + kDqK * kPairBytes;
  static_assert(kDqV * kPairBytes == 2 * kRowBytes, "Q and dO where V goes later");
  uint8_t* q_s = v_s;
  uint8_t* g_s = q_s + kRowBytes;
  uint8_t* o_s = k_s;  // and o, for delta, where K goes later
  DqSmem* S = reinterpret_cast<DqSmem*>(v_s + kDqV * kPairBytes);
  const TileList tl = tile_list(p, cap, S + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (__syncthreads_or(timed_out_before(err) ? 1 : 0)) return;
  const int b = blockIdx.y / p.Hkv, hk = blockIdx.y - b * p.Hkv;
  const int t0 = blockIdx.x * p.tpt;
  const int nt = min(p.tpt, p.Nq - t0);
  const int len = seq_len(p, lengths, b);
  const int32_t* slots = idx + (static_cast<size_t>(blockIdx.y) * p.Nq + t0) * p.n_sel;

  if (tid == 0) {
    S->abort = 0;
    for (int s = 0; s < kDqK; ++s) {
      mbar_init(smem_u32(&S->k_full[s]), 1);
      mbar_init(smem_u32(&S->k_empty[s]), 1);
    }
    for (int s = 0; s < kDqV; ++s) {
      mbar_init(smem_u32(&S->v_full[s]), 1);
      mbar_init(smem_u32(&S->v_empty[s]), 1);
    }
    mbar_init(smem_u32(&S->s_full), 1);
    mbar_init(smem_u32(&S->s_read), 8);   // one arrival per dS warp
    mbar_init(smem_u32(&S->dp_full), 1);
    mbar_init(smem_u32(&S->ds_full), 8);
    mbar_init(smem_u32(&S->q_full), 1);
    mbar_init(smem_u32(&S->mma_final), 1);
#ifdef SVOO_TEST_STALL
    mbar_init(smem_u32(&S->stall), 1);
#endif
    fence_mbar_init();
    const uint32_t bar = smem_u32(&S->q_full);
    mbar_arrive_expect_tx(bar, 3 * p.tpt * p.G * D * 2);
    load_query_rows<D>(&qmap, q_s, bar, hk * p.G, t0, b);
    load_query_rows<D>(&gmap, g_s, bar, hk * p.G, t0, b);
    load_query_rows<D>(&omap, o_s, bar, hk * p.G, t0, b);
  }
  if (warp == 9) {
    __syncwarp();
    tmem_alloc(smem_u32(&S->tmem_base), 512);
    tmem_relinquish();
  }
  const int tiles = make_tile_list<kDqThreads>(p, tl, slots, t0, nt, len, S->limit, &S->max_limit, &S->tiles, err);
  const int steps = (tiles + 1) / 2;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = S->tmem_base;
  volatile int* abort = &S->abort;
  const uint32_t k_u = smem_u32(k_s), v_u = smem_u32(v_s);
  const bool loaded = mbar_wait(smem_u32(&S->q_full), 0, abort);
  __syncwarp();
  if (warp < 8 && loaded) {
    // group 0 moves its row of Q to tensor memory, group 1 its row of dO, and
    // takes delta from it on the way
    const int h = warp >> 2, r = tid & 127, ti = (r * p.inv_g) >> 16, g = r - ti * p.G;
    const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 384 + h * 64;
    const uint8_t* from = h ? g_s : q_s;
    float dl = 0.f;
#pragma unroll
    for (int c4 = 0; c4 < D / 32; ++c4) {
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = sw128_offset(r, (c4 * 4 + i) * 8, kRowTile);
        const uint4 y = *reinterpret_cast<const uint4*>(from + at);
        x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
        if (h) {
          const uint4 z = *reinterpret_cast<const uint4*>(o_s + at);
          const uint32_t zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
          for (int k2 = 0; k2 < 4; ++k2) {
            dl = fmaf(__uint_as_float(x[4 * i + k2] << 16), __uint_as_float(zs[k2] << 16), dl);
            dl = fmaf(__uint_as_float(x[4 * i + k2] & 0xffff0000u), __uint_as_float(zs[k2] & 0xffff0000u), dl);
          }
        }
      }
      tmem_st16(to + c4 * 16, x);
    }
    if (h) {
      S->delta[r] = dl;
      if (ti < nt) delta[(static_cast<size_t>(b) * p.H + hk * p.G + g) * p.Nq + t0 + ti] = dl;
    }
    tmem_wait_st();
  }
  fence_proxy_async_smem();  // the rows' place goes to the TMA
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int k_armed = -1, v_armed = -1;

  if (warp == 8) {
    // ---------------------------------------------------------------- producer
    const size_t row0 = static_cast<size_t>(blockIdx.y) * p.cap;
    auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {
      int okl = 1;
      if (lane == 0) okl = mbar_wait(bar, parity, abort) ? 1 : 0;
      return __shfl_sync(0xffffffffu, okl, 0) != 0;
    };
    if (lane == 0) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    for (int j = 0; j < steps; ++j) {
      const int ks = j % kDqK, vs = j % kDqV;
      const int key[2] = {static_cast<int>(tl.list[2 * j] & 0xffffu) * kKeyTile,
                          2 * j + 1 < tiles ? static_cast<int>(tl.list[2 * j + 1] & 0xffffu) * kKeyTile : -1};
      if (j >= kDqK && !warp_wait(smem_u32(&S->k_empty[ks]), (j / kDqK - 1) & 1)) break;
      load_key_pair<D>(&kmap, k, k_s + ks * kPairBytes, smem_u32(&S->k_full[ks]), row0, len, key);
      k_armed = j;
      if (j >= kDqV && !warp_wait(smem_u32(&S->v_empty[vs]), (j / kDqV - 1) & 1)) break;
      load_key_pair<D>(&vmap, v, v_s + vs * kPairBytes, smem_u32(&S->v_full[vs]), row0, len, key);
      v_armed = j;
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16_f32(kRowTile, kDqPair, false, false);
      const uint32_t idesc_q = idesc_bf16_f32(kRowTile, D, false, true);
      auto rows_by_keys = [&](uint32_t d, uint32_t a_tmem, uint32_t b_u) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16_a_tmem(d, a_tmem + kk * 8, sw128_desc(b_u + (kk >> 2) * kDqPair * 128 + (kk & 3) * 32, 16, 1024),
                          idesc_s, kk > 0 ? 1u : 0u);
      };
      auto issue_s = [&](int j) -> bool {  // S(j-1) has been read
        if (!mbar_wait(smem_u32(&S->k_full[j % kDqK]), (j / kDqK) & 1, abort)) return false;
        tc_fence_after();
        rows_by_keys(tmem, tmem + 384, k_u + (j % kDqK) * kPairBytes);
        umma_commit(smem_u32(&S->s_full));
        return true;
      };
      auto issue_dp = [&](int j) -> bool {  // over dS(j-1), whose product is ahead in the queue
        const int vs = j % kDqV;
        if (!mbar_wait(smem_u32(&S->v_full[vs]), (j / kDqV) & 1, abort)) return false;
        tc_fence_after();
        rows_by_keys(tmem + 128, tmem + 448, v_u + vs * kPairBytes);
        umma_commit(smem_u32(&S->dp_full));
        umma_commit(smem_u32(&S->v_empty[vs]));
        return true;
      };
      bool ok = steps > 0;
#ifdef SVOO_TEST_STALL
      ok = ok && mbar_wait(smem_u32(&S->stall), 0, abort);  // nothing completes it
#endif
      ok = ok && issue_s(0) && issue_dp(0);
      for (int j = 0; j < steps && ok; ++j) {
        const bool more = j + 1 < steps;
        if (more && (!mbar_wait(smem_u32(&S->s_read), j & 1, abort) || !issue_s(j + 1))) break;
        if (!mbar_wait(smem_u32(&S->ds_full), j & 1, abort)) break;
        tc_fence_after();
        const uint32_t kt = k_u + (j % kDqK) * kPairBytes;
#pragma unroll
        for (int kk = 0; kk < 2 * kDqPair / 16; ++kk) {
          const int part = kk & 1, key = kk >> 1;  // 16 keys
          umma_f16_a_tmem(tmem + 256, tmem + 128 + (key >> 2) * 64 + part * 32 + (key & 3) * 8,
                          sw128_desc(kt + key * 16 * 128, kDqPair * 128, 1024), idesc_q, (j > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(smem_u32(&S->k_empty[j % kDqK]));
        if (more && !issue_dp(j + 1)) break;
      }
      umma_commit(smem_u32(&S->mma_final));
      mbar_wait_cleanup(smem_u32(&S->mma_final), 0);
    }
  } else {
    // ---------------------------------------------------------------- dS
    const int h = warp >> 2, r = tid & 127;  // tile of the step, row
    const int ti = (r * p.inv_g) >> 16, g = r - ti * p.G;
    const bool live = ti < nt;
    const int lim = live ? S->limit[ti] : 0;
    const size_t row = (static_cast<size_t>(b) * p.H + hk * p.G + (live ? g : 0)) * p.Nq + t0 + (live ? ti : 0);
    const float lse2 = lse[row] * 1.4426950408889634f;
    const float dl = S->delta[r];
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t* my_word = tl.mask + (live ? ti >> 5 : 0);
    auto visible = [&](int j) {  // keys of this thread's tile in step j that the row sees
      if (2 * j + h >= tiles) return 0;
      const uint32_t e = tl.list[2 * j + h];
      const bool sel = live && ((my_word[(e >> 16) * tl.words] >> (ti & 31)) & 1u);
      return sel ? max(0, min(kKeyTile, lim - static_cast<int>(e & 0xffffu) * kKeyTile)) : 0;
    };
    const uint64_t sc2 = f2pack(scale_log2, scale_log2), nd2 = f2pack(-dl, -dl);
    bool ok = true;
    int nv = steps > 0 ? visible(0) : 0;
    for (int j = 0; j < steps; ++j) {
      const bool some = __any_sync(0xffffffffu, nv > 0);
      const bool whole = __all_sync(0xffffffffu, nv == kKeyTile || nv == 0);
      const uint32_t s_col = lane_base + h * kKeyTile, p_col = s_col + 128;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->s_full), j & 1, abort));
      if (!ok) break;
      tc_fence_after();
      float s[kKeyTile];
      if (some) {
        tmem_ld32f(s_col, s);
        tmem_ld32f(s_col + 32, s + 32);
        tmem_wait_ld_f(s);
        tmem_wait_ld_f(s + 32);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->s_read));
      if (some) {
        if (!whole) {  // the row's own limit falls into this tile
#pragma unroll
          for (int c = 0; c < kKeyTile; ++c)
            if (c >= nv) s[c] = -INFINITY;
        }
        // P = 2^(s - lse); a row that does not take part: 2^(s - inf) = 0
        const float nl = nv > 0 ? -lse2 : -INFINITY;
        const uint64_t nl2 = f2pack(nl, nl);
#pragma unroll
        for (int c = 0; c < kKeyTile; c += 2) {
          f2unpack(f2fma(f2pack(s[c], s[c + 1]), sc2, nl2), s[c], s[c + 1]);
          s[c] = ex2_approx(s[c]);
          s[c + 1] = ex2_approx(s[c + 1]);
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->dp_full), j & 1, abort));
      if (!ok) break;
      tc_fence_after();
      uint32_t pk[32], lo[32];
      if (some) {
        // dS = P (dP - delta), as two bf16 parts
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
          float x[32];
          tmem_ld32f(p_col + q4 * 32, x);
          tmem_wait_ld_f(x);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float e0, e1;
            f2unpack(f2mul(f2pack(s[q4 * 32 + 2 * c], s[q4 * 32 + 2 * c + 1]),
                           f2add(f2pack(x[2 * c], x[2 * c + 1]), nd2)),
                     e0, e1);
            const uint32_t hi = pack_bf16x2(e0, e1);
            pk[q4 * 16 + c] = hi;
            lo[q4 * 16 + c] = pack_bf16x2(e0 - __uint_as_float(hi << 16), e1 - __uint_as_float(hi & 0xffff0000u));
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = lo[c] = 0u;
      }
      tmem_st32(p_col, pk);  // over dP that this warp alone has read
      tmem_st32(p_col + 32, lo);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->ds_full));
      if (j + 1 < steps) nv = visible(j + 1);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->mma_final), 0, abort));
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < D / 64; ++c0) {  // half of the columns each
        const int col = h * (D / 2) + c0 * 32;
        uint32_t x[32];
        if (steps > 0) {
          tmem_ld32(lane_base + 256 + col, x);
          tmem_wait_ld_regs(x);
        }
        if (live) {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (steps > 0 && lim > 0) {  // a query outside its sequence may hold anything
              w.x = pack_bf16x2(__uint_as_float(x[c8 * 8 + 0]) * scale, __uint_as_float(x[c8 * 8 + 1]) * scale);
              w.y = pack_bf16x2(__uint_as_float(x[c8 * 8 + 2]) * scale, __uint_as_float(x[c8 * 8 + 3]) * scale);
              w.z = pack_bf16x2(__uint_as_float(x[c8 * 8 + 4]) * scale, __uint_as_float(x[c8 * 8 + 5]) * scale);
              w.w = pack_bf16x2(__uint_as_float(x[c8 * 8 + 6]) * scale, __uint_as_float(x[c8 * 8 + 7]) * scale);
            }
            reinterpret_cast<uint4*>(dq + row * D + col)[c8] = w;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    if (tid == 0) report_error(err, kErrTimeoutAttn);
    if (warp == 8 && lane == 0) {  // copies still in flight land before the shared memory goes away
      for (int j = max(0, k_armed - kDqK + 1); j <= k_armed; ++j)
        mbar_wait_cleanup(smem_u32(&S->k_full[j % kDqK]), (j / kDqK) & 1);
      for (int j = max(0, v_armed - kDqV + 1); j <= v_armed; ++j)
        mbar_wait_cleanup(smem_u32(&S->v_full[j % kDqV]), (j / kDqV) & 1);
      mbar_wait_cleanup(smem_u32(&S->q_full), 0);
    }
    __syncthreads();
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dk, dv

// threads; 128 of them took longer to issue a tile's 64 KB (585 us against 551 for the case below, which 32-bit row
// numbers then brought to 526)
constexpr int kDkvLoaders = 256;
constexpr int kDkvThreads = 256 + kDkvLoaders + 32;  // warps 0-3, 4-7: dS of even / odd row tiles; 8-15: loads; 16: MMA issuer
constexpr int kDkvIssuer = kDkvThreads / 32 - 1;

struct DkvSmem {
  uint64_t full[2], free_[2], s_full[2], ds_full[2], mma_final;
#ifdef SVOO_TEST_STALL
  uint64_t stall;  // test-only: a barrier that nothing completes
#endif
  uint32_t tmem_base;
  int abort;
  float lse2[2][kRowTile];
  float delta[2][kRowTile];
  uint8_t nv[2][kRowTile];  // valid keys of the row in this key tile
  int row[kRowTile];        // gather: the rows of the tile being loaded
};

template <int D>
constexpr size_t dkv_tile_bytes() {
  return 2 * static_cast<size_t>(kKeyTile) * D * 2 + 4 * static_cast<size_t>(kRowTile) * D * 2 +
         4 * static_cast<size_t>(kRowTile) * kKeyTile * 2;
}

// Per row tile: S = Q K^T and dP = dO V^T (rows x 64 keys) into tensor memory;
// P and dS back to shared memory in bf16; dV^T += dO^T P and dK^T += Q^T dS
// with the model dimension as the product's 128 rows (d = 64: dO and Q side by
// side, each product uses its own half of the lanes), so that a tile of 64
// keys runs at M = 128.
// Bound by the chain of a stage (rows in, two products, dS, two products, with 64 KB
// of rows to each of two stages): 526 us at 16384 tokens, 16/4 heads, d = 128, 16
// blocks of 64 keys, of which the products alone would be 180 and the rows' bytes
// out of L2 about 210.
// TMEM: S, dP of stage s at s * 128 + {0, 64}; dV^T at 256, dK^T at 320.
template <int D>
__global__ void __launch_bounds__(kDkvThreads, 1)
    block_dkv_kernel(BlockDims p, int ktiles, int piece, const uint16_t* __restrict__ q,
                     const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, const uint16_t* __restrict__ go,
                     const float* __restrict__ lse, const float* __restrict__ delta,
                     const int32_t* __restrict__ lengths, const int32_t* __restrict__ total,
                     const int32_t* __restrict__ start, const int32_t* __restrict__ list,
                     const int4* __restrict__ items, const int32_t* __restrict__ counts, float scale,
                     float scale_log2, uint16_t* __restrict__ dk, uint16_t* __restrict__ dv,
                     float* __restrict__ parts, int* __restrict__ err) {
  constexpr int kRowBytes = kRowTile * D * 2;
  constexpr int kKvBytes = kKeyTile * D * 2;
  constexpr int kPBytes = kRowTile * kKeyTile * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // no room to round up in: the declared alignment has to hold
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) report_error(err, kErrBadPlan);
    return;
  }
  uint8_t* row_s = smem_raw;             // stage s: dO at s * 2 * kRowBytes, Q behind it
  uint8_t* p_s = row_s + 4 * kRowBytes;  // stage s: P, dS
  uint8_t* k_s = p_s + 4 * kPBytes;
  uint8_t* v_s = k_s + kKvBytes;
  DkvSmem* S = reinterpret_cast<DkvSmem*>(v_s + kKvBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (static_cast<int>(blockIdx.x) >= counts[0]) return;
  if (__syncthreads_or(timed_out_before(err) ? 1 : 0)) return;
  const int4 item = items[blockIdx.x];
  const int bh = item.x / ktiles, kt = item.x - bh * ktiles, key0 = kt * kKeyTile;
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int len = seq_len(p, lengths, b);
  const size_t at = static_cast<size_t>(bh) * p.nb + kt / p.nsub;
  const int32_t* toks = list + static_cast<size_t>(bh) * p.Nq * p.n_sel + start[at];
  const long long all_rows = static_cast<long long>(total[at]) * p.G;
  const long long row0 = static_cast<long long>(item.y) * piece;
  const int rows = static_cast<int>(min(static_cast<long long>(piece), all_rows - row0));
  const int nj = (max(rows, 0) + kRowTile - 1) / kRowTile;

  if (tid == 0) {
    S->abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&S->full[s]), kDkvLoaders);
      mbar_init(smem_u32(&S->free_[s]), 1);
      mbar_init(smem_u32(&S->s_full[s]), 1);
      mbar_init(smem_u32(&S->ds_full[s]), 4);
    }
    mbar_init(smem_u32(&S->mma_final), 1);
#ifdef SVOO_TEST_STALL
    mbar_init(smem_u32(&S->stall), 1);
#endif
    fence_mbar_init();
  }
  if (nj > 0) {
    const size_t krow = static_cast<size_t>(bh) * p.cap + key0;
    load_key_rows<D>(k_s, k, krow, len - key0, tid, kDkvThreads);
    load_key_rows<D>(v_s, v, krow, len - key0, tid, kDkvThreads);
    fence_proxy_async_smem();
  }
  if (warp == kDkvIssuer) {
    __syncwarp();
    tmem_alloc(smem_u32(&S->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  volatile int* abort = &S->abort;
  const uint32_t row_u = smem_u32(row_s), p_u = smem_u32(p_s), k_u = smem_u32(k_s), v_u = smem_u32(v_s);

  if (warp >= 8 && warp < kDkvIssuer) {
    // ---------------------------------------------------------------- row gather
    const int t = tid - 256;  // one row's list entry and scalars per thread
    constexpr int kChunks = D / 8;
    const int ch = t % kChunks, r0 = t / kChunks;
    // Read ahead, so that no load is waited for where it is issued: the list
    // entry of tile j + 2, and the scalars of tile j + 1.
    const unsigned first_row = static_cast<unsigned>(row0), G = p.G;  // 32 bits: 64-bit divisions took 500 cycles a tile
    auto entry = [&](int j) {  // the query of this thread's row in tile j, -1 behind the last
      const int f = j * kRowTile + t;
      return t < kRowTile && f < rows ? toks[(first_row + f) / G] : -1;
    };
    int row = -1, nv = 0;
    float l2 = INFINITY, dl = 0.f;
    auto scalars = [&](int j, int tok) {
      row = -1;
      nv = 0;
      l2 = INFINITY;  // a row that does not take part: P = 2^(s - inf) = 0
      dl = 0.f;
      if (tok >= 0) {
        const int g = (first_row + j * kRowTile + t) % G;
        row = (b * p.H + hk * p.G + g) * p.Nq + tok;
        nv = max(0, min(kKeyTile, query_limit(p, len, tok) - key0));
        if (nv > 0) {
          l2 = lse[row];
          dl = delta[row];
        }
      }
    };
    int tok = -1;
    if (nj > 0) {
      scalars(0, entry(0));
      tok = entry(1);
    }
    for (int j = 0; j < nj; ++j) {
      const int st = j & 1;
      const bool free = j < 2 || mbar_wait(smem_u32(&S->free_[st]), ((j - 2) >> 1) & 1, abort);
      if (t < kRowTile) S->row[t] = row;
      if (!loaders_agree<kDkvLoaders>(free)) break;  // all warps go on or leave together
      const uint32_t g_dst = row_u + st * 2 * kRowBytes, q_dst = g_dst + kRowBytes;
#pragma unroll 8
      for (int r = r0; r < kRowTile; r += kDkvLoaders / kChunks) {
        const int src = S->row[r];
        const uint32_t off = sw128_offset(r, ch * 8, kRowTile);
        const size_t at = static_cast<size_t>(src < 0 ? 0 : src) * D + ch * 8;
        cp_async16_or_zero(g_dst + off, go + at, src >= 0);
        cp_async16_or_zero(q_dst + off, q + at, src >= 0);
      }
      if (t < kRowTile) {
        S->nv[st][t] = static_cast<uint8_t>(nv);
        S->lse2[st][t] = l2 * 1.4426950408889634f;
        S->delta[st][t] = dl;
      }
      scalars(j + 1, tok);
      tok = entry(j + 2);
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&S->full[st]));  // this thread's part of row tile j is in
      loaders_agree<kDkvLoaders>(true);  // S->row is free again
    }
  } else if (warp == kDkvIssuer) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16_f32(kRowTile, kKeyTile, false, false);
      const uint32_t idesc_g = idesc_bf16_f32(128, kKeyTile, true, true);
      // S, dP of tile js and the sums of tile jg, whichever can go first: a tile
      // that has not landed does not hold back the sums that its stage waits for
      int js = 0, jg = 0;
      bool go = true;
#ifdef SVOO_TEST_STALL
      go = nj == 0 || mbar_wait(smem_u32(&S->stall), 0, abort);  // nothing completes it
#endif
      long long since = clock64();
      while (jg < nj && go) {
        bool did = false;
        if (js < nj && js < jg + 2 && mbar_try_wait(smem_u32(&S->full[js & 1]), (js >> 1) & 1)) {
          const int st = js & 1;
          const uint32_t g_u = row_u + st * 2 * kRowBytes, q_u = g_u + kRowBytes;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ro = (kk >> 2) * kRowTile * 128 + (kk & 3) * 32;
            const uint32_t ko = (kk >> 2) * kKeyTile * 128 + (kk & 3) * 32;
            umma_f16(tmem + st * 128, sw128_desc(q_u + ro, 16, 1024), sw128_desc(k_u + ko, 16, 1024), idesc_s,
                     kk > 0 ? 1u : 0u);
            umma_f16(tmem + st * 128 + 64, sw128_desc(g_u + ro, 16, 1024), sw128_desc(v_u + ko, 16, 1024), idesc_s,
                     kk > 0 ? 1u : 0u);
          }
          umma_commit(smem_u32(&S->s_full[st]));
          ++js;
          did = true;
        }
        if (jg < js && mbar_try_wait(smem_u32(&S->ds_full[jg & 1]), (jg >> 1) & 1)) {
          const int st = jg & 1;
          const uint32_t g_u = row_u + st * 2 * kRowBytes;
          const uint32_t a_v = g_u, a_k = D == 128 ? g_u + kRowBytes : g_u;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kRowTile / 16; ++kk) {
            const uint32_t step = kk * 16 * 128;
            const uint64_t bp = sw128_desc(p_u + st * 2 * kPBytes + step, 16, 1024);
            const uint64_t bs = sw128_desc(p_u + st * 2 * kPBytes + kPBytes + step, 16, 1024);
            umma_f16(tmem + 256, sw128_desc(a_v + step, kRowTile * 128, 1024), bp, idesc_g,
                     (jg > 0 || kk > 0) ? 1u : 0u);
            umma_f16(tmem + 320, sw128_desc(a_k + step, kRowTile * 128, 1024), bs, idesc_g,
                     (jg > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(smem_u32(&S->free_[st]));
          ++jg;
          did = true;
        }
        if (did) {
          since = clock64();
        } else if (*abort || clock64() - since > kWaitBudgetCycles) {
          *abort = 1;
          break;
        }
      }
      umma_commit(smem_u32(&S->mma_final));
      mbar_wait_cleanup(smem_u32(&S->mma_final), 0);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- P, dS
    const int st = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + st * 128;
    uint8_t* prow = p_s + st * 2 * kPBytes;
    bool ok = true;
    for (int j = st; j < nj; j += 2) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->s_full[st]), (j >> 1) & 1, abort));
      if (!ok) break;
      tc_fence_after();
      // the row's scalars came with its tile, which S was computed from
      const int nv = S->nv[st][r];
      const float lse2 = S->lse2[st][r], dl = S->delta[st][r];
      const bool whole = __all_sync(0xffffffffu, nv == kKeyTile || nv == 0);
      const uint64_t sc2 = f2pack(scale_log2, scale_log2), nl2 = f2pack(-lse2, -lse2), nd2 = f2pack(-dl, -dl);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s[32], x[32];
        tmem_ld32f(lane_base + h * 32, s);
        tmem_ld32f(lane_base + 64 + h * 32, x);
        tmem_wait_ld_f(s);
        tmem_wait_ld_f(x);
        if (!whole) {  // a row's own limit falls into this tile
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (h * 32 + c >= nv) s[c] = -INFINITY;
        }
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
          uint32_t pp[4], ds[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = c8 * 8 + 2 * c;
            float e0, e1;
            f2unpack(f2fma(f2pack(s[i], s[i + 1]), sc2, nl2), e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            pp[c] = pack_bf16x2(e0, e1);
            f2unpack(f2mul(f2pack(e0, e1), f2add(f2pack(x[i], x[i + 1]), nd2)), e0, e1);
            ds[c] = pack_bf16x2(e0, e1);
          }
          const uint32_t off = sw128_offset(r, h * 32 + c8 * 8, kRowTile);
          *reinterpret_cast<uint4*>(prow + off) = make_uint4(pp[0], pp[1], pp[2], pp[3]);
          *reinterpret_cast<uint4*>(prow + kPBytes + off) = make_uint4(ds[0], ds[1], ds[2], ds[3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->ds_full[st]));
    }
    // ---------------------------------------------------------------- epilogue
    // warps 0-3 write dv, 4-7 dk: thread = one model dimension (TMEM lane)
    // (not free_: this group may be a phase behind it, and a parity tells no more)
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S->mma_final), 0, abort));
    if (ok) {
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 + st * 64;
      const int dim = D == 128 ? r : r - st * 64;  // d = 64: dv in lanes 0-63, dk in lanes 64-127
      const bool mine = D == 128 || (dim >= 0 && dim < 64);
      const float mul = st ? scale : 1.f;
      uint16_t* dst = st ? dk : dv;
      const int nkeys = min(kKeyTile, p.Nk - key0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[32];
        if (nj > 0) {
          tmem_ld32(acc + h * 32, x);
          tmem_wait_ld_regs(x);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0u;
        }
        if (!mine) continue;
        if (item.w >= 0) {
          float* o = parts + (static_cast<size_t>(item.w) * 2 + st) * kKeyTile * D + dim;
#pragma unroll
          for (int c = 0; c < 32; ++c) o[(h * 32 + c) * D] = __uint_as_float(x[c]) * mul;
        } else {
          uint16_t* o = dst + (static_cast<size_t>(bh) * p.Nk + key0) * D + dim;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (h * 32 + c < nkeys)
              o[static_cast<size_t>(h * 32 + c) * D] =
                  static_cast<uint16_t>(pack_bf16x2(__uint_as_float(x[c]) * mul, 0.f) & 0xffffu);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort) report_error(err, kErrTimeoutAttn);
  if (warp == kDkvIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// adds the parts of the key tiles whose list was cut, in order; grid.y eighths of
// a tile's dv and dk
template <int D>
__global__ void __launch_bounds__(256)
    block_dkv_sum_kernel(BlockDims p, int ktiles, const int4* __restrict__ items, const int32_t* __restrict__ counts,
                         const float* __restrict__ parts, uint16_t* __restrict__ dk, uint16_t* __restrict__ dv) {
  if (static_cast<int>(blockIdx.x) >= counts[0]) return;
  const int4 item = items[blockIdx.x];
  if (item.z < 2 || item.y != 0) return;
  const int bh = item.x / ktiles, key0 = (item.x - bh * ktiles) * kKeyTile;
  const int nkeys = min(kKeyTile, p.Nk - key0);
  const float* src = parts + static_cast<size_t>(item.w) * 2 * kKeyTile * D;
  constexpr int kAll = 2 * kKeyTile * D;
  for (int i = (blockIdx.y * 256 + threadIdx.x) * 4; i < kAll; i += 8 * 256 * 4) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < item.z; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(src + static_cast<size_t>(c) * kAll + i);
      a.x += x.x;
      a.y += x.y;
      a.z += x.z;
      a.w += x.w;
    }
    const int which = i / (kKeyTile * D), rest = i - which * kKeyTile * D, key = rest / D;
    if (key < nkeys)
      *reinterpret_cast<uint2*>((which ? dk : dv) + (static_cast<size_t>(bh) * p.Nk + key0) * D + rest) =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

static_assert(dkv_tile_bytes<128>() + sizeof(DkvSmem) <= kMaxSmem, "dk, dv: shared memory of one SM");

// ------------------------------------------------------------------ host side

// Rows of one piece: a quarter of an SM's share of all rows, so that a block
// which every query keeps does not leave one SM with the last word, and at least
// 8 tiles, below which a piece's own start and its part's bytes show. (An eighth
// cut most of the lists of ordinary length too: the parts' sum alone took 78 us
// of 2000 at 16384 tokens.)
inline int piece_rows(const BlockDims& p) {
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.Nq * p.n_sel * p.nsub * p.G;
  long long piece = rows / (148 * 4);
  piece = (piece + kRowTile - 1) / kRowTile * kRowTile;
  if (piece < 8 * kRowTile) piece = 8 * kRowTile;
  return static_cast<int>(piece < (1 << 28) ? piece : (1 << 28));
}

struct GradPlan {
  int ktiles, chunk, nchunk, piece;
  long long max_items, max_slots;
  float *delta, *parts;
  int32_t *hist, *total, *start, *list, *counts;
  int4* items;
  size_t bytes;
};

GradPlan grad_plan(const BlockDims& p, int d, void* ws) {
  GradPlan g;
  const long long BHk = static_cast<long long>(p.B) * p.Hkv;
  const long long rows = BHk * p.Nq * p.n_sel * p.nsub * p.G;  // over all key tiles, at most
  g.ktiles = (p.Nk + kKeyTile - 1) / kKeyTile;
  g.chunk = sel_chunk(p);
  g.nchunk = (p.Nq + g.chunk - 1) / g.chunk;
  g.piece = piece_rows(p);
  g.max_items = BHk * g.ktiles + rows / g.piece;
  g.max_slots = 2 * (rows / g.piece);  // a cut list has more rows than one piece
  Carver c(ws);
  g.delta = c.take<float>(static_cast<size_t>(p.B) * p.H * p.Nq);
  g.hist = c.take<int32_t>(static_cast<size_t>(BHk) * g.nchunk * p.nb);
  g.total = c.take<int32_t>(static_cast<size_t>(BHk) * p.nb);
  g.start = c.take<int32_t>(static_cast<size_t>(BHk) * p.nb);
  g.list = c.take<int32_t>(static_cast<size_t>(BHk) * p.Nq * p.n_sel);
  g.counts = c.take<int32_t>(2);
  g.items = c.take<int4>(static_cast<size_t>(g.max_items));
  g.parts = c.take<float>(static_cast<size_t>(g.max_slots) * 2 * kKeyTile * d);
  g.bytes = (c.used + 255) / 256 * 256;
  return g;
}

template <int D>
svoo_status launch_block_grad(const BlockDims& p, const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* go, const int32_t* idx, const int32_t* lengths,
                              float scale, void* dq, void* dk, void* dv, void* ws, int32_t* dev_err,
                              cudaStream_t st) {
  const GradPlan g = grad_plan(p, D, ws);
  const int BHk = p.B * p.Hkv;
  const uint16_t *qp = static_cast<const uint16_t*>(q), *kp = static_cast<const uint16_t*>(k),
                 *vp = static_cast<const uint16_t*>(v), *gp = static_cast<const uint16_t*>(go);
  const BlockDims t = fit_tile(p, kMaxSmem - dq_smem<D>());  // as row tiles take them
  CUtensorMap qm, gm, om, km, vm;
  const uint64_t krows = mapped_key_rows(p);
  if (p.Nq > 0 && (encode_token_major(&qm, q, t.B, t.H, t.Nq, D, t.G, t.tpt) != CUDA_SUCCESS ||
                   encode_token_major(&gm, go, t.B, t.H, t.Nq, D, t.G, t.tpt) != CUDA_SUCCESS ||
                   encode_token_major(&om, o, t.B, t.H, t.Nq, D, t.G, t.tpt) != CUDA_SUCCESS))
    return SVOO_ERR_CUDA;
  if (encode_tiled_2d(&km, k, krows, D, kKeyTile, 64) != CUDA_SUCCESS ||
      encode_tiled_2d(&vm, v, krows, D, kKeyTile, 64) != CUDA_SUCCESS)
    return SVOO_ERR_CUDA;
  const size_t dkv_smem = dkv_tile_bytes<D>() + sizeof(DkvSmem);
  const size_t cnt_smem = static_cast<size_t>(p.nb) * 4;
  if (!allow_smem(block_dq_kernel<D>, kMaxSmem) || !allow_smem(block_dkv_kernel<D>, dkv_smem) ||
      !allow_smem(sel_walk_kernel<kSelCount>, kMaxBlocks * 4) || !allow_smem(sel_walk_kernel<kSelList>, kMaxBlocks * 4))
    return SVOO_ERR_CUDA;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (p.Nq > 0) {
    sel_walk_kernel<kSelCount><<<dim3(g.nchunk, BHk), 32, cnt_smem, st>>>(p, idx, lengths, g.chunk, g.nchunk, g.hist,
                                                                      nullptr, nullptr, nullptr);
  }
  sel_scan_kernel<<<dim3((p.nb + 31) / 32, BHk), 256, 0, st>>>(p, g.nchunk, g.hist, g.total);
  sel_items_kernel<<<1, 1024, 0, st>>>(p, g.ktiles, g.piece, g.total, g.start, g.items, g.counts);
  if (p.Nq > 0) {
    sel_walk_kernel<kSelList><<<dim3(g.nchunk, BHk), 32, cnt_smem, st>>>(p, idx, lengths, g.chunk, g.nchunk, g.hist,
                                                                     g.start, g.list, nullptr);
    block_dq_kernel<D><<<dim3((t.Nq + t.tpt - 1) / t.tpt, BHk), kDqThreads, dq_smem<D>() + tile_list_bytes(t), st>>>(
        qm, gm, om, km, vm, t, static_cast<int>(union_cap(t)), kp, vp, lse, g.delta, idx, lengths, scale, scale_log2,
        static_cast<uint16_t*>(dq), dev_err);
  }
  block_dkv_kernel<D><<<static_cast<unsigned>(g.max_items), kDkvThreads, dkv_smem, st>>>(
      p, g.ktiles, g.piece, qp, kp, vp, gp, lse, g.delta, lengths, g.total, g.start, g.list, g.items, g.counts, scale,
      scale_log2, static_cast<uint16_t*>(dk), static_cast<uint16_t*>(dv), g.parts, dev_err);
  if (g.max_slots > 0)
    block_dkv_sum_kernel<D><<<dim3(static_cast<unsigned>(g.max_items), 8), 256, 0, st>>>(
        p, g.ktiles, g.items, g.counts, g.parts, static_cast<uint16_t*>(dk), static_cast<uint16_t*>(dv));
  return launch_status();
}

}  // namespace

}  // namespace svoo

using namespace svoo;

extern "C" size_t svoo_block_attn_backward_workspace_size(const svoo_block_shape* shape) {
  if (!block_shape_ok(shape)) return 0;
  return grad_plan(block_dims(shape), shape->d, nullptr).bytes;
}

extern "C" svoo_status svoo_block_attn_backward(const svoo_block_shape* shape, const void* q, const void* k,
                                                const void* v, const void* o, const float* lse, const void* grad_o,
                                                const int32_t* idx, const int32_t* lengths, float scale, void* dq,
                                                void* dk, void* dv, void* workspace, size_t workspace_bytes,
                                                int32_t* dev_err, void* stream) {
  if (!block_shape_ok(shape) || !k || !v || !dk || !dv || !workspace || !scale_ok(scale)) return SVOO_ERR_INVALID_ARG;
  // tensors without queries are empty and have no address; dk and dv are then zeros
  if (shape->Nq > 0 && (!q || !o || !lse || !grad_o || !idx || !dq)) return SVOO_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, o, grad_o, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    if (!aligned(x, 16)) return SVOO_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(idx, 4) || !aligned(lse, 4) || !aligned(lengths, 4) ||
      !aligned(dev_err, 4))
    return SVOO_ERR_INVALID_ARG;
  const BlockDims p = block_dims(shape);
  if (workspace_bytes < grad_plan(p, shape->d, nullptr).bytes) return SVOO_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128)
    return launch_block_grad<128>(p, q, k, v, o, lse, grad_o, idx, lengths, scale, dq, dk, dv, workspace, dev_err, st);
  return launch_block_grad<64>(p, q, k, v, o, lse, grad_o, idx, lengths, scale, dq, dk, dv, workspace, dev_err, st);
}
