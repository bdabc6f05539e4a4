// block_select.cu -- block means of the keys and the blocks that every query
// selects.
//
//   pool[c] = mean of block c's valid keys  (summed in fp64, rounded once)
//   score(t, c) = (sum over the group's heads of q[t, h]) . pool[c]
//
// A query keeps its forced blocks (the first `sink`; when causal the `local`
// up to its own) and fills its n_sel slots with the best of the others; equal
// scores go to the lower block. The choice is that of an fp64 evaluation:
// scores are computed in fp32, and where the last block taken and the first
// one left out lie within twice the error bound of each other, the candidates
// around that border are scored again in fp64.
//
// When causal, only blocks that end before the query's own block are scored,
// and the own block is always kept: a mean never shows a query a key behind it.
#include "blocks.cuh"

namespace svoo {

namespace {

// ------------------------------------------------------------------ pool

// grid (blocks, B * Hkv); 128 threads, each 8 columns of every (1024 / D)-th row
template <int D>
__global__ void __launch_bounds__(128)
    block_pool_kernel(BlockDims p, const uint16_t* __restrict__ k, const int32_t* __restrict__ lengths, int last,
                      float* __restrict__ pool) {
  constexpr int kCols = D / 8, kRows = 128 / kCols;
  __shared__ double part[kRows][D];
  const int bh = blockIdx.y, len = seq_len(p, lengths, bh / p.Hkv);
  int c = blockIdx.x;
  if (last) c = (len + p.block - 1) / p.block - 1 - c;
  if (c < 0) return;
  const int n = max(0, min(p.block, len - c * p.block));
  const int col = (threadIdx.x % kCols) * 8, r0 = threadIdx.x / kCols;
  const uint16_t* src = k + (static_cast<size_t>(bh) * p.cap + static_cast<size_t>(c) * p.block) * D + col;
  double a[8] = {0., 0., 0., 0., 0., 0., 0., 0.};
#pragma unroll 4
  for (int r = r0; r < n; r += kRows) {
    const uint4 x = *reinterpret_cast<const uint4*>(src + static_cast<size_t>(r) * D);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] += static_cast<double>(__uint_as_float(w[i] << 16));
      a[2 * i + 1] += static_cast<double>(__uint_as_float(w[i] & 0xffff0000u));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[r0][col + i] = a[i];
  __syncthreads();
  const int d = threadIdx.x;
  if (d < D) {
    double s = 0.;
#pragma unroll
    for (int r = 0; r < kRows; ++r) s += part[r][d];
    pool[(static_cast<size_t>(bh) * p.nb + c) * D + d] = static_cast<float>(s / (n > 0 ? n : 1));
  }
}

// ------------------------------------------------------------------ select

constexpr int kSelThreads = 256;
constexpr int kAmb = 64;  // border candidates kept with their exact scores

// unsigned keys in the order of the floats
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct SelWarp {
  double val[kAmb];
  int blk[kAmb];
};

// The queries' candidate range: blocks [0, nc), of which [lo, hi) are chosen
// by score and the others forced; nc = 0 for a query outside its sequence.
struct Candidates {
  int nc, lo, hi;
};
__device__ __forceinline__ Candidates candidates(const BlockDims& p, int len, int t) {
  Candidates c;
  if (p.causal) {
    const int pos = query_pos(p, len, t);
    c.nc = pos >= 0 && pos < len ? pos / p.block + 1 : 0;
  } else {
    c.nc = (len + p.block - 1) / p.block;
  }
  c.lo = min(p.sink, c.nc);
  c.hi = max(c.lo, c.nc - p.local);
  return c;
}

// TQ queries of one key head per CTA: fp32 scores of all their candidate
// blocks into shared memory (lane = block, a register per query), then one
// warp per query finds its border.
template <int D, int TQ>
__global__ void __launch_bounds__(kSelThreads)
    block_select_kernel(BlockDims p, int pitch, const uint16_t* __restrict__ q, const float* __restrict__ pool,
                        const int32_t* __restrict__ lengths, int32_t* __restrict__ idx) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelWarp* amb = reinterpret_cast<SelWarp*>(smem_raw);
  float* qs = reinterpret_cast<float*>(amb + kSelThreads / 32);  // [TQ][D]
  float* sc = qs + TQ * D;                                       // [TQ][pitch]
  __shared__ int pool_norm2;                                     // largest |pool[c]|^2 seen, as bits
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y / p.Hkv, hk = blockIdx.y - b * p.Hkv;
  const int len = seq_len(p, lengths, b);
  const int t0 = blockIdx.x * TQ, nt = min(TQ, p.Nq - t0);
  const float* pl = pool + static_cast<size_t>(blockIdx.y) * p.nb * D;
  const uint16_t* qh = q + (static_cast<size_t>(b) * p.H + hk * p.G) * p.Nq * D;  // head 0 of the group
  const size_t head = static_cast<size_t>(p.Nq) * D;
  if (tid == 0) pool_norm2 = 0;
  for (int i = tid; i < TQ * D; i += kSelThreads) {
    const int t = i / D, d = i - t * D;
    float a = 0.f;
    if (t < nt)
      for (int g = 0; g < p.G; ++g) a += bf16_to_f32(qh[g * head + static_cast<size_t>(t0 + t) * D + d]);
    qs[i] = a;
  }
  // the tile's last query inside the sequence has the most candidates
  int most = (len + p.block - 1) / p.block;
  if (p.causal) {
    const int pos = min(query_pos(p, len, t0 + nt - 1), len - 1);
    most = pos >= 0 ? pos / p.block + 1 : 0;
  }
  const int nmax = most - p.local;
  __syncthreads();
  if (most > p.n_sel) {
    float big = 0.f;
    for (int c0 = warp * 32; c0 < nmax; c0 += kSelThreads) {
      const int c = c0 + lane;
      const float4* row = reinterpret_cast<const float4*>(pl + static_cast<size_t>(min(c, nmax - 1)) * D);
      float acc[TQ], n2 = 0.f;
#pragma unroll
      for (int t = 0; t < TQ; ++t) acc[t] = 0.f;
#pragma unroll 2
      for (int d = 0; d < D / 4; ++d) {
        const float4 x = row[d];
        n2 = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, fmaf(x.w, x.w, n2))));
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
          const float4 y = *reinterpret_cast<const float4*>(qs + t * D + d * 4);
          acc[t] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc[t]))));
        }
      }
      big = fmaxf(big, n2);
      if (c < nmax) {
#pragma unroll
        for (int t = 0; t < TQ; ++t) sc[t * pitch + c] = acc[t];
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    if (lane == 0) atomicMax(&pool_norm2, __float_as_int(big));
  }
  __syncthreads();

  for (int t = warp; t < nt; t += kSelThreads / 32) {
    const Candidates cd = candidates(p, len, t0 + t);
    int32_t* out = idx + (static_cast<size_t>(blockIdx.y) * p.Nq + t0 + t) * p.n_sel;
    float* s = sc + t * pitch;
    const int m = p.n_sel - (cd.nc - (cd.hi - cd.lo));  // slots left beside the forced blocks
    const bool all = cd.nc <= p.n_sel;
    float cut = INFINITY;   // scores above it are taken
    bool incl = false;      // ... and those equal to it
    if (!all && m > 0) {
      // m-th largest score: bisection over the ordered keys
      uint32_t lo = 0xffffffffu, hi = 0;
      for (int c = cd.lo + lane; c < cd.hi; c += 32) {
        const uint32_t k = order_key(s[c]);
        lo = min(lo, k);
        hi = max(hi, k);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        int n = 0;
        for (int c = cd.lo + lane; c < cd.hi; c += 32) n += order_key(s[c]) >= mid;
        n = __reduce_add_sync(0xffffffffu, n);
        if (n >= m) lo = mid;
        else hi = mid - 1;
        if (n == m) break;
      }
      // smallest score taken, largest left out, how many are taken
      uint32_t in = 0xffffffffu, outk = 0;
      int n = 0;
      for (int c = cd.lo + lane; c < cd.hi; c += 32) {
        const uint32_t k = order_key(s[c]);
        if (k >= lo) {
          in = min(in, k);
          ++n;
        } else {
          outk = max(outk, k);
        }
      }
      in = __reduce_min_sync(0xffffffffu, in);
      outk = __reduce_max_sync(0xffffffffu, outk);
      n = __reduce_add_sync(0xffffffffu, n);
      const float tau = key_value(in);
      float q2 = 0.f;
      for (int d = lane; d < D; d += 32) q2 = fmaf(qs[t * D + d], qs[t * D + d], q2);
#pragma unroll
      for (int o = 16; o; o >>= 1) q2 += __shfl_xor_sync(0xffffffffu, q2, o);
      // |fp32 score - score| <= (D + G + 2) 2^-24 sum |q_d pool_d| <= (D + G + 2) 2^-24 |q||pool|,
      // and the norms themselves are good to far better than the 1.5 spent on them
      const float e2 = 3.f * (D + p.G + 2) * 5.9604645e-8f * sqrtf(q2) * sqrtf(__int_as_float(pool_norm2));
      if (n == m && tau - key_value(outk) > e2) {
        cut = tau;
        incl = true;
      } else {
        // border: scored again in fp64, the best `need` of them are taken
        cut = tau + e2;
        int sure = 0, na = 0;
        double qd[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          qd[i] = 0.;
          for (int g = 0; g < p.G; ++g)
            qd[i] += static_cast<double>(bf16_to_f32(qh[g * head + static_cast<size_t>(t0 + t) * D + i * 32 + lane]));
        }
        auto exact = [&](int c) {
          double x = 0.;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            x = fma(qd[i], static_cast<double>(pl[static_cast<size_t>(c) * D + i * 32 + lane]), x);
#pragma unroll
          for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          return x;
        };
        for (int c0 = cd.lo; c0 < cd.hi; c0 += 32) {
          const int c = c0 + lane;
          const float x = c < cd.hi ? s[c] : 0.f;
          sure += __popc(__ballot_sync(0xffffffffu, c < cd.hi && x > cut));
          const unsigned near = __ballot_sync(0xffffffffu, c < cd.hi && x <= cut && x >= tau - e2);
          const int at = na + __popc(near & ((1u << lane) - 1u));
          if (((near >> lane) & 1u) && at < kAmb) amb[warp].blk[at] = c;
          na += __popc(near);
        }
        __syncwarp();
        const int need = min(m - sure, na);
        if (na <= kAmb) {
          for (int i = 0; i < na; ++i) {
            const double x = exact(amb[warp].blk[i]);
            if (lane == 0) amb[warp].val[i] = x;
          }
          __syncwarp();
          for (int i = lane; i < na; i += 32) {
            const double x = amb[warp].val[i];
            int rank = 0;
            for (int j = 0; j < na; ++j) {
              const double y = amb[warp].val[j];
              rank += y > x || (y == x && j < i);
            }
            if (rank < need) s[amb[warp].blk[i]] = INFINITY;
          }
          __syncwarp();
        } else {
          // more candidates than the list holds (many equal blocks): one at a time
          for (int pick = 0; pick < need; ++pick) {
            double best = 0.;
            int at = -1;
            for (int c = cd.lo; c < cd.hi; ++c) {
              const float x = s[c];
              if (!(x <= cut && x >= tau - e2)) continue;
              const double y = exact(c);
              if (at < 0 || y > best) {
                best = y;
                at = c;
              }
            }
            __syncwarp();
            if (lane == 0 && at >= 0) s[at] = INFINITY;
            __syncwarp();
          }
        }
      }
    }
    int n = 0;
    for (int c0 = 0; c0 < cd.nc; c0 += 32) {
      const int c = c0 + lane;
      bool take = c < cd.nc && (all || c < cd.lo || c >= cd.hi);
      if (!take && c < cd.hi && m > 0) take = s[c] > cut || (incl && s[c] == cut);
      const unsigned bal = __ballot_sync(0xffffffffu, take);
      const int at = n + __popc(bal & ((1u << lane) - 1u));
      if (take && at < p.n_sel) out[at] = c;
      n += __popc(bal);
    }
    for (int i = min(n, p.n_sel) + lane; i < p.n_sel; i += 32) out[i] = -1;
  }
}

template <int D, int TQ>
svoo_status launch_select(const BlockDims& p, const void* q, const float* pool, const int32_t* lengths, int32_t* idx,
                          cudaStream_t st) {
  const int pitch = (p.nb + 31) / 32 * 32;
  const size_t smem = sizeof(SelWarp) * (kSelThreads / 32) + static_cast<size_t>(TQ) * (D + pitch) * 4;
  if (cudaFuncSetAttribute(block_select_kernel<D, TQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return SVOO_ERR_CUDA;
  block_select_kernel<D, TQ><<<dim3((p.Nq + TQ - 1) / TQ, p.B * p.Hkv), kSelThreads, smem, st>>>(
      p, pitch, static_cast<const uint16_t*>(q), pool, lengths, idx);
  return launch_status();
}

template <int D>
svoo_status launch_select_d(const BlockDims& p, const void* q, const float* pool, const int32_t* lengths, int32_t* idx,
                            cudaStream_t st) {
  // as many queries per CTA as the scores' shared memory allows (32 x 1024
  // blocks are 128 KB), one where there are few
  if (p.Nq < 8 || p.nb > 4096) return launch_select<D, 1>(p, q, pool, lengths, idx, st);
  if (p.nb > 1024) return launch_select<D, 8>(p, q, pool, lengths, idx, st);
  return launch_select<D, 32>(p, q, pool, lengths, idx, st);
}

}  // namespace

}  // namespace svoo

using namespace svoo;

extern "C" svoo_status svoo_block_pool(const svoo_block_shape* shape, const void* k, const int32_t* lengths, int last,
                                       float* pool, void* stream) {
  if (!block_shape_ok(shape) || !k || !pool || last < 0) return SVOO_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(pool, 16) || !aligned(lengths, 4)) return SVOO_ERR_INVALID_ARG;
  const BlockDims p = block_dims(shape);
  const dim3 grid(last > 0 && last < p.nb ? last : p.nb, p.B * p.Hkv);
  const int tail = last > 0 && last < p.nb ? 1 : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128)
    block_pool_kernel<128><<<grid, 128, 0, st>>>(p, static_cast<const uint16_t*>(k), lengths, tail, pool);
  else
    block_pool_kernel<64><<<grid, 128, 0, st>>>(p, static_cast<const uint16_t*>(k), lengths, tail, pool);
  return launch_status();
}

extern "C" svoo_status svoo_block_select(const svoo_block_shape* shape, const void* q, const float* pool,
                                         const int32_t* lengths, int32_t* idx, void* stream) {
  if (!block_shape_ok(shape) || !q || !pool || !idx) return SVOO_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(idx, 4) || !aligned(lengths, 4)) return SVOO_ERR_INVALID_ARG;
  if (shape->Nq == 0) return SVOO_OK;
  const BlockDims p = block_dims(shape);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128) return launch_select_d<128>(p, q, pool, lengths, idx, st);
  return launch_select_d<64>(p, q, pool, lengths, idx, st);
}
