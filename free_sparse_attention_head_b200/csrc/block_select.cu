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
// around that border are scored again in fp64. The bound counts the sum over the
// heads too, whose fp32 additions err by the heads' sizes, not by the sum's:
// (G - 1) 2^-24 |A| |pool| with A_d = sum |q_hd|, and |A|^2 <= G sum q_hd^2.
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

// how many of N values in registers reach x
template <int N>
__device__ __forceinline__ int reach(const float (&s)[N], float x) {
  int n[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < N; ++c) n[c & 3] += s[c] >= x;
  return (n[0] + n[1]) + (n[2] + n[3]);
}

// A search's next probe in [lo, hi): n_lo values reach lo, n_hi reach hi, about
// `want` are to reach the probe. By the counts and by halves in turn.
__device__ __forceinline__ float probe_at(float lo, float hi, int n_lo, int n_hi, int want, int it) {
  float f = 0.5f;
  if (!(it & 1)) f = fminf(fmaxf(__fdividef(n_lo - want - 0.5f, static_cast<float>(n_lo - n_hi)), 0.1f), 0.9f);
  return lo + f * (hi - lo);
}

// A norm for an error bound from its square in fp32, at least 1e-18: squares of
// less than that lose bits there. It is infinite where the square is: the row is
// then decided in fp64 throughout.
__device__ __forceinline__ float bound_norm(float square) { return sqrtf(fmaxf(square, 1e-36f)); }
// (G - 1) |A| of a sum over G heads, from the sum of their squares
__device__ __forceinline__ float heads_error(int G, float h2) { return G > 1 ? (G - 1) * bound_norm(G * h2) : 0.f; }
constexpr float kMostFp32 = 3.402823466e38f;

struct SelWarp {
  double val[kAmb];
  int blk[kAmb];
};

// Scores in fp64, by a warp: eight lanes hold a query's sum over its heads (`q`:
// its row in the first one, `head` elements from one to the next), D / 8 dimensions
// each, four times over, and each of the four scores a block.
template <int D>
__device__ __forceinline__ void query64(const uint16_t* q, int G, size_t head, double (&qd)[D / 8]) {
  const int part = threadIdx.x & 7;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) qd[i] = 0.;
  for (int g = 0; g < G; ++g) {
    const uint4* src = reinterpret_cast<const uint4*>(q + g * head + part * (D / 8));
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint4 x = src[c];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qd[c * 8 + 2 * i] += static_cast<double>(__uint_as_float(w[i] << 16));
        qd[c * 8 + 2 * i + 1] += static_cast<double>(__uint_as_float(w[i] & 0xffff0000u));
      }
    }
  }
}
template <int D>
__device__ __forceinline__ double score64(const double (&qd)[D / 8], const float* pool, int block) {
  const float4* pc = reinterpret_cast<const float4*>(pool + static_cast<size_t>(block) * D + (threadIdx.x & 7) * (D / 8));
  double x = 0.;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const float4 v = pc[c];
    x = fma(qd[4 * c], static_cast<double>(v.x), x);
    x = fma(qd[4 * c + 1], static_cast<double>(v.y), x);
    x = fma(qd[4 * c + 2], static_cast<double>(v.z), x);
    x = fma(qd[4 * c + 3], static_cast<double>(v.w), x);
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// An unsigned key in the order of the values, -0 as 0.
__device__ __forceinline__ unsigned long long order64(double x) {
  const unsigned long long u = x == 0. ? 0ull : __double_as_longlong(x);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ void warp_min_max(unsigned long long& lo, unsigned long long& hi) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

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

// The `need` best of a query's candidates in [lo, hi) whose score lies in [edge, cut],
// marked by an infinite score: by bisection over fp64 scores that every pass computes
// anew, in order and four at a time; equal scores to the lower block. One warp.
template <int D>
__device__ __noinline__ void best_near(const uint16_t* q, int G, size_t head, const float* pl, float* s, int lo, int hi,
                                       float edge, float cut, int need) {
  const int lane = threadIdx.x & 31, part = lane & 7, who = lane >> 3;
  double qd[D / 8];
  query64<D>(q, G, head, qd);
  auto each = [&](auto f) {
    for (int c0 = lo; c0 < hi; c0 += 4) {
      const int c = c0 + who;
      const bool near = c < hi && s[c] <= cut && s[c] >= edge;
      if (!__any_sync(0xffffffffu, near)) continue;
      const unsigned long long k = order64(score64<D>(qd, pl, min(c, hi - 1)));
      f(c, near && part == 0, k);
    }
  };
  unsigned long long kl = ~0ull, kh = 0ull;
  each([&](int, bool near, unsigned long long k) {
    if (near) {
      kl = min(kl, k);
      kh = max(kh, k);
    }
  });
  warp_min_max(kl, kh);
  int over = 0;        // candidates above kl, once kl = kh
  bool all = false;    // exactly `need` of them reach kl
  while (kl < kh && !all) {
    const unsigned long long mid = kl + (kh - kl) / 2 + 1;
    int n = 0;
    each([&](int, bool near, unsigned long long k) { n += near && k >= mid; });
    n = __reduce_add_sync(0xffffffffu, n);
    all = n == need;
    if (n >= need) {
      kl = mid;
    } else {
      kh = mid - 1;
      over = n;
    }
  }
  int equal = 0;
  each([&](int c, bool near, unsigned long long k) {
    const unsigned eq = __ballot_sync(0xffffffffu, near && k == kl);
    const int rank = equal + __popc(eq & ((1u << lane) - 1u));
    if (near && (k > kl || (k == kl && (all || rank < need - over)))) s[c] = INFINITY;
    equal += __popc(eq);
  });
  __syncwarp();
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
  float* hs = qs + TQ * D;                                       // [TQ][D] sums of the heads' squares,
  float* sc = TQ == 1 ? hs + D : hs;                             // [TQ][pitch] which scores overwrite
  __shared__ float2 norm2[TQ];                                   // squared norms: of the sums, of the heads
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
    float a = 0.f, sq = 0.f;
    if (t < nt)
#pragma unroll 8
      for (int g = 0; g < p.G; ++g) {
        const float x = bf16_to_f32(qh[g * head + static_cast<size_t>(t0 + t) * D + d]);
        a += x;
        sq = fmaf(x, x, sq);
      }
    qs[i] = a;
    hs[i] = sq;
  }
  // the tile's last query inside the sequence has the most candidates
  int most = (len + p.block - 1) / p.block;
  if (p.causal) {
    const int pos = min(query_pos(p, len, t0 + nt - 1), len - 1);
    most = pos >= 0 ? pos / p.block + 1 : 0;
  }
  const int nmax = most - p.local;
  auto norms = [&](int t) {  // one warp
    float q2 = 0.f, h2 = 0.f;
    for (int d = lane; d < D; d += 32) {
      q2 = fmaf(qs[t * D + d], qs[t * D + d], q2);
      h2 += hs[t * D + d];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      q2 += __shfl_xor_sync(0xffffffffu, q2, o);
      h2 += __shfl_xor_sync(0xffffffffu, h2, o);
    }
    if (lane == 0) norm2[t] = make_float2(q2, h2);
    __syncwarp();
  };
  __syncthreads();
  if (TQ > 1 && most > p.n_sel) {  // before the scores go where the squares are
    for (int t = warp; t < TQ; t += kSelThreads / 32) norms(t);
    __syncthreads();
  }
  if (most > p.n_sel) {
    float big = 0.f;
    if (TQ == 1) {
      // one query: a warp reads whole rows (128 / D of them at a time, eight
      // loads in flight) and sums across lanes
      constexpr int kLanes = D / 4, kRows = 32 / kLanes;
      const int part = lane % kLanes, sub = lane / kLanes;
      const float4 y = *reinterpret_cast<const float4*>(qs + part * 4);
      for (int c0 = warp * kRows * 8; c0 < nmax; c0 += (kSelThreads / 32) * kRows * 8) {
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = min(c0 + i * kRows + sub, nmax - 1);
          x[i] = *reinterpret_cast<const float4*>(pl + static_cast<size_t>(c) * D + part * 4);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // largest partial norm of each lane; their sum bounds every row's
          big = fmaxf(big, fmaf(x[i].x, x[i].x, fmaf(x[i].y, x[i].y, fmaf(x[i].z, x[i].z, x[i].w * x[i].w))));
          float a = fmaf(x[i].x, y.x, fmaf(x[i].y, y.y, fmaf(x[i].z, y.z, x[i].w * y.w)));
#pragma unroll
          for (int o = kLanes / 2; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
          const int c = c0 + i * kRows + sub;
          if (part == 0 && c < nmax) sc[c] = a;
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) big += __shfl_xor_sync(0xffffffffu, big, o);
    } else
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
      if (TQ == 1) norms(0);
      const float q2 = norm2[t].x, h2 = norm2[t].y;
      // |fp32 score - score| <= 2^-24 ((D + 2) |q| + (G - 1) |A|) |pool|, and the norms themselves
      // are good to far better than the 1.5 spent on them
      float e2 = 3.f * 5.9604645e-8f * ((D + 2) * bound_norm(q2) + heads_error(p.G, h2)) *
                 bound_norm(__int_as_float(pool_norm2));
      if (e2 > kMostFp32) {  // no fp32 score says anything: all of them stand at the border
        e2 = 0.f;
        for (int c = cd.lo + lane; c < cd.hi; c += 32) s[c] = 0.f;
        __syncwarp();
      }
      // the m-th largest score, between `lo`, which n_lo >= m scores reach, and
      // `hi`, which fewer do; up to 32 a lane in registers
      constexpr int kHeld = 32;
      const bool few = cd.hi - cd.lo <= 32 * kHeld;
      float held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int c = cd.lo + i * 32 + lane;
        held[i] = few && c < cd.hi ? s[c] : -INFINITY;
      }
      auto count = [&](float x) {
        int n = 0;
        if (few) {
          if (cd.hi - cd.lo <= 128) {
#pragma unroll
            for (int i = 0; i < 4; ++i) n += held[i] >= x;
          } else {
            n = reach(held, x);
          }
        } else {
          for (int c = cd.lo + lane; c < cd.hi; c += 32) n += s[c] >= x;
        }
        return static_cast<int>(__reduce_add_sync(0xffffffffu, n));
      };
      float lo = INFINITY, hi = -INFINITY;
      for (int c = cd.lo + lane; c < cd.hi; c += 32) {
        lo = fminf(lo, s[c]);
        hi = fmaxf(hi, s[c]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      int n = cd.hi - cd.lo, n_hi = 1;
      for (int it = 0; it < 48 && n != m; ++it) {
        const float mid = probe_at(lo, hi, n, n_hi, m, it);
        if (mid <= lo || mid >= hi || hi - lo < e2) break;
        const int k = count(mid);
        if (k >= m) {
          lo = mid;
          n = k;
        } else {
          hi = mid;
          n_hi = k;
        }
      }
      // smallest score taken, largest left out
      float in = INFINITY, out_s = -INFINITY;
      for (int c = cd.lo + lane; c < cd.hi; c += 32) {
        if (s[c] >= lo) in = fminf(in, s[c]);
        else out_s = fmaxf(out_s, s[c]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        in = fminf(in, __shfl_xor_sync(0xffffffffu, in, o));
        out_s = fmaxf(out_s, __shfl_xor_sync(0xffffffffu, out_s, o));
      }
      if (n == m && in - out_s > e2) {
        cut = in;
        incl = true;
      } else {
        // border: scored again in fp64, the best `need` of them are taken
        if (n == m) lo = hi = in;
        const float edge = lo - e2;
        cut = hi + e2;
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
          const unsigned near = __ballot_sync(0xffffffffu, c < cd.hi && x <= cut && x >= edge);
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
          // more candidates than the list holds (many equal blocks)
          best_near<D>(qh + static_cast<size_t>(t0 + t) * D, p.G, head, pl, s, cd.lo, cd.hi, edge, cut, need);
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

// ------------------------------------------------------------------ select, many queries
//
// 128 queries of one key head per CTA, their scores from the tensor cores: the
// queries' group sums and the means are split into two bf16 parts each (hi, lo;
// what is left is below 2^-16 of the value), and hi.hi + hi.lo + lo.hi
// accumulate in fp32. With u = 2^-16 a part product's neglected rest is at most
// 3 u sum |q_d pool_d|, the 3 D additions at most 3 D 2^-23 of the same sum, and
// the sum at most |q||pool|: with the sum over the heads (above) that is the error
// bound of the border test.
//
// A thread owns a query (= TMEM lane) and streams its scores, 64 blocks a step,
// through a list of at most kList candidates: a score enters when it is not
// below the running cut; when a step's would not fit, the cut rises to just
// below the m-th best so far (minus the border) and the list is packed. Scores
// never leave the SM. Two CTAs share an SM, so one streams while the other loads.
// (A first pass over the products for the cut alone, from the maxima of groups of
// blocks, was no faster: 520 against 502 us at 65536 queries of 1024 blocks.)
// Warps 0-3 stream, 4 loads the means (TMA), 5 issues the products.
// TMEM: A hi [0, 64), A lo [64, 128), scores [128, 192) and [192, 256).

constexpr int kMmaSelThreads = 192;
constexpr int kList = 64;         // candidates of a query
constexpr int kMaxChosen = 48;    // blocks chosen by score: leaves room for six more and ten ties
constexpr int kMmaMaxBlocks = 6144;  // exact scores of a whole row fit where the lists were

struct MmaSelSmem {
  uint64_t full[2], empty[2], s_full[2], s_empty[2], mma_final;
#ifdef SVOO_TEST_STALL
  uint64_t stall;  // test-only: a barrier that nothing completes
#endif
  uint32_t tmem_base;
  int abort;
  int hard;             // queries whose ties overran the list, or whose norms are out of fp32's range
  float pool_norm2;
};

template <int D>
__host__ __device__ constexpr size_t sel_stage_bytes() {
  return 2 * static_cast<size_t>(kKeyTile) * D * 2;  // 64 blocks, hi and lo
}
template <int D>
__host__ __device__ constexpr size_t sel_area_bytes() {  // the stages; at other times the group sums, and the selected ids
  const size_t st = 2 * sel_stage_bytes<D>(), ids = 128 * static_cast<size_t>(64) * 4;
  return st > ids ? st : ids;
}
template <int D>
constexpr size_t mma_sel_smem() {
  return sel_area_bytes<D>() + static_cast<size_t>(kList + 1) * 128 * 6 + sizeof(MmaSelSmem);
}
static_assert(2 * (mma_sel_smem<128>() + 1024) <= 233472, "two CTAs on an SM");

// fp32 means as bf16 hi and lo parts, 64 blocks per CTA (zeros behind the last
// block), and the largest squared norm among them
template <int D>
__global__ void __launch_bounds__(256)
    pool_split_kernel(int nb, int nbp, size_t lo_at, const float* __restrict__ pool, uint16_t* __restrict__ parts,
                      float* __restrict__ norms) {
  constexpr int kT = D / 4;  // threads per row
  const int c0 = blockIdx.x * 64, bh = blockIdx.y;
  __shared__ float best[8];
  float big = 0.f;
  for (int i = threadIdx.x; i < 64 * kT; i += 256) {
    const int c = c0 + i / kT, d = (i % kT) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < nb) x = *reinterpret_cast<const float4*>(pool + (static_cast<size_t>(bh) * nb + c) * D + d);
    const uint32_t h0 = pack_bf16x2(x.x, x.y), h1 = pack_bf16x2(x.z, x.w);
    const uint32_t l0 = pack_bf16x2(x.x - __uint_as_float(h0 << 16), x.y - __uint_as_float(h0 & 0xffff0000u));
    const uint32_t l1 = pack_bf16x2(x.z - __uint_as_float(h1 << 16), x.w - __uint_as_float(h1 & 0xffff0000u));
    uint16_t* dst = parts + (static_cast<size_t>(bh) * nbp + c) * D + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(h0, h1);
    *reinterpret_cast<uint2*>(dst + lo_at) = make_uint2(l0, l1);
    float n2 = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
#pragma unroll
    for (int o = kT / 2 < 16 ? kT / 2 : 16; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
    big = fmaxf(big, n2);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = big;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) big = fmaxf(big, best[w]);
    norms[static_cast<size_t>(bh) * gridDim.x + blockIdx.x] = big;
  }
}

template <int N>
struct Width {
  static constexpr int value = N;
};

__device__ __forceinline__ int warp_max(int x) { return __reduce_max_sync(0xffffffffu, x); }

// The rows of the four list warps with `hard` set (thread = row), each by its warp and
// one at a time: every free candidate in fp64, four at a time, where the lists were
// (as many warps at once as rows of scores fit there), the m-th best by bisection.
// Keys or queries of all zeros bring every row here (16384 queries of 256 blocks, 16/4
// heads, d = 128: 1.55 ms against 0.11; one row of a CTA at a time, its sum over the
// heads made anew for every block, took 48). A function of its own: inside the kernel
// its code cost other calls time (13.4 against 13.2 us at 1024 queries of 16 blocks).
template <int D>
__device__ __noinline__ void rows_in_fp64(const uint16_t* q, int G, size_t head, const float* pl, int nb, int n_sel,
                                          bool hard, Candidates cd, int m, float* lists, int32_t* ids) {
  constexpr int kDims = D / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 7, who = lane >> 3;
  const int room = (kList + 1) * 128 * 6 / (nb * 8), at_once = room >= 4 ? 4 : room >= 2 ? 2 : 1;
  for (int w = 0; w < 4; w += at_once) {
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (warp < w || warp >= w + at_once) continue;
    double* ex = reinterpret_cast<double*>(lists) + static_cast<size_t>(warp - w) * nb;
    unsigned todo = __ballot_sync(0xffffffffu, hard);
    while (todo) {
      const int src = __ffs(todo) - 1, r = (warp << 5) + src;
      todo &= todo - 1;
      const int lo_c = __shfl_sync(0xffffffffu, cd.lo, src), hi_c = __shfl_sync(0xffffffffu, cd.hi, src);
      const int nc = __shfl_sync(0xffffffffu, cd.nc, src), mr = __shfl_sync(0xffffffffu, m, src);
      unsigned long long lo = ~0ull, hi = 0ull;
      double qd[kDims];
      query64<D>(q + static_cast<size_t>(r) * D, G, head, qd);
#pragma unroll 2
      for (int c0 = lo_c; c0 < hi_c; c0 += 4) {
        const double x = score64<D>(qd, pl, min(c0 + who, hi_c - 1));
        if (part == 0 && c0 + who < hi_c) ex[c0 + who] = x;
      }
      __syncwarp();
      for (int c = lo_c + lane; c < hi_c; c += 32) {
        lo = min(lo, order64(ex[c]));
        hi = max(hi, order64(ex[c]));
      }
      warp_min_max(lo, hi);
      while (lo < hi) {
        const unsigned long long mid = lo + (hi - lo) / 2 + 1;
        int k = 0;
        for (int c = lo_c + lane; c < hi_c; c += 32) k += order64(ex[c]) >= mid;
        k = __reduce_add_sync(0xffffffffu, k);
        if (k >= mr) lo = mid;
        else hi = mid - 1;
      }
      int over = 0;
      for (int c = lo_c + lane; c < hi_c; c += 32) over += order64(ex[c]) > lo;
      over = __reduce_add_sync(0xffffffffu, over);
      int equal = 0, at = 0;
      for (int c0 = 0; c0 < nc; c0 += 32) {
        const int c = c0 + lane;
        const bool forced = c < nc && (c < lo_c || c >= hi_c), open = c < nc && !forced;
        const unsigned eq = __ballot_sync(0xffffffffu, open && order64(ex[c]) == lo);
        const bool take = forced || (open && (order64(ex[c]) > lo || (((eq >> lane) & 1u) &&
                                                                  equal + __popc(eq & ((1u << lane) - 1u)) < mr - over)));
        equal += __popc(eq);
        const unsigned bal = __ballot_sync(0xffffffffu, take);
        const int to = at + __popc(bal & ((1u << lane) - 1u));
        if (take && to < n_sel) ids[r * n_sel + to] = c;
        at += __popc(bal);
      }
      __syncwarp();
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kMmaSelThreads, 2)
    mma_select_kernel(const __grid_constant__ CUtensorMap pmap, BlockDims p, int nbp, const uint16_t* __restrict__ q,
                      const float* __restrict__ pool, const float* __restrict__ norms,
                      const int32_t* __restrict__ lengths, int32_t* __restrict__ idx, int* __restrict__ err) {
  constexpr int kSub = D / 64;
  constexpr int kTile = kKeyTile * D * 2;     // one part of a stage
  constexpr int kHalf = kRowTile * D * 2;     // group sums, one part
  extern __shared__ __align__(1024) uint8_t sel_smem[];
  uint8_t* stage = sel_smem;
  float* lv = reinterpret_cast<float*>(sel_smem + sel_area_bytes<D>());  // [kList + 1][128], the last is scrap
  uint16_t* li = reinterpret_cast<uint16_t*>(lv + (kList + 1) * 128);
  MmaSelSmem* S = reinterpret_cast<MmaSelSmem*>(li + (kList + 1) * 128);
  int32_t* ids = reinterpret_cast<int32_t*>(sel_smem);  // [128][n_sel], once the products are done

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sel_smem) & 1023u) {  // the declared alignment has to hold
    if (tid == 0) report_error(err, kErrBadPlan);
    return;
  }
  if (__syncthreads_or(timed_out_before(err) ? 1 : 0)) return;
  const int b = blockIdx.y / p.Hkv, hk = blockIdx.y - b * p.Hkv;
  const int len = seq_len(p, lengths, b);
  const int t0 = blockIdx.x * kRowTile, nt = min(kRowTile, p.Nq - t0);
  const uint16_t* qh = q + (static_cast<size_t>(b) * p.H + hk * p.G) * p.Nq * D;
  const size_t head = static_cast<size_t>(p.Nq) * D;
  int most = (len + p.block - 1) / p.block;
  if (p.causal) {
    const int pos = min(query_pos(p, len, t0 + nt - 1), len - 1);
    most = pos >= 0 ? pos / p.block + 1 : 0;
  }
  const int steps = most > p.n_sel ? (most - p.local + kKeyTile - 1) / kKeyTile : 0;

  if (tid == 0) {
    S->abort = 0;
    S->hard = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), 1);
      mbar_init(smem_u32(&S->s_full[s]), 1);
      mbar_init(smem_u32(&S->s_empty[s]), 4);
    }
    mbar_init(smem_u32(&S->mma_final), 1);
#ifdef SVOO_TEST_STALL
    mbar_init(smem_u32(&S->stall), 1);
#endif
    fence_mbar_init();
  }
  // one step of at most 64 blocks: the means' parts are made here, without a
  // kernel of their own before this one (2.3 us and its launch)
  const bool own = norms == nullptr;
  if (warp == 4) {
    float big = 0.f;
    for (int i = lane; !own && i < nbp / 64; i += 32)
      big = fmaxf(big, norms[static_cast<size_t>(blockIdx.y) * (nbp / 64) + i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    if (lane == 0) S->pool_norm2 = big;
  }
  if (warp == 5) {
    __syncwarp();
    tmem_alloc(smem_u32(&S->tmem_base), 256);
    tmem_relinquish();
  }
  // the heads' squares, summed over 8 columns each, where the lists begin later
  constexpr int kChunks = D / 8;
  float* squares = lv;  // [128][kChunks]
  if (steps > 0) {
    // group sums: coalesced loads (four rows at a time in flight), fp32 sums,
    // bf16 parts to shared memory
    constexpr int kStep = kMmaSelThreads / kChunks;
    static_assert(kMmaSelThreads % kChunks == 0, "a thread keeps its columns");
    const int ch = tid % kChunks;
    for (int r0 = tid / kChunks; r0 < kRowTile; r0 += 4 * kStep) {
      uint64_t a[4][4], sq[4] = {0ull, 0ull, 0ull, 0ull};  // pairs of columns: their sums, and their squares'
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) a[k][i] = 0ull;
#pragma unroll 2
      for (int g = 0; g < p.G; ++g) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = r0 + k * kStep;
          x[k] = r < nt ? *reinterpret_cast<const uint4*>(qh + g * head + static_cast<size_t>(t0 + r) * D + ch * 8)
                        : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t y = f2pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            a[k][i] = f2add(a[k][i], y);
            sq[k] = f2fma(y, y, sq[k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k * kStep;
        if (r >= kRowTile) break;
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          f2unpack(a[k][i], x, y);
          h[i] = pack_bf16x2(x, y);
          l[i] = pack_bf16x2(x - __uint_as_float(h[i] << 16), y - __uint_as_float(h[i] & 0xffff0000u));
        }
        float x, y;
        f2unpack(sq[k], x, y);
        squares[r * kChunks + ch] = x + y;
        const uint32_t off = r * D * 2 + ((ch ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(stage + off) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(stage + kHalf + off) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  volatile int* abort = &S->abort;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  constexpr int kMean = D / 4, kMeans = (64 * kMean + kMmaSelThreads - 1) / kMmaSelThreads;  // 16-byte pieces
  auto mean_at = [&](int i) {
    const int at = i * kMmaSelThreads + tid;
    return at / kMean < min(p.nb, 64)
               ? *reinterpret_cast<const float4*>(pool + static_cast<size_t>(blockIdx.y) * p.nb * D + at * 4)
               : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  constexpr bool kAhead = D == 64;  // at d = 128 there are no registers for it
  float4 mean[kAhead ? kMeans : 1];
  if (kAhead && own && steps > 0) {
#pragma unroll
    for (int i = 0; i < kMeans; ++i) mean[kAhead ? i : 0] = mean_at(i);
  }
  float q2 = 0.f, h2 = 0.f;
  if (steps > 0 && warp < 4) {
    // this query's parts into tensor memory, and its norms
#pragma unroll
    for (int i = 0; i < kChunks; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(squares + tid * kChunks + i);
      h2 += (x.x + x.y) + (x.z + x.w);
    }
#pragma unroll
    for (int c4 = 0; c4 < D / 32; ++c4) {
      uint32_t h[16], l[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = tid * D * 2 + (((c4 * 4 + i) ^ (tid & 7)) << 4);
        const uint4 x = *reinterpret_cast<const uint4*>(stage + off);
        const uint4 y = *reinterpret_cast<const uint4*>(stage + kHalf + off);
        h[4 * i] = x.x, h[4 * i + 1] = x.y, h[4 * i + 2] = x.z, h[4 * i + 3] = x.w;
        l[4 * i] = y.x, l[4 * i + 1] = y.y, l[4 * i + 2] = y.z, l[4 * i + 3] = y.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = __uint_as_float(h[i] << 16) + __uint_as_float(l[i] << 16);
        const float y = __uint_as_float(h[i] & 0xffff0000u) + __uint_as_float(l[i] & 0xffff0000u);
        q2 = fmaf(x, x, fmaf(y, y, q2));
      }
      tmem_st16(lane_base + c4 * 16, h);
      tmem_st16(lane_base + 64 + c4 * 16, l);
    }
    tmem_wait_st();
  }
  fence_proxy_async_smem();  // the staging area goes to the TMA
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (own && steps > 0) {
    float big = 0.f;
#pragma unroll(kAhead ? kMeans : 4)
    for (int i = 0; i < kMeans; ++i) {
      const int at = i * kMmaSelThreads + tid, c = at / kMean, d = at % kMean * 4;
      if (c >= 64) break;  // a warp's pieces end together
      const float4 x = kAhead ? mean[kAhead ? i : 0] : mean_at(i);
      const uint32_t h0 = pack_bf16x2(x.x, x.y), h1 = pack_bf16x2(x.z, x.w);
      const uint32_t l0 = pack_bf16x2(x.x - __uint_as_float(h0 << 16), x.y - __uint_as_float(h0 & 0xffff0000u));
      const uint32_t l1 = pack_bf16x2(x.z - __uint_as_float(h1 << 16), x.w - __uint_as_float(h1 & 0xffff0000u));
      uint8_t* dst = stage + sw128_offset(c, d & ~7, kKeyTile) + (d & 4) * 2;
      *reinterpret_cast<uint2*>(dst) = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>(dst + kTile) = make_uint2(l0, l1);
      float n2 = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
#pragma unroll
      for (int o = kMean / 2; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      big = fmaxf(big, n2);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    if (lane == 0) atomicMax(reinterpret_cast<int*>(&S->pool_norm2), __float_as_int(big));  // 0 and above
    fence_proxy_async_smem();
    __syncthreads();
  }
  int armed = -1;

  const Candidates cd = warp < 4 && tid < nt ? candidates(p, len, t0 + tid) : Candidates{0, 0, 0};
  const bool all = cd.nc <= p.n_sel;                  // no choice to make
  const int m = p.n_sel - (cd.nc - (cd.hi - cd.lo));  // to be chosen by score
  // twice the error bound, with a tenth more for the fp32 norms and this product
  const float e2 = 2.2f * ((3.f * 1.52587890625e-5f + 3.f * D * 1.1920929e-7f) * bound_norm(q2) +
                           5.9604645e-8f * heads_error(p.G, h2)) * bound_norm(S->pool_norm2);
  int cnt = 0;
  bool hard = !all && m > 0 && e2 > kMostFp32;  // decided in fp64: no fp32 score says anything
  float* mv = lv + (tid & 127);
  uint16_t* mi = li + (tid & 127);

  if (warp == 4) {
    if (own) {
      if (lane == 0 && steps > 0) mbar_arrive(smem_u32(&S->full[0]));
    } else if (lane == 0 && steps > 0) {
      tma_prefetch_desc(&pmap);
      const int row0 = blockIdx.y * nbp, lo_row = p.B * p.Hkv * nbp;
      for (int j = 0; j < steps; ++j) {
        const int st = j & 1, c0 = j * kKeyTile;
        if (j >= 2 && !mbar_wait(smem_u32(&S->empty[st]), ((j - 2) >> 1) & 1, abort)) break;
        const uint32_t bar = smem_u32(&S->full[st]), dst = smem_u32(stage) + st * 2 * kTile;
        mbar_arrive_expect_tx(bar, 2 * kTile);
        for (int s = 0; s < kSub; ++s) {
          tma_load_2d(&pmap, dst + s * kKeyTile * 128, bar, s * 64, row0 + c0);
          tma_load_2d(&pmap, dst + kTile + s * kKeyTile * 128, bar, s * 64, lo_row + row0 + c0);
        }
        armed = j;
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kRowTile, kKeyTile, false, false);
      bool go = true;
#ifdef SVOO_TEST_STALL
      go = steps == 0 || mbar_wait(smem_u32(&S->stall), 0, abort);  // nothing completes it
#endif
      for (int j = 0; j < steps && go; ++j) {
        const int st = j & 1;
        if (!mbar_wait(smem_u32(&S->full[st]), (j >> 1) & 1, abort)) break;
        if (j >= 2 && !mbar_wait(smem_u32(&S->s_empty[st]), ((j - 2) >> 1) & 1, abort)) break;
        tc_fence_after();
        const uint32_t u = smem_u32(stage) + st * 2 * kTile, d = tmem + 128 + st * 64;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kKeyTile * 128 + (kk & 3) * 32;
          const uint64_t bh = sw128_desc(u + off, 16, 1024), bl = sw128_desc(u + kTile + off, 16, 1024);
          umma_f16_a_tmem(d, tmem + kk * 8, bh, idesc, kk > 0 ? 1u : 0u);
          umma_f16_a_tmem(d, tmem + kk * 8, bl, idesc, 1u);
          umma_f16_a_tmem(d, tmem + 64 + kk * 8, bh, idesc, 1u);
        }
        umma_commit(smem_u32(&S->s_full[st]));
        umma_commit(smem_u32(&S->empty[st]));
      }
      umma_commit(smem_u32(&S->mma_final));
      mbar_wait_cleanup(smem_u32(&S->mma_final), 0);
    }
  } else {
    const bool list = !all && m > 0 && !hard;
    const int lo_c = list ? cd.lo : 0, hi_c = list ? cd.hi : 0;
    float cut = -kMostFp32;  // nothing below it can be among the m best
    float s[kKeyTile];
    // Raises the cut to just below a value that m to m + 6 of the list's entries
    // and this step's scores reach, and packs the list.
    auto raise = [&]() {
      const int nmax = (warp_max(cnt) + 7) & ~7;
      float lo = INFINITY, hi = -INFINITY;
#pragma unroll
      for (int c = 0; c < kKeyTile; ++c) {
        if (s[c] >= cut) lo = fminf(lo, s[c]);
        hi = fmaxf(hi, s[c]);
      }
#pragma unroll 8
      for (int i = 0; i < nmax; ++i) {
        const float x = mv[i * 128];
        if (i < cnt && x >= cut) {
          lo = fminf(lo, x);
          hi = fmaxf(hi, x);
        }
      }
      auto both = [&](float x) {
        int n[4] = {reach(s, x), 0, 0, 0};
#pragma unroll 8
        for (int i = 0; i < nmax; ++i) n[i & 3] += i < cnt && mv[i * 128] >= x;
        return (n[0] + n[1]) + (n[2] + n[3]);
      };
      int n_lo = both(lo), n_hi = 1;
      const bool some = n_lo > m;
      bool go = n_lo > m + 6;
      for (int it = 0; it < 32 && __any_sync(0xffffffffu, go); ++it) {
        const float mid = probe_at(lo, hi, n_lo, n_hi, m + 3, it);
        const int n = both(mid);
        if (go) {
          if (mid <= lo || mid >= hi || hi - lo < e2) go = false;
          else if (n >= m) {
            lo = mid;
            n_lo = n;
            go = n > m + 6;
          } else {
            hi = mid;
            n_hi = n;
          }
        }
      }
      if (some) cut = fmaxf(cut, lo - e2);
      int w = 0;
      for (int i0 = 0; i0 < nmax; i0 += 8) {
        float x[8];
        uint16_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = mv[(i0 + i) * 128];
          c[i] = mi[(i0 + i) * 128];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // w <= i0 + i: nothing unread is written over
          mv[w * 128] = x[i];
          mi[w * 128] = c[i];
          w += i0 + i < cnt && x[i] >= cut;
        }
      }
      cnt = w;
    };
    // the next 64 scores into registers; what is not to be chosen at -inf
    auto next = [&](int j, int c0) {
      const int st = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&S->s_full[st]), (j >> 1) & 1, abort))) return false;
      tc_fence_after();
      tmem_ld32f(lane_base + 128 + st * 64, s);
      tmem_ld32f(lane_base + 128 + st * 64 + 32, s + 32);
      tmem_wait_ld_f(s);
      tmem_wait_ld_f(s + 32);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&S->s_empty[st]));
      if (!__all_sync(0xffffffffu, lo_c <= c0 && hi_c >= c0 + kKeyTile)) {
#pragma unroll
        for (int c = 0; c < kKeyTile; ++c)
          if (c0 + c < lo_c || c0 + c >= hi_c) s[c] = -INFINITY;
      }
      return true;
    };
    for (int j = 0; j < steps && next(j, j * kKeyTile); ++j) {
      // the first step's cut from its own scores alone: most of them need not be listed
      if ((j == 0 && steps > 1) || __any_sync(0xffffffffu, cnt + reach(s, cut) > kList)) {
        raise();
        if (cnt + reach(s, cut) > kList) {  // more ties than the list holds
          hard = true;
          cnt = 0;
          cut = INFINITY;
        }
      }
#pragma unroll
      for (int g = 0; g < kKeyTile / 8; ++g) {
        float top = fmaxf(s[g * 8], s[g * 8 + 1]);
#pragma unroll
        for (int c = 2; c < 8; c += 2) top = fmax3(top, s[g * 8 + c], s[g * 8 + c + 1]);
        if (!__any_sync(0xffffffffu, top >= cut)) continue;
#pragma unroll
        for (int c = g * 8; c < g * 8 + 8; ++c) {  // written in any case, kept when the count moves
          mv[cnt * 128] = s[c];
          mi[cnt * 128] = static_cast<uint16_t>(j * kKeyTile + c);
          cnt += s[c] >= cut;
        }
      }
    }
  }
  __syncthreads();
  constexpr int kDims = D / 8;
  const int part = lane & 7, who = lane >> 3;
  const float* pl = pool + static_cast<size_t>(blockIdx.y) * p.nb * D;
  if (*abort) {
    if (tid == 0) report_error(err, kErrTimeoutAttn);
    if (warp == 4 && lane == 0)
      for (int j = max(0, armed - 1); j <= armed; ++j) mbar_wait_cleanup(smem_u32(&S->full[j & 1]), (j >> 1) & 1);
  } else if (warp < 4) {
    // m-th best of the list, and whether the border is clear
    const bool pick = !all && m > 0 && !hard && cnt > m;
    float above = -INFINITY;           // scores from here on are taken
    float edge_lo = 0.f, edge_hi = 0.f;  // of an unclear border
    bool unclear = false;
    auto border = [&](auto width) {
      constexpr int N = decltype(width)::value;
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = pick && i < cnt ? mv[i * 128] : -INFINITY;
      float lo = INFINITY, hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i < cnt) lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
      }
      // the m-th best lies in [lo, hi]: n_lo >= m values reach lo, fewer reach
      // hi, unless all the best are equal to it
      bool go = pick;
      int n_lo = cnt, n_hi = 1;
      for (int it = 0; it < 40 && __any_sync(0xffffffffu, go); ++it) {
        const float mid = probe_at(lo, hi, n_lo, n_hi, m, it);
        const int n = reach(x, mid);
        if (go) {
          if (mid <= lo || mid >= hi || hi - lo < e2) go = false;  // as near as the border test asks for
          else if (n >= m) {
            lo = mid;
            n_lo = n;
            go = n != m;
          } else {
            hi = mid;
            n_hi = n;
          }
        }
      }
      float in = INFINITY, out = -INFINITY;  // smallest taken, largest left out
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (x[i] >= lo) in = fminf(in, x[i]);
        else out = fmaxf(out, x[i]);
      }
      if (pick) {
        above = in;
        unclear = !(n_lo == m && in - out > e2);
        if (n_lo == m) lo = hi = in;
        edge_lo = lo - e2;
        edge_hi = hi + e2;
      }
    };
    const int longest = warp_max(pick ? cnt : 0);
    if (longest > 32) border(Width<kList>());
    else if (longest > 0) border(Width<32>());
    unsigned todo = __ballot_sync(0xffffffffu, unclear);
    while (todo) {
      // one unclear query at a time, the whole warp: its border in fp64
      const int src = __ffs(todo) - 1, r = (warp << 5) + src;
      todo &= todo - 1;
      const float el = __shfl_sync(0xffffffffu, edge_lo, src), eh = __shfl_sync(0xffffffffu, edge_hi, src);
      const int nr = __shfl_sync(0xffffffffu, cnt, src), mr = __shfl_sync(0xffffffffu, m, src);
      double qd[kDims];
      query64<D>(qh + static_cast<size_t>(t0 + r) * D, p.G, head, qd);
      int sure = 0;
      double ex[2] = {0., 0.};
      bool near[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = h * 32 + lane;
        const float x = i < nr ? lv[i * 128 + r] : -INFINITY;
        sure += __popc(__ballot_sync(0xffffffffu, x > eh));
        near[h] = i < nr && x <= eh && x >= el;
        unsigned bal = __ballot_sync(0xffffffffu, near[h]);
        while (bal) {
          // the next four candidates, one for every eight lanes
          int at[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            at[k] = bal ? __ffs(bal) - 1 : -1;
            bal &= bal - 1;
          }
          const int mine = at[who] < 0 ? at[0] : at[who];
          const double x64 = score64<D>(qd, pl, li[(h * 32 + mine) * 128 + r]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const double y = __shfl_sync(0xffffffffu, x64, k * 8);
            if (lane == at[k]) ex[h] = y;
          }
        }
      }
      const int need = mr - sure;
      int rank[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned bal = __ballot_sync(0xffffffffu, near[h]);
        while (bal) {
          const int at = __ffs(bal) - 1;
          bal &= bal - 1;
          const double y = __shfl_sync(0xffffffffu, ex[h], at);
#pragma unroll
          for (int k = 0; k < 2; ++k) rank[k] += y > ex[k] || (y == ex[k] && h * 32 + at < k * 32 + lane);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (near[h]) lv[(h * 32 + lane) * 128 + r] = rank[h] < need ? INFINITY : -INFINITY;
      if (lane == src) above = nextafterf(eh, INFINITY);  // INF marks the near ones that are taken
      __syncwarp();
    }
    if (tid < nt) {
      int32_t* row = ids + tid * p.n_sel;
      int w = 0;
      if (all) {
        for (; w < cd.nc; ++w) row[w] = w;
      } else if (!hard) {
        for (; w < cd.lo; ++w) row[w] = w;
        if (m > 0)
          for (int i0 = 0; i0 < cnt; i0 += 8) {
            float x[8];
            uint16_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] = mv[(i0 + i) * 128];
              c[i] = mi[(i0 + i) * 128];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i0 + i < cnt && x[i] >= above && w < p.n_sel) row[w++] = c[i];
          }
        for (int c = cd.hi; c < cd.nc && w < p.n_sel; ++c) row[w++] = c;
      }
      for (; w < p.n_sel; ++w) row[w] = -1;
    }
    if (hard) atomicAdd(&S->hard, 1);
  }
  __syncthreads();
  const bool fine = !*abort;
  if (fine && S->hard && warp < 4) {
    rows_in_fp64<D>(qh + static_cast<size_t>(t0) * D, p.G, head, pl, p.nb, p.n_sel, hard, cd, m, lv, ids);
  }
  __syncthreads();
  if (fine) {
    int32_t* out = idx + (static_cast<size_t>(blockIdx.y) * p.Nq + t0) * p.n_sel;
    for (int i = tid; i < nt * p.n_sel; i += kMmaSelThreads) out[i] = ids[i];
  }
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// The tensor-core kernel from 64 queries on, while its lists and ids fit; below
// that its 128-query tile would be mostly empty.
inline bool mma_select(const BlockDims& p) {
  return p.Nq >= 64 && p.n_sel <= 64 && p.n_sel - p.sink - p.local <= kMaxChosen && p.nb <= kMmaMaxBlocks;
}

struct SelectPlan {
  int nbp;
  bool split;  // the means' parts by a kernel of their own
  uint16_t* parts;
  float* norms;
  size_t bytes;
};
SelectPlan select_plan(const BlockDims& p, int d, void* ws) {
  SelectPlan s;
  s.nbp = (p.nb + 63) / 64 * 64;
  const size_t rows = static_cast<size_t>(p.B) * p.Hkv * s.nbp;
  Carver c(ws);
  const bool mma = mma_select(p);
  s.split = mma && p.nb > 64;
  s.parts = c.take<uint16_t>(s.split ? 2 * rows * d : 0);
  s.norms = c.take<float>(s.split ? rows / 64 : 0);
  s.bytes = (c.used + 255) / 256 * 256;
  return s;
}

template <int D>
svoo_status launch_mma_select(const BlockDims& p, const void* q, const float* pool, const int32_t* lengths,
                              int32_t* idx, void* ws, int32_t* dev_err, cudaStream_t st) {
  const SelectPlan s = select_plan(p, D, ws);
  const int BHk = p.B * p.Hkv;
  const uint64_t rows = static_cast<uint64_t>(BHk) * s.nbp;
  CUtensorMap pm = {};
  if (s.split && encode_tiled_2d(&pm, s.parts, 2 * rows, D, kKeyTile, 64) != CUDA_SUCCESS) return SVOO_ERR_CUDA;
  if (!allow_smem(mma_select_kernel<D>, mma_sel_smem<D>())) return SVOO_ERR_CUDA;
  if (s.split)
    pool_split_kernel<D><<<dim3(s.nbp / 64, BHk), 256, 0, st>>>(p.nb, s.nbp, rows * D, pool, s.parts, s.norms);
  mma_select_kernel<D><<<dim3((p.Nq + kRowTile - 1) / kRowTile, BHk), kMmaSelThreads, mma_sel_smem<D>(), st>>>(
      pm, p, s.nbp, static_cast<const uint16_t*>(q), pool, s.split ? s.norms : nullptr, lengths, idx, dev_err);
  return launch_status();
}

// Queries of a CTA by the blocks: as many as the scores' shared memory allows (32 x
// 1024 blocks are 128 KB).
constexpr int sel_most_blocks(int tq) { return tq == 32 ? 1024 : tq == 8 ? 4096 : kMaxBlocks; }
constexpr size_t sel_scores_smem(int d, int tq, int pitch) {
  return sizeof(SelWarp) * (kSelThreads / 32) +
         static_cast<size_t>(tq) * (tq == 1 ? 2 * d + pitch : d + (pitch > d ? pitch : d)) * 4;
}

template <int D, int TQ>
svoo_status launch_select(const BlockDims& p, const void* q, const float* pool, const int32_t* lengths, int32_t* idx,
                          cudaStream_t st) {
  const int pitch = (p.nb + 31) / 32 * 32;
  if (!allow_smem(block_select_kernel<D, TQ>, sel_scores_smem(D, TQ, sel_most_blocks(TQ)))) return SVOO_ERR_CUDA;
  block_select_kernel<D, TQ><<<dim3((p.Nq + TQ - 1) / TQ, p.B * p.Hkv), kSelThreads, sel_scores_smem(D, TQ, pitch), st>>>(
      p, pitch, static_cast<const uint16_t*>(q), pool, lengths, idx);
  return launch_status();
}

template <int D>
svoo_status launch_select_d(const BlockDims& p, const void* q, const float* pool, const int32_t* lengths, int32_t* idx,
                            cudaStream_t st) {
  // one query a CTA where there are few
  if (p.Nq < 8 || p.nb > sel_most_blocks(8)) return launch_select<D, 1>(p, q, pool, lengths, idx, st);
  if (p.nb > sel_most_blocks(32)) return launch_select<D, 8>(p, q, pool, lengths, idx, st);
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
  const int tail = last > 0 ? 1 : 0;  // blocks behind a sequence stay, however many are asked for
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->d == 128)
    block_pool_kernel<128><<<grid, 128, 0, st>>>(p, static_cast<const uint16_t*>(k), lengths, tail, pool);
  else
    block_pool_kernel<64><<<grid, 128, 0, st>>>(p, static_cast<const uint16_t*>(k), lengths, tail, pool);
  return launch_status();
}

extern "C" size_t svoo_block_select_workspace_size(const svoo_block_shape* shape) {
  if (!block_shape_ok(shape)) return 0;
  return select_plan(block_dims(shape), shape->d, nullptr).bytes;
}

extern "C" svoo_status svoo_block_select(const svoo_block_shape* shape, const void* q, const float* pool,
                                         const int32_t* lengths, int32_t* idx, void* workspace, size_t workspace_bytes,
                                         int32_t* dev_err, void* stream) {
  if (!block_shape_ok(shape)) return SVOO_ERR_INVALID_ARG;
  if (shape->Nq == 0) return SVOO_OK;  // empty tensors have no address
  if (!q || !pool || !idx) return SVOO_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(idx, 4) || !aligned(lengths, 4) || !aligned(dev_err, 4) ||
      !aligned(workspace, 256))
    return SVOO_ERR_INVALID_ARG;
  const BlockDims p = block_dims(shape);
  const size_t need = select_plan(p, shape->d, nullptr).bytes;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SVOO_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (mma_select(p)) {
    if (shape->d == 128) return launch_mma_select<128>(p, q, pool, lengths, idx, workspace, dev_err, st);
    return launch_mma_select<64>(p, q, pool, lengths, idx, workspace, dev_err, st);
  }
  if (shape->d == 128) return launch_select_d<128>(p, q, pool, lengths, idx, st);
  return launch_select_d<64>(p, q, pool, lengths, idx, st);
}
