/*
 * svoo.h -- C ABI of the B200 (sm_100a) library for online QK co-clustered
 * block-sparse attention in video diffusion transformers.
 *
 * The path (one attention call of one layer), after the pages that describe it:
 *
 *   1. svoo_cluster      per head, bidirectional k-means of the query and key
 *                        tokens under the query-key interaction metric
 *                        ("Attention Sparsity is Input-Stable ... Online QK
 *                        Co-Clustering" (SVOO), abstract; "iCATS" sections 3.1
 *                        and 4.1: a quadratic form in feature space, the first
 *                        query step in feature space, later query steps under
 *                        the key-cluster metric, key steps under the
 *                        just-updated query clusters).
 *   2. svoo_build_mask   per head, the estimated attention mass of every
 *                        (query cluster, key cluster) pair from the centroids,
 *                        a keep-ratio or top-p selection of pairs ("PSA"
 *                        section 2 on SVG2's centroid scores and top-k cluster
 *                        selection; iCATS section 4.2 top-p; SVOO's offline
 *                        per-layer level enters as the keep ratio), then iCATS
 *                        tail merging of the query clusters (section 4.3,
 *                        appendix E.1).
 *   3. svoo_permute      stable permutation of the tokens into cluster order
 *                        (PSA section 2, SVG2's semantic-aware permutation),
 *                        query tiles, and the gathered Q, K, V in that order.
 *   4. svoo_sparse_attn  flash-style softmax(scale Q K^T) V restricted to the
 *                        kept cluster pairs, online softmax over the kept key
 *                        tiles only, O written back in token order.
 *
 * A second source of the plan replaces steps 1-2 for heads with a static
 * pattern: svoo_psa_mask writes the stripe mask of "PSA: Parameterized Stripe
 * Attention" (section 3.2, Algorithm 1) with every PSABlock as one group;
 * steps 3-4 then run unchanged.
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never allocates, frees or synchronises. Work is enqueued on `stream` (a
 *    cudaStream_t passed as void*; NULL = legacy default stream) in call order.
 *  - Q, K, V, O are bf16 [B, H, N, d] row-major; the N tokens of a head are
 *    N - n_text video tokens followed by n_text always-kept text tokens.
 *  - Arguments are validated on the host before any launch; a bad argument
 *    returns SVOO_ERR_INVALID_ARG and enqueues nothing. Launch failures return
 *    SVOO_ERR_CUDA.
 *  - Device-side problems (a pipeline wait that exceeded its time budget,
 *    out-of-range plan metadata) set bits in the caller's int32 error word
 *    `dev_err` (device memory, may be NULL) with atomicOr; the caller reads it
 *    when it chooses: 1 = attention wait timeout, 2 = clustering wait timeout,
 *    4 = plan metadata out of range, 8 = cluster label out of range. While a
 *    timeout bit (1 or 2) is set, the pipelined kernels skip their work, so
 *    clear the word after handling a timeout.
 *  - Limits (of the calls that take a svoo_shape): 1 <= B*H <= 65535, B*H*N < 2^31 - 256, 1 <= N - n_text, N <= 2^20,
 *    d in {64, 128},
 *    1 <= n_qc, n_kc <= 256, block_q in {64, 128}, 0 <= n_text, iters >= 1.
 *    Inputs must be finite. Centroid member sums are exact (fp64, with
 *    components |x| < 2^-24 counted as zero, so every partial sum is a
 *    multiple of 2^-31 below 2^22), and a centroid is its exact mean rounded
 *    once to fp32, whatever the order in which the GPU added the members.
 */
#ifndef SVOO_H
#define SVOO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SVOO_OK = 0,
    SVOO_ERR_INVALID_ARG = 1,
    SVOO_ERR_WORKSPACE = 2,
    SVOO_ERR_UNSUPPORTED = 3,
    SVOO_ERR_CUDA = 4,
    SVOO_ERR_TIMEOUT = 5,
    SVOO_ERR_INTERNAL = 6
} svoo_status;

/* Shape of one attention call. */
typedef struct {
    int B;      /* batch */
    int H;      /* heads */
    int N;      /* tokens per head, video then text */
    int d;      /* head dimension: 64 or 128 */
    int n_text; /* trailing always-kept text tokens (HunyuanVideo), 0 if none */
} svoo_shape;

/* Device buffers of one call's sparse plan; every array is caller-allocated
 * with the element counts that svoo_plan_counts returns. BH = B*H,
 * Gq = n_qc + (n_text > 0), Gk = n_kc + (n_text > 0), W = ceil(Gk / 64),
 * Tcap = ceil(N / block_q) + Gq, Ucap = ceil(N / 256) + Gq. All int32 unless
 * stated. */
typedef struct {
    uint64_t *kmask;     /* [BH][Gq][W] bit b of row a: query group a attends key group b.
                            Written by svoo_build_mask (after tail merging). */
    int32_t *q_label;    /* [BH][N]   merged query group of every token (text: n_qc) */
    int32_t *q_sizes;    /* [BH][Gq]  tokens per merged query group */
    int32_t *stats;      /* [BH][8]   kept pairs, non-empty query clusters, identical-mask
                            merges, tail moves round 1, tail moves round 2, query tiles
                            before merging, query tiles after, moved tokens */
    int32_t *q_perm;     /* [BH][N]   position in cluster order -> token (svoo_permute) */
    int32_t *q_off;      /* [BH][Gq+1] group start positions in q_perm */
    int32_t *k_perm;     /* [BH][N] */
    int32_t *k_off;      /* [BH][Gk+1] */
    int32_t *tiles;      /* [BH][Tcap][4] query tile: group, start position, rows, kv length */
    int32_t *tile_count; /* [BH] tiles in use per head */
    int32_t *units;      /* [BH][Ucap][4] attention work units: up to 256 consecutive rows of
                            one query group (two 128-row MMA tiles sharing every key/value
                            tile): group, start position, rows, kv length (svoo_permute) */
    int32_t *unit_count; /* [BH] units in use per head */
} svoo_plan;

/* Element counts of the svoo_plan arrays (in field order) for a shape. */
svoo_status svoo_plan_counts(const svoo_shape *shape, int n_qc, int n_kc, int block_q,
                             int64_t counts[12]);

/* ------------------------------------------------------------------ clustering
 * Bytes of device workspace svoo_cluster / svoo_cluster_step need. */
size_t svoo_cluster_workspace_size(const svoo_shape *shape, int n_qc, int n_kc);

#define SVOO_CLUSTER_WARM 1
#define SVOO_CLUSTER_IDENTITY 2

/* Co-clusters the video tokens of every head.
 *  q, k      : bf16 [B,H,N,d] (only the first N - n_text tokens are clustered).
 *  iters     : rounds of (query step, key step), each an assignment + update.
 *  flags     : bitwise OR of
 *              SVOO_CLUSTER_WARM: start from q_cent, k_cent, k_sizes as given
 *                (e.g. the previous timestep's), first query step under the
 *                key-cluster metric; without it, start from the tokens at
 *                floor(j*Nv/C) with a feature-space first query step;
 *              SVOO_CLUSTER_IDENTITY: every step in feature space (M = I):
 *                plain k-means of queries and keys separately, the
 *                independent Euclidean clustering (SVG2's) that iCATS sec. 3.1
 *                and App. D (Table 3) compare the co-clustering against.
 *              Any other bit is SVOO_ERR_INVALID_ARG.
 *  q_assign, k_assign : int32 [BH][N - n_text] cluster of every video token.
 *  q_cent, k_cent     : fp32 [BH][n_qc|n_kc][d] centroids (in/out).
 *  q_sizes, k_sizes   : int32 [BH][n_qc|n_kc] members per cluster (k_sizes in/out).
 * Assignment: argmin_j (x - mu_j)^T M (x - mu_j), ties to the smaller j, where
 * M is the normalised second moment of the other side's clusters (identity in
 * the cold first query step, and in every step under SVOO_CLUSTER_IDENTITY);
 * M, nu_j = M mu_j and kappa_j = mu_j . nu_j in
 * fp64. Scores come from tcgen05 MMAs against nu split into two bf16 rows
 * (with kappa folded in); when more than one cluster lies within the MMA's
 * error bound of the best, those candidates (or, when there are many, all
 * clusters) are compared exactly in fp64, so the result is that of an fp64
 * evaluation. Update: member means from exact sums (see the limits above), so
 * equal labels give bit-identical centroids; an empty cluster keeps its
 * centroid. Each side's first step of a call sums all members; later steps
 * move only the tokens whose label changed (exact, so the same bits). The
 * workspace holds those kept sums, so calls sharing one workspace must not
 * overlap on the GPU. */
svoo_status svoo_cluster(const svoo_shape *shape, const void *q, const void *k, int n_qc,
                         int n_kc, int iters, int flags, int32_t *q_assign, int32_t *k_assign,
                         float *q_cent, float *k_cent, int32_t *q_sizes, int32_t *k_sizes,
                         void *workspace, size_t workspace_bytes, int32_t *dev_err,
                         void *stream);

/* One half-step of the above for one side: assigns the video tokens of x to
 * the centroids `cent` (in/out) under the metric of (metric_cent, metric_sizes)
 * (metric_C clusters; identity if metric_cent is NULL, and metric_C is then
 * ignored), then updates `cent` and `sizes`. Used for warm starts and for
 * step-level parity checks. */
svoo_status svoo_cluster_step(const svoo_shape *shape, const void *x, int C, float *cent,
                              int32_t *sizes, int32_t *assign, const float *metric_cent,
                              const int32_t *metric_sizes, int metric_C, void *workspace,
                              size_t workspace_bytes, int32_t *dev_err, void *stream);

/* Allocation-free variant of svoo_cluster_step. The paper pages have no
 * counterpart: it exists for callers that may not allocate device memory
 * themselves (code inside a host framework that owns all device memory through
 * its own pool, or a latency-critical loop that forbids allocation after
 * start-up). Arguments as svoo_cluster_step minus the workspace; the scratch
 * is a fixed array of SVOO_STATIC_SCRATCH_BYTES compiled into the library,
 * held on every GPU that loads it until the process exits. Shapes whose
 * scratch would exceed it return SVOO_ERR_WORKSPACE and enqueue nothing (16 MiB
 * covers, e.g., B*H = 12, d = 128, 128 clusters). The first call on a device
 * looks up the array's device address (make it before any stream capture).
 * All calls share the array and each clears the accumulators it uses; calls
 * that overlap on the GPU (e.g. on two streams) race. */
#define SVOO_STATIC_SCRATCH_BYTES (16u << 20)
svoo_status svoo_cluster_step_static(const svoo_shape *shape, const void *x, int C, float *cent,
                                     int32_t *sizes, int32_t *assign, const float *metric_cent,
                                     const int32_t *metric_sizes, int metric_C, int32_t *dev_err,
                                     void *stream);

/* ------------------------------------------------------------------ mask
 * Bytes of device workspace svoo_build_mask needs. */
size_t svoo_mask_workspace_size(const svoo_shape *shape, int n_qc, int n_kc);

/* Builds the key-cluster mask of every query cluster and tail-merges them.
 *  keep[BH] (fp32, device): select_mode 0 -> keep ratio r in (0, 1]: the head
 *    keeps K = ceilf(r * (n_qc*n_kc)) pairs (fp32 product), at least each query
 *    cluster's best pair; select_mode 1 -> top-p p in [0, 1]: the shortest
 *    prefix of the same order whose mass (fixed point floor(w * 2^32)) reaches
 *    ceil(p * total), again at least the per-cluster best pairs.
 *  Pair order: per-cluster best first, then w descending, then query cluster
 *    ascending, then key cluster ascending; w is the estimated attention mass
 *    n_a * n_b e^(s_ab - m_a) / Z_a with s_ab = scale * mu_a . c_b, computed
 *    in fp32 with a fixed operation order (bit-identical to the oracle).
 *  Tail merging: identical masks merge into the lowest id; then merge_rounds
 *    rounds in which mutually nearest (Hamming distance of masks) clusters
 *    whose tails (size mod block_q) fit one block move the smaller tail into
 *    the other, whose mask becomes the union. Text tokens (if any) form query
 *    group n_qc attending everything, and key group n_kc, which every query
 *    group keeps; they are outside the budget and the merging.
 *  Writes plan->kmask, q_label, q_sizes, stats. */
svoo_status svoo_build_mask(const svoo_shape *shape, const float *q_cent, const float *k_cent,
                            const int32_t *q_sizes, const int32_t *k_sizes,
                            const int32_t *q_assign, const float *keep, int n_qc, int n_kc,
                            int select_mode, int block_q, int merge_rounds, float scale,
                            const svoo_plan *plan, void *workspace, size_t workspace_bytes,
                            int32_t *dev_err, void *stream);

/* ------------------------------------------------------------------ static stripe mask
 * Number of PSABlocks, ceil(T/bt) ceil(H/bh) ceil(W/bw), of a token grid; 0
 * for a non-positive argument. */
int svoo_psa_block_count(int grid_t, int grid_h, int grid_w, int block_t, int block_h,
                         int block_w);

#define SVOO_PSA_INF 2147483647 /* stride "infinity": one diagonal band on that axis */

/* The plan of the stripe mask M(Tw, To, Ts, Sw, So, Ss) of PSA ("PSA:
 * Parameterized Stripe Attention", section 3.2 and Algorithm 1), in place of
 * svoo_cluster + svoo_build_mask.
 *  grid_t, grid_h, grid_w : the video tokens form a (T, H, W) grid in raster
 *        order (T*H*W must equal N - n_text).
 *  block_t, block_h, block_w : the PSABlock. The block grid is (T', H', W') =
 *        (ceil(T/bt), ceil(H/bh), ceil(W/bw)), nb = T'H'W' <= 256 blocks,
 *        numbered in raster order; blocks on the far edges hold only the
 *        tokens that exist (no padding).
 *  params : int32 [B*H][6], DEVICE: (Tw, To, Ts, Sw, So, Ss) of each head.
 *        Tw, Sw >= 0; Ts, Ss >= 1, SVOO_PSA_INF for infinity. A head with a
 *        parameter out of range gets no video block pair (its text group, if
 *        any, is still kept) and sets bit 4 in dev_err.
 *  Masking is at PSABlock granularity: query block a keeps key block b when
 *  Algorithm 1 holds for the block indices (frame = index / (H'W'), in-frame
 *  position = index % (H'W')), i.e. the frame distance D satisfies
 *  (|D - To| mod Ts) <= Tw - 1 and the in-frame distance E satisfies
 *  (|E - So| mod Ss) <= Sw - 1. Text tokens form group nb, which attends
 *  every group and which every group attends.
 *  Writes plan->kmask, q_label (a token's block), q_sizes and stats (kept
 *  video block pairs, nb, 0, 0, 0, query tiles, query tiles, 0), sized by
 *  svoo_plan_counts(shape, nb, nb, block_q), and k_assign (int32
 *  [B*H][N - n_text], the key block of every video token) for svoo_permute.
 *  Then call svoo_permute and svoo_sparse_attn with n_qc = n_kc = nb: the
 *  stable sort lays every block's tokens out contiguously in raster order,
 *  which is PSA's block-centric (T', H', W', bt, bh, bw) layout. */
svoo_status svoo_psa_mask(const svoo_shape *shape, int grid_t, int grid_h, int grid_w,
                          int block_t, int block_h, int block_w, const int32_t *params,
                          int block_q, svoo_plan *plan, int32_t *k_assign, int32_t *dev_err,
                          void *stream);

/* ------------------------------------------------------------------ permutation
 * Stable counting sorts of the merged query labels (plan->q_label) and of the
 * key labels (k_assign, text tokens as group n_kc): q_perm/q_off, k_perm/k_off;
 * the query tile table and per-head tile counts; and the gathered copies
 *   qp[p] = q[q_perm[p]], kp[p] = k[k_perm[p]], vp[p] = v[k_perm[p]]
 * (bf16 [B,H,N,d], caller-allocated) that svoo_sparse_attn reads. */
svoo_status svoo_permute(const svoo_shape *shape, const void *q, const void *k, const void *v,
                         const int32_t *k_assign, int n_qc, int n_kc, int block_q,
                         const svoo_plan *plan, void *qp, void *kp, void *vp, int32_t *dev_err,
                         void *stream);

/* ------------------------------------------------------------------ attention
 * o[token] = softmax(scale * q_token . K_kept^T) V_kept over the keys of the
 * key groups that the token's query group keeps, for every query tile of the
 * plan; qp/kp/vp are the cluster-ordered copies from svoo_permute; o is bf16
 * [B,H,N,d] in token order. A query whose kept key groups are all empty gets
 * o = 0. tcgen05 MMAs (bf16 in, fp32 accumulate) into tensor memory, online
 * softmax in fp32, P rounded to bf16 for the second product. */
svoo_status svoo_sparse_attn(const svoo_shape *shape, const void *qp, const void *kp,
                             const void *vp, const svoo_plan *plan, int n_qc, int n_kc,
                             int block_q, float scale, void *o, int32_t *dev_err, void *stream);

/* ------------------------------------------------------------------ top-p schedule
 * SNR-guided top-p of every call of a denoising run ("iCATS" section 4.2 and
 * appendix A: top-p follows a smooth function of the log signal-to-noise
 * ratio, fixed offline from the noise schedule, with dense attention before
 * the first sparse call; the budget stays steady early and late and falls in
 * the middle). The pages give no formula; this library reads it as
 *   s = 1 - t/steps, sigma = shift*s / (1 + (shift - 1)*s)   (flow matching),
 *   p(t) = p_min + (tau - p_min) / (1 + SNR(t)),  SNR = ((1 - sigma)/sigma)^2,
 * i.e. a logistic in log SNR: tau at pure noise, p_min in the noise-free
 * limit, (tau + p_min)/2 where SNR = 1; p(t) = 1 for t < warmup.
 * Host code only (no GPU work): writes p[0..steps-1] (HOST memory, fp32),
 * ready to be passed as the per-head keep values of svoo_build_mask with
 * select_mode 1. Requires steps >= 1, warmup >= 0, 0 <= p_min <= tau <= 1,
 * shift > 0; otherwise SVOO_ERR_INVALID_ARG and p is left untouched. */
svoo_status svoo_snr_top_p(int steps, int warmup, double p_min, double tau, double shift,
                           float *p);

/* ------------------------------------------------------------------ block-selected attention
 * Attention of language models over the key blocks that every query selects by
 * a cheap score, its gradient, and its form for single tokens over a cache.
 * The H query heads form groups of H / Hkv that share a key head and one
 * selection; the N-token shape limits of this header's other calls do not
 * apply, those of svoo_block_shape do. */

/* Shape of one call.
 *  q, o : bf16 [B][H][Nq][d];  k, v : bf16 [B][Hkv][cap][d], of which the first
 *  Nk rows of every head are keys (cap > Nk: a view into a longer buffer, which
 *  may begin anywhere in it: nothing behind the last head's last key is read).
 *  lengths (int32 [B], DEVICE, may be NULL = Nk): the valid keys of every
 *  sequence, 0 <= lengths[b] <= Nk (clamped). What lies behind them is never
 *  used and may hold anything, NaN included.
 *  Position of query i: q_start + i, or with q_start = -1 lengths[b] - Nq + i
 *  (the queries are the last Nq tokens of their sequence). Causal: a query sees
 *  the keys up to its own position, and nothing when its position is outside
 *  [0, lengths[b]). Not causal: every query sees all keys of its sequence.
 *  Limits: 1 <= H / Hkv <= 128, B*H <= 65535, 0 <= Nq <= 2^20,
 *  1 <= Nk <= cap <= 2^20, B*H*Nq and B*Hkv*cap < 2^31 - 256, d in {64, 128},
 *  block a multiple of 64 up to 1024, 1 <= n_sel <= 256, sink + local <= n_sel,
 *  local >= 1 when causal and 0 when not, -1 <= q_start <= 2^20. Valid rows of
 *  q, k, v must be finite. */
typedef struct {
    int B, H, Hkv;
    int Nq, Nk, cap;
    int d;
    int block;   /* keys per block */
    int n_sel;   /* blocks per query, forced ones included */
    int sink;    /* the first blocks, kept by every query */
    int local;   /* causal: the query's own block and the local - 1 before it */
    int causal;  /* 0 or 1 */
    int q_start; /* position of query 0, or -1 */
} svoo_block_shape;

/* pool[b][hk][c] = mean of block c's valid keys: fp32 [B][Hkv][ceil(Nk / block)][d],
 * summed in fp64 and rounded once; a block without keys gets zeros. last > 0
 * renews only the last `last` blocks that hold keys of each sequence (after a
 * token was appended, 1), and leaves the others as they are. Uses B, Hkv, Nk,
 * cap, d and block of the shape. */
svoo_status svoo_block_pool(const svoo_block_shape *shape, const void *k, const int32_t *lengths,
                            int last, float *pool, void *stream);

/* idx: int32 [B][Hkv][Nq][n_sel], ascending block ids, then -1. The forced
 * blocks and the best of the others by
 *   score(t, c) = (sum over the group's heads of q[t]) . pool[c],
 * equal scores to the lower block; decided as in fp64 for all finite q and pool. Causal: the blocks up to
 * the query's own, which is always kept and never scored. A query outside its
 * sequence selects nothing. The workspace (256-byte aligned; a call of few
 * queries needs none, 0 bytes) must not be shared by calls that overlap on the
 * GPU. */
size_t svoo_block_select_workspace_size(const svoo_block_shape *shape);
svoo_status svoo_block_select(const svoo_block_shape *shape, const void *q, const float *pool,
                              const int32_t *lengths, int32_t *idx, void *workspace,
                              size_t workspace_bytes, int32_t *dev_err, void *stream);

/* o = softmax(scale q K^T) V and lse (fp32 [B][H][Nq]) = log of the softmax's
 * denominator, over the keys that the query sees in its selected blocks. idx as
 * above, from svoo_block_select or anywhere else: a query's list ends at the
 * first entry that is out of range or not above the one before it, and an entry
 * other than -1 there sets bit 4 in dev_err. A query without keys gets o = 0,
 * lse = -inf. sink and local are not used. fp32 softmax and sums; P is rounded
 * to bf16 for the second product. The workspace (256-byte aligned) must not be
 * shared by calls that overlap on the GPU. Most calls need none (0 bytes); where
 * neighbouring queries' selections, blocks of a multiple of 128 keys, would
 * together be nearly all blocks, a call keeps every query's part of each 128
 * selected keys there: 4 * (d + 2) bytes each, up to 4.5 GB. */
size_t svoo_block_attn_workspace_size(const svoo_block_shape *shape);
svoo_status svoo_block_attn(const svoo_block_shape *shape, const void *q, const void *k,
                            const void *v, const int32_t *idx, const int32_t *lengths, float scale,
                            void *o, float *lse, void *workspace, size_t workspace_bytes,
                            int32_t *dev_err, void *stream);

/* Gradient of svoo_block_attn with respect to q, k and v (the selection is a
 * constant): dq bf16 [B][H][Nq][d]; dk, dv bf16 [B][Hkv][Nk][d], contiguous
 * whatever cap is, zero for keys that no query attends to. o, lse: what the
 * forward call wrote. grad_o: bf16 [B][H][Nq][d]. fp32 sums; P and dS are
 * rounded to bf16 for the products of dv and dk, dS enters dq's as two bf16
 * parts, rowsum(grad_o * o) is taken from the rounded o: with the outputs' own
 * rounding some 2.5e-3 of the formula in the 2-norm, and where terms cancel (a
 * query of one key) the error goes by the terms, not by their sum. Every sum
 * runs in a fixed order, so equal calls give equal bits. The workspace (256-byte aligned) must
 * not be shared by calls that overlap on the GPU. */
size_t svoo_block_attn_backward_workspace_size(const svoo_block_shape *shape);
svoo_status svoo_block_attn_backward(const svoo_block_shape *shape, const void *q, const void *k,
                                     const void *v, const void *o, const float *lse,
                                     const void *grad_o, const int32_t *idx, const int32_t *lengths,
                                     float scale, void *dq, void *dk, void *dv, void *workspace,
                                     size_t workspace_bytes, int32_t *dev_err, void *stream);

/* One token per sequence (Nq = 1) over a cache of cap slots, all valid ones
 * visible (the order of the slots does not matter; causal and q_start are not
 * used): o bf16 [B][H][1][d], lse fp32 [B][H][1].
 * fp32 softmax and sums; P is rounded to bf16 for the second product, weights
 * are not.
 *  idx (int32 [B][Hkv][1][n_sel], may be NULL): only the slots of those blocks.
 *  weight (fp32 [B][Hkv][cap], may be NULL): weight[slot] += sum over the
 *  group's heads of the slot's softmax weight, for every valid slot. A call that
 *  times out, or finds a timeout bit in dev_err, leaves them as they were
 *  (without dev_err there is no word to tell it by). idx and weight together are
 *  SVOO_ERR_UNSUPPORTED.
 * Workspace: svoo_cache_attn_workspace_size(shape, idx != NULL, weight != NULL)
 * bytes (may be 0), 256-byte aligned, not shared by calls that overlap on the
 * GPU. */
size_t svoo_cache_attn_workspace_size(const svoo_block_shape *shape, int selected, int weights);
svoo_status svoo_cache_attn(const svoo_block_shape *shape, const void *q, const void *k,
                            const void *v, const int32_t *lengths, const int32_t *idx, float scale,
                            float *weight, void *o, float *lse, void *workspace,
                            size_t workspace_bytes, int32_t *dev_err, void *stream);

/* Brings every sequence that holds more than `keep` slots down to `keep`, in
 * place and for each key head by itself. Kept are the slots of the first `sink`
 * positions (pos < sink), those of the last `recent` (of the largest position
 * in the cache), then the heaviest by weight; equal weights keep the lower slot,
 * NaN counts as the lightest. Kept rows stay where they are, except that the
 * i-th evicted slot below `keep` receives the i-th kept one at or behind it: k,
 * v (bf16 [B][Hkv][cap][d]), weight (fp32 [B][Hkv][cap]) and pos (int32
 * [B][Hkv][cap], the token position of every slot) move together. Slots at or
 * behind `keep` are left as they were. lengths[b] becomes min(lengths[b], keep).
 * Requires 1 <= keep, 0 <= sink, recent, sink + recent <= keep. */
size_t svoo_cache_evict_workspace_size(int B, int Hkv, int cap, int keep);
svoo_status svoo_cache_evict(int B, int Hkv, int cap, int d, int keep, int sink, int recent,
                             void *k, void *v, float *weight, int32_t *pos, int32_t *lengths,
                             void *workspace, size_t workspace_bytes, void *stream);

const char *svoo_status_string(svoo_status s);

/* Library version, (major << 16) | minor. */
int svoo_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SVOO_H */
