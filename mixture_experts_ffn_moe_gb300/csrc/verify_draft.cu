// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Mathematics.  Row 0 of a sequence's target rows is the distribution after its committed tokens, row 1 + j the
// one after drafted node j.  Node j was drafted as a child of parent(j); the coin of the parent's row decides it.
//  * With draft probabilities q (a chain): token x is kept iff coin * q(x) < p(x); the first refused one is
//    replaced by a sample of max(p - q, 0).  (Speculative sampling; the result is distributed as p.)
//  * Without (a tree of candidates): the children of a node share [0, 1) in order, p(child) each; the child whose
//    share holds the node's coin is kept, else the next token is a sample of p without the children.
// Where all of a path is kept, the next token is a sample of the last row.  A sample is the first token x with
// sum_{i <= x} w_i > u * sum_i w_i.
//
// Arithmetic.  coin * q is exact in 64 bits.  The weights count as integers in units of 2^-60 (rounded to nearest;
// any p of 2^-37 and more is a whole number of them), so their sums are exact, do not depend on the order of the
// threads, and the comparison with the threshold is one of integers.  The integers are not formed one by one: adding
// 1, 1.5 * 2^-23 and 1.5 * 2^-37 to p and to what each sum leaves over puts three pieces of the integer into the low
// mantissa bits of three floats, whose bit patterns are added up as 32-bit integers (the constants' share is known and
// taken off at the end).  That is 8 additions of floats and 3 of integers a weight; shifting the mantissa into place
// took about 45 instructions and bound the kernel, and FP64 runs at a sixtieth of the fp32 rate here.
//
// Bound: the one row (two with q) of the vocabulary that is sampled from; everything else is a gather of at most
// 64 probabilities.  In practice a chain of dependent reads: offsets, nodes, their probabilities, the row, and the
// part of it that holds the threshold.  A cluster of CTAs shares a sequence's row, a warp takes tiles of 1024
// tokens with all of its loads in flight, the CTAs' sums meet through distributed shared memory, and one warp
// reads the one tile again in which the running sum passes the threshold.
//
// Measured: 32 chains of 7 tokens, 129,280 words, with the draft's probabilities: 13.2 us; 2 trees of 24 nodes, 32,003 words:
// 8.7 us.  The pass over the rows takes about 4 us of the former, the reads that depend on one another the rest.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "step_ops.cuh"

namespace gbmoe {
namespace {

namespace cg = cooperative_groups;

constexpr int kVThreads = 256;   // two CTAs an SM at about 120 registers
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kVTile = 1024;     // tokens of a tile: 32 a lane
constexpr int kVTiles = 2048;    // tiles of a CTA at most

struct VerifyArgs {
  const float* target;  // [N + B, V], row stride ldt
  const float* draft;   // [N, V], row stride ldd; null: a tree of candidates
  long long ldt, ldd;
  const int32_t* tokens;   // [N]
  const int32_t* parents;  // [N] or null (chain)
  const int32_t* offsets;  // [B + 1]
  const float* coins;      // [N + B]
  const float* last;       // [B]
  int32_t* out_tokens;     // [B, max_nodes + 1]
  int32_t* path;           // [B, max_nodes]
  int32_t* accepted;       // [B]
  int N, V, max_nodes;
};

// The sum of weights as three 32-bit sums of bit patterns (up to 32 of them).
struct Levels {
  uint32_t a = 0, b = 0, c = 0;
};
constexpr float kC2 = 0x1.8p-23f, kC3 = 0x1.8p-37f;  // spacing 2^-46 and 2^-60
__device__ __forceinline__ void split3(float p, uint32_t& x, uint32_t& y, uint32_t& z) {
  const float t = __fadd_rn(p, 1.f), r = __fadd_rn(p, -__fadd_rn(t, -1.f)), u = __fadd_rn(r, kC2);
  x = __float_as_uint(t);
  y = __float_as_uint(u);
  z = __float_as_uint(__fadd_rn(__fadd_rn(r, -__fadd_rn(u, -kC2)), kC3));
}
// Probabilities above 1 count as 1, negative ones and NaN as 0.
__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.f), 1.f); }
// Adds p, or max(p - q, 0).
template <bool Q>
__device__ __forceinline__ void add_weight(Levels& l, float p, float q) {
  uint32_t x, y, z;
  if constexpr (Q) {
    const bool more = p > q;
    split3(more ? p : 0.f, x, y, z);
    uint32_t x2, y2, z2;
    split3(more ? q : 0.f, x2, y2, z2);
    l.a += x - x2;
    l.b += y - y2;
    l.c += z - z2;
  } else {
    split3(p, x, y, z);
    l.a += x;
    l.b += y;
    l.c += z;
  }
}
// The integer of a sum of n weights.
template <bool Q>
__device__ __forceinline__ uint64_t integer(const Levels& l, int n) {
  const uint32_t k = Q ? 0u : static_cast<uint32_t>(n);
  const int64_t a = static_cast<int32_t>(l.a - k * 0x3f800000u);
  const int64_t b = static_cast<int32_t>(l.b - k * 0x34400000u);  // kC2
  const int64_t c = static_cast<int32_t>(l.c - k * 0x2d400000u);  // kC3
  return static_cast<uint64_t>((a << 37) + (b << 14) + c);
}
__device__ __forceinline__ uint64_t integer_of(float p) {
  Levels l;
  add_weight<false>(l, p, 0.f);
  return integer<false>(l, 1);
}

// u * 2^64 (rounded down) for u in [0, 1); what lies outside is brought to the nearest end.
__device__ __forceinline__ uint64_t fraction64(float u) {
  const uint32_t b = __float_as_uint(fminf(u > 0.f ? u : 0.f, 0x1.fffffep-1f));
  const int e = static_cast<int>(b >> 23) - 86;  // u = m * 2^(e - 64)
  const uint64_t m = e <= -86 ? 0 : (b & 0x7fffffu) | 0x800000u;
  return e >= 0 ? m << e : (e < -63 ? 0 : m >> -e);
}

// The two halves of a cluster barrier: every thread of every CTA arrives, and waits for all of them.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's 32 probabilities of the tile at `base` (clamped), all loads in flight: 4 neighbours of every 128 tokens, as
// 16 bytes where rows start on them (VEC).
constexpr int kGroups = 8;  // of 128 tokens
template <bool VEC, bool Q>
__device__ __forceinline__ void load_tile(const float* p, const float* q, int base, int V, int lane, float (&a)[32], float (&b)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const int at = base + (i / 4 * 32 + lane) * 4;
    if constexpr (VEC) {
      const bool in = at + 3 < V;  // V is a multiple of 4
      const float4 x = in ? __ldg(reinterpret_cast<const float4*>(p + at)) : make_float4(0.f, 0.f, 0.f, 0.f);
      a[i] = x.x; a[i + 1] = x.y; a[i + 2] = x.z; a[i + 3] = x.w;
      if constexpr (Q) {
        const float4 y = in ? __ldg(reinterpret_cast<const float4*>(q + at)) : make_float4(0.f, 0.f, 0.f, 0.f);
        b[i] = y.x; b[i + 1] = y.y; b[i + 2] = y.z; b[i + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[i + j] = at + j < V ? __ldg(p + at + j) : 0.f;
        if constexpr (Q) b[i + j] = at + j < V ? __ldg(q + at + j) : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a[i] = clamp01(a[i]);
    if constexpr (Q) b[i] = clamp01(b[i]);
  }
}

// The sum of a tile's weights in units of 2^-60 (a lane's share), and the plain sum of its probabilities into fs.
template <bool VEC, bool Q>
__device__ __forceinline__ uint64_t sum_tile(const float* p, const float* q, int base, int V, int lane, float& fs) {
  float a[32], b[32];
  load_tile<VEC, Q>(p, q, base, V, lane, a, b);
  Levels l;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    add_weight<Q>(l, a[i], b[i]);
    fs += a[i];
  }
  return integer<Q>(l, 32);
}

// The first token of the tile at `base` with before + (running sum) > level, by a whole warp; -1 if there is none.
// Tokens of the n nodes whose parent is `stop` count nothing.
template <bool VEC, bool Q>
__device__ __forceinline__ int search_tile(const float* p, const float* q, int base, int V, int lane, uint64_t before, uint64_t level,
                                           const int* tok, const int* par, int n, int stop) {
  float a[32], b[32];
  load_tile<VEC, Q>(p, q, base, V, lane, a, b);
  for (int j = 0; j < n; ++j)
    if (par[j] == stop && tok[j] >= base && tok[j] < base + kVTile) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (base + (i / 4 * 32 + lane) * 4 + i % 4 == tok[j]) a[i] = 0.f;
    }
  // tokens in order: groups of 128, in them 4 a lane.  The groups' sums do not wait for each other.
  uint64_t grp[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    Levels l;
#pragma unroll
    for (int j = 0; j < 4; ++j) add_weight<Q>(l, a[i * 4 + j], b[i * 4 + j]);
    grp[i] = integer<Q>(l, 4);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kGroups; ++i) grp[i] += __shfl_xor_sync(0xffffffffu, grp[i], o);
  int at = -1;
  float ga[4], gb[4];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    if (at >= 0) continue;
    if (before + grp[i] > level) {
      at = i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ga[j] = a[i * 4 + j];
        if constexpr (Q) gb[j] = b[i * 4 + j];
      }
    } else {
      before += grp[i];
    }
  }
  if (at < 0) return -1;
  uint64_t w[4], run = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    Levels l;
    add_weight<Q>(l, ga[j], gb[j]);
    w[j] = integer<Q>(l, 1);
    run += w[j];
  }
  const uint64_t own = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  const unsigned hit = __ballot_sync(0xffffffffu, before + run > level);
  const int who = __ffs(hit) - 1;  // the group's last lane at the latest
  uint64_t sum = before + run - own;
  int x = base + (at * 32 + lane) * 4;
  bool here = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sum += w[j];
    if (!here && sum > level) { here = true; x += j; }
  }
  return __shfl_sync(0xffffffffu, x, who);
}

struct Shared {
  int tok[64], par[64];
  float p[64];
  unsigned char again[64];
  unsigned long long taken, okmask;
  uint64_t share[64];  // p in units of 2^-60
  int bad;
  uint64_t warp_tot[kVWarps];
  float warp_f[kVWarps];
  uint64_t cta_tot[kMaxCluster];
  float cta_f[kMaxCluster];
  int found;
};

template <bool VEC>
__global__ void __launch_bounds__(kVThreads, 2) verify_kernel(VerifyArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  cluster_arrive();  // waited for before the first store to another CTA, on every path
  pdl_wait();

  // ---- the nodes: probabilities of every drafted token, gathered at once
  const int lo = a.offsets[b], hi = a.offsets[b + 1];
  const int n = hi - lo;
  const bool bad_range = lo < 0 || hi < lo || hi > a.N || n > a.max_nodes;
  if (tid == 0) { sh.bad = bad_range; sh.taken = 0; sh.okmask = 0; sh.found = -1; }
  __syncthreads();
  const long long row0 = static_cast<long long>(lo) + b;
  float coin = 0.f, q = 0.f;
  if (!bad_range && tid < n) {
    const int tok = a.tokens[lo + tid], par = a.parents ? a.parents[lo + tid] : tid - 1;
    const bool ok = tok >= 0 && tok < a.V && par >= -1 && par < tid;
    float p = 0.f;
    if (ok) {  // (all three loads under way before any is used)
      p = __ldg(a.target + (row0 + par + 1) * a.ldt + tok);
      coin = __ldg(a.coins + row0 + par + 1);
      if (a.draft) q = __ldg(a.draft + (lo + tid) * a.ldd + tok);
    }
    if (!ok) sh.bad = 1;
    p = clamp01(p);
    q = clamp01(q);
    sh.tok[tid] = tok;
    sh.par[tid] = par;
    sh.p[tid] = p;
    sh.share[tid] = integer_of(p);
  }
  __syncthreads();
  const bool bad = sh.bad != 0;
  if (!bad && tid < n) {  // a sibling's repeat has no share of its own
    bool again = false;
    const int my_par = sh.par[tid], my_tok = sh.tok[tid];
#pragma unroll 8
    for (int j = 0; j < tid; ++j) again |= (sh.par[j] == my_par) & (sh.tok[j] == my_tok);
    sh.again[tid] = again;
  }
  __syncthreads();
  if (!bad && tid < n) {
    bool taken;
    if (a.draft) {
      taken = static_cast<double>(coin) * static_cast<double>(q) < static_cast<double>(sh.p[tid]);
    } else {
      uint64_t before = 0;  // the earlier siblings' shares
      float about = 0.f;    // the same in fp32: 64 bits hold sums below 16
      const int my_par = sh.par[tid];
#pragma unroll 8
      for (int j = 0; j < tid; ++j) {
        const bool counts = sh.par[j] == my_par && !sh.again[j];
        before += counts ? sh.share[j] : 0;
        about += counts ? sh.p[j] : 0.f;
      }
      const uint64_t c = fraction64(coin) >> 4;
      taken = !sh.again[tid] && about < 8.f && c >= before && c < before + sh.share[tid];
    }
    if (taken) atomicOr(&sh.taken, 1ull << tid);
  }
  __syncthreads();
  if (!bad && tid < n) {  // kept: taken, and so is every ancestor
    const unsigned long long taken = sh.taken;
    int up = tid;
    while (up >= 0 && ((taken >> up) & 1)) up = sh.par[up];
    if (up < 0) atomicOr(&sh.okmask, 1ull << tid);
  }
  __syncthreads();
  // the kept nodes are one path, so the last one is the deepest
  const int stop = 63 - __clzll(static_cast<long long>(sh.okmask)), count = __popcll(sh.okmask);

  // ---- the row that the next token is drawn from
  const float* prow = a.target + (row0 + stop + 1) * a.ldt;
  const bool has_q = a.draft && stop + 1 < n;
  const float* qrow = has_q ? a.draft + (lo + static_cast<long long>(stop) + 1) * a.ldd : nullptr;
  extern __shared__ uint64_t tile_sum[];  // [tiles of this CTA]
  const int tiles = (a.V + kVTile - 1) / kVTile, per_cta = (tiles + C - 1) / C;
  const int tile0 = min(tiles, rank * per_cta), my_tiles = min(tiles, tile0 + per_cta) - tile0;
  int next = -1;
  // A CTA's shared memory may be written from outside only once that CTA is known to run: every one has arrived at its
  // start, so the reads of the nodes hide this wait.
  cluster_wait();
  // residual: 1 = the draft's share, or the refused children, taken away; 0 = the plain row where nothing is left
  for (int residual = 1; !bad && residual >= 0 && next < 0; --residual) {
    const bool use_q = has_q && residual;
    float fs = 0.f;
    uint64_t mine = 0;  // lane 0: the warp's tiles
    for (int t = warp; t < my_tiles; t += kVWarps) {
      const int at = (tile0 + t) * kVTile;
      uint64_t sum = use_q ? sum_tile<VEC, true>(prow, qrow, at, a.V, lane, fs) : sum_tile<VEC, false>(prow, nullptr, at, a.V, lane, fs);
      if (!a.draft && residual)
        for (int j = lane; j < n; j += 32)
          if (sh.par[j] == stop && !sh.again[j] && sh.tok[j] / kVTile == tile0 + t) sum -= sh.share[j];
      sum = warp_sum64(sum);
      if (lane == 0) tile_sum[t] = sum;
      mine += sum;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fs += __shfl_xor_sync(0xffffffffu, fs, o);
    if (lane == 0) { sh.warp_tot[warp] = mine; sh.warp_f[warp] = fs; }
    __syncthreads();
    if (tid < C) {  // this CTA's total into slot `rank` of every CTA of the cluster
      uint64_t tot = 0;
      float f = 0.f;
      for (int w = 0; w < kVWarps; ++w) { tot += sh.warp_tot[w]; f += sh.warp_f[w]; }
      Shared* other = cluster.map_shared_rank(&sh, tid);
      other->cta_tot[rank] = tot;
      other->cta_f[rank] = f;
    }
    cluster.sync();
    uint64_t total = 0, before = 0;
    float f = 0.f;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += sh.cta_tot[r];
      total += sh.cta_tot[r];
      f += sh.cta_f[r];
    }
    if (!(f <= 8.f)) break;  // not probabilities: 64 bits would overflow at 16
    if (total != 0) {
      // floor(u * total) for u in [0, 1): x is the first token whose running sum is above it
      const uint64_t level = __umul64hi(fraction64(a.last[b]), total);
      if (warp == 0 && level >= before && level < before + sh.cta_tot[rank]) {  // in this CTA's part
        int t = 0;
        for (int t0 = 0; t0 < my_tiles; t0 += 32) {  // the tile
          uint64_t run = t0 + lane < my_tiles ? tile_sum[t0 + lane] : 0;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, before + run > level);
          if (hit) {
            const int l = __ffs(hit) - 1;
            t = t0 + l;
            const uint64_t upto = __shfl_sync(0xffffffffu, run, l ? l - 1 : 0);
            before += l ? upto : 0;
            break;
          }
          before += __shfl_sync(0xffffffffu, run, 31);
        }
        const int at = (tile0 + t) * kVTile, gone = a.draft || !residual ? 0 : n;
        const int x = use_q ? search_tile<VEC, true>(prow, qrow, at, a.V, lane, before, level, sh.tok, sh.par, gone, stop)
                            : search_tile<VEC, false>(prow, nullptr, at, a.V, lane, before, level, sh.tok, sh.par, gone, stop);
        if (lane == 0) cluster.map_shared_rank(&sh, 0)->found = x;
      }
    }
    cluster.sync();  // found has arrived; the sums may be written again
    if (total != 0) next = 0;
  }
  if (rank == 0) {
    const int x = next < 0 ? -1 : sh.found;
    const bool fail = bad || x < 0;
    if (tid == 0) a.accepted[b] = fail ? -1 : count;
    // accepted nodes in order, then the next token, then -1
    if (tid <= a.max_nodes) {
      int node = -1;
      if (!fail && tid < count) {
        unsigned long long m = sh.okmask;
        for (int i = 0; i < tid; ++i) m &= m - 1;
        node = __ffsll(static_cast<long long>(m)) - 1;
      }
      a.out_tokens[static_cast<long long>(b) * (a.max_nodes + 1) + tid] = node >= 0 ? sh.tok[node] : (!fail && tid == count ? x : -1);
      if (tid < a.max_nodes) a.path[static_cast<long long>(b) * a.max_nodes + tid] = node;
    }
  }
}

}  // namespace
}  // namespace gbmoe

extern "C" moe_status_t moe_verify_draft(const float* target_probs, int64_t target_stride, const float* draft_probs,
                                         int64_t draft_stride, const int32_t* tokens, const int32_t* parents,
                                         const int32_t* node_offsets, const float* coins, const float* last_coins,
                                         int batch, int nodes, int vocab, int max_nodes, int32_t* out_tokens,
                                         int32_t* path, int32_t* accepted, moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_verify_draft", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_verify_draft: ") + m); };
    if (batch < 0 || nodes < 0 || vocab <= 0 || max_nodes < 0) return bad("sizes must be positive");
    if (max_nodes > MOE_MAX_TREE_NODES)
      return report_error(MOE_ERR_UNSUPPORTED, "moe_verify_draft: more than MOE_MAX_TREE_NODES nodes a sequence");
    if (vocab > kVTile * kVTiles || batch > (1 << 20))
      return report_error(MOE_ERR_UNSUPPORTED, "moe_verify_draft: problem too large");
    if (batch == 0) return MOE_OK;
    if (!target_probs || !node_offsets || !coins || !last_coins || !out_tokens || !accepted || (max_nodes && !path) ||
        (nodes && !tokens))
      return bad("NULL pointer");
    if (draft_probs && parents) return bad("draft probabilities are verified along a chain (no parents)");
    if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return bad("a row stride is shorter than its row");
    const VerifyArgs a{target_probs, draft_probs, target_stride, draft_stride, tokens, parents, node_offsets, coins,
                       last_coins, out_tokens, path, accepted, nodes, vocab, max_nodes};
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_verify_draft: no CUDA device");
    int C = 1;
    const int tiles = (vocab + kVTile - 1) / kVTile;
    while (C < kMaxCluster && 2 * C * batch <= 2 * sms && tiles > C * kVWarps / 2) C *= 2;
    // 16-byte loads where every row starts on 16 bytes
    const bool vec = vocab % 4 == 0 && target_stride % 4 == 0 && aligned(target_probs, 16) &&
                     (!draft_probs || (draft_stride % 4 == 0 && aligned(draft_probs, 16)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(batch) * C);
    cfg.blockDim = dim3(kVThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>((tiles + C - 1) / C) * 8;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched("moe_verify_draft", vec ? cudaLaunchKernelEx(&cfg, verify_kernel<true>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<false>, a));
  });
}
