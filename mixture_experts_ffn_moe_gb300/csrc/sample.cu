// Sampling with temperature, top-k, top-p and min-p from given random numbers, and the filtered probabilities.
//
// Mathematics.  w_x = 2^(-d_x), d_x = (max l - l_x) log2 e / T.  The tokens in order of their logits (ties: the lower index
// first) are cut three times: after the first top_k; of these after the shortest prefix whose weight is at least top_p of
// theirs; of these where w falls below min_p (the largest weight is 1).  All three leave a prefix of that order, so what is
// kept is known by its last token, the cut.  The sample is the first token x, in the order of indices, with
//   sum of kept w_i, i <= x  >  coin * sum of kept w_i.
//
// Arithmetic.  Weights are odd integers in units of 2^-44 (cut to even and one added: right on average), so their sums are
// exact, do not depend on the order of threads, and compare as integers with top_p and the coin.  d is a pair of floats;
// its fraction, less the nearest 64th, goes through the series of exp, whose value times 2^(-i/64) (a table) is formed in
// integers: a weight is off by 2^-28 of itself and a unit (fp32's exp: 2^-22, which at 100,000 tokens moves one coin in a few
// hundred across a border; FP64 runs at a sixtieth of the fp32 rate here).  Tokens with d >= 45 have no weight.
//
// Work split.  A cluster of CTAs shares a row.  One pass finds the largest logit, and every thread the largest of its own.
//   top_k: the top_k-th largest of the threads' largest bounds the top_k-th token from below, so the threads' largest alone are
//   counted in bins of d of 1/32 (32 tokens a thread: counting all of them took 7 us of 20 for a row of 129,280);
//   top_p: the next pass sums all weights and counts all tokens in such bins, whose tokens weigh the same within 2%.
// Either way the counts tell up to where the cut may lie.  As a rule at most 2048 tokens stand up to there: they are gathered in
// one CTA and decide everything, up to 256 by their order, more by exact weights of 1024 finer bins, of which only the one that
// holds a cut is put in order (ordering all took 9 to 36 us), and of runs of indices for the sample.  Where there are too
// many, the bins that may hold the cut alone are gathered and give it, beside the weights of those ahead (where even these are
// too many, bins of keys, and at equal keys of indices, split them first).
//
// Bound: the logits, read once; the later passes find them in L1 or L2.  In practice chains of latency for few rows (every
// pass ends in a cluster barrier) and the 59 instructions of a weight for many.  Measured, 129,280 words: one row with top_k 50
// and top_p 0.9 14.7 us, uncut 16; 64 rows, bf16, top_k 50 23 us, uncut 31, top_p 0.9 50 to 65, settings of their own 80.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "step_ops.cuh"

namespace gbmoe {
namespace {

namespace cg = cooperative_groups;

constexpr int kSThreads = 512;
constexpr int kSWarps = kSThreads / 32;
constexpr int kSCluster = 8;
constexpr int kSTile = 1024;            // tokens of a tile
constexpr int kSSlice = 65536;          // tokens of a CTA (a tile more where a row starts between 16-byte borders)
constexpr int kSVocab = 8 * 65536;
constexpr int kBins = 1440;             // of d in [0, 45): 32 a power of two
constexpr float kFar = 45.f;
constexpr int kList = 2048;             // tokens that are sorted at once
constexpr int kShort = 256;             // tokens whose order is found by counting
constexpr int kUnit = 44;               // weights count in units of 2^-44

// round(2^(30 - i / 64))
__device__ const int kExp2[64] = {
    1073741824, 1062175491, 1050733751, 1039415261, 1028218693, 1017142735, 1006186087, 995347464, 984625594,
    974019220, 963527098, 953147997, 942880699, 932724001, 922676710, 912737649, 902905651, 893179563,
    883558244, 874040567, 864625413, 855311680, 846098274, 836984114, 827968132, 819049271, 810226483,
    801498734, 792865000, 784324269, 775875538, 767517817, 759250125, 751071493, 742980960, 734977579,
    727060411, 719228525, 711481005, 703816941, 696235434, 688735596, 681316545, 673977412, 666717336,
    659535466, 652430958, 645402981, 638450708, 631573326, 624770026, 618040012, 611382493, 604796689,
    598281827, 591837143, 585461881, 579155293, 572916640, 566745190, 560640218, 554601009, 548626854,
    542717053};

struct SampleArgs {
  const void* logits;
  long long ld;
  const float* temperature;  // [rows] each, or null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* coins;
  int32_t* tokens;  // null: probabilities only
  float* probs;     // null: tokens only
  long long probs_ld;
  int V;
};

// u * 2^64 (rounded down) for u in [0, 1); what lies outside is brought to the nearest end (NaN to 0).
__device__ __forceinline__ uint64_t unit_fraction(float u) {
  const uint32_t b = __float_as_uint(fminf(u > 0.f ? u : 0.f, 0x1.fffffep-1f));
  const int e = static_cast<int>(b >> 23) - 86;  // u = m * 2^(e - 64)
  const uint64_t m = e <= -86 ? 0 : (b & 0x7fffffu) | 0x800000u;
  return e >= 0 ? m << e : (e < -63 ? 0 : m >> -e);
}
// The share u of `total`, rounded up.
__device__ __forceinline__ uint64_t share_of(float u, uint64_t total) {
  const uint64_t f = unit_fraction(u);
  return __umul64hi(f, total) + (f * total != 0 ? 1 : 0);
}

// Order-preserving keys of floats; -0 counts as 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) { return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xffffffffu)); }
// Tokens in the order of the cuts have descending ranks.
__device__ __forceinline__ uint64_t rank_of(float l, int i) { return static_cast<uint64_t>(key_of(l)) << 32 | (0xffffffffu - static_cast<uint32_t>(i)); }

// Two floats in one register pair: GB300's fp32 units take two at once.
struct F2 { uint64_t v; };
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

struct Weigher {
  float top, hi, lo;  // the largest logit; log2 e / T as a pair
  const int* table;

  __device__ __forceinline__ float distance(float l) const { return (l == top ? 0.f : top - l) * hi; }
  // The weights of two logits (0 for NaN and what is too far away), and their distances.
  __device__ __forceinline__ void weights(float l0, float l1, uint64_t& w0, uint64_t& w1, float& p0, float& p1) const {
    if (top == INFINITY) {  // infinite logits share the row
      p0 = distance(l0);
      p1 = distance(l1);
      w0 = l0 == top ? 1ull << kUnit | 1 : 0;
      w1 = l1 == top ? 1ull << kUnit | 1 : 0;
      return;
    }
    const F2 t = f2(top), l = f2(l0, l1), one = f2(-1.f);
    const F2 s = fma2(l, one, t);                                        // top - l = s + e
    const F2 b = s + f2(-top);
    const F2 e = fma2(l + b, one, fma2(fma2(b, one, s), one, t));
    const F2 q = s * f2(-hi);                                            // -p
    const F2 tail = fma2(s, f2(lo), fma2(e, f2(hi), fma2(s, f2(hi), q)));  // d = p + tail
    const F2 n = fma2(q, f2(-64.f), f2(12582912.f));                     // 64 p to the nearest integer, above 1.5 * 2^23
    const F2 r = fma2(n + f2(-12582912.f), f2(0.015625f), q);            // exact: -(p - 64ths)
    const F2 z = fma2(tail, one, r) * f2(0x1.62e43p-1f);                 // 2^(r - tail) = exp(z), |z| below 2^-7.5
    const float2 v = parts(fma2(z * z, fma2(z, f2(1.f / 6.f), f2(0.5f)), z) * f2(0x1p32f));  // (exp(z) - 1) * 2^32
    const float2 pp = parts(q), nn = parts(n);
    p0 = -pp.x;
    p1 = -pp.y;
    w0 = p0 < kFar ? scaled(v.x, __float_as_uint(nn.x)) : 0;
    w1 = p1 < kFar ? scaled(v.y, __float_as_uint(nn.y)) : 0;
  }
  __device__ __forceinline__ void weights(float l0, float l1, uint64_t& w0, uint64_t& w1) const {
    float p0, p1;
    weights(l0, l1, w0, w1, p0, p1);
  }
  __device__ __forceinline__ uint64_t scaled(float v, uint32_t n) const {  // 2^-(n / 64) * (1 + v / 2^32)
    const int t = table[n & 63];
    const int m = t + static_cast<int>((static_cast<int64_t>(t) * __float2int_rn(v) + 0x80000000ll) >> 32);
    return (static_cast<uint64_t>(static_cast<uint32_t>(m)) << 14) >> ((n >> 6) & 63) | 1;
  }
  __device__ __forceinline__ uint64_t weight(float l) const {
    uint64_t a, b;
    weights(l, l, a, b);
    return a;
  }
};

// What the leader finds out and tells the cluster.
struct Decision {
  int found;               // the range below holds the cut
  uint32_t bin0, bin1;     // the bins of d that (as good as surely) hold the cut
  uint32_t last;           // the first bin up to which it lies for certain, and
  uint32_t klo, khi;       // keys of the range, and its indices (bins of keys and indices)
  uint32_t ilo, ihi;
  uint32_t count;          // tokens up to `last`, or of the range
  uint32_t before;         // tokens ahead of it, and their weight (bins with exact weights)
  uint64_t before_w;
  uint64_t total, need;    // weight of all that is left, and what the kept prefix has to reach
  uint64_t cut;            // rank of the last kept token
};

struct SShared {
  float best[kSCluster];
  uint32_t best_at[kSCluster];
  uint64_t sums[kSCluster];
  uint32_t counts[kSCluster];
  float wait[kSWarps][96];  // logits of tokens that wait to be weighed
  uint64_t warp[kSWarps];
  uint32_t warp_n[kSWarps];
  Decision dec;
  uint32_t listed[8];      // tokens of every list that is gathered, one after the other
  uint32_t mine, base;     // of this CTA's share: tokens, and its place in the leader's list
  uint32_t border_n;       // the leader's bin that holds a cut, and its tokens
  int border_bin;
  uint32_t border_before;
  uint64_t border_before_w;
  uint64_t border[kShort], border_w[kShort];
  int table[64];
};

// Dynamic shared memory: region A, the bins of this CTA (counts and three 15-bit pieces of weights) or the sorted list; region
// B, the cluster's bins at the leader (weights, counts) or the list's weights; then the sums of this CTA's tiles.
constexpr int kRegionA = kBins * 16, kRegionB = kBins * 12;
static_assert(kRegionA >= kList * 8 && kRegionB >= kList * 8, "the list fits");

// A row of V logits.  Its tokens stand at places: token i at place i + off, so that places that are multiples of N start on 16
// bytes.
template <typename T>
struct Row {
  static constexpr int N = 16 / sizeof(T);
  const T* p;
  int V, off;
  __device__ __forceinline__ float at(int i) const {
    if constexpr (std::is_same<T, float>::value) return __ldg(p + i);
    else return Elem<T>::to_float(p[i]);
  }
  __device__ __forceinline__ uint4 load(int place) const {  // -infinity outside the row
    const int i = place - off;
    if (i >= 0 && i + N <= V) return __ldg(reinterpret_cast<const uint4*>(p + i));
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (std::is_same<T, float>::value) {
        w[j] = i + j >= 0 && i + j < V ? __float_as_uint(__ldg(p + i + j)) : 0xff800000u;
      } else {
        const float a = i + 2 * j >= 0 && i + 2 * j < V ? at(i + 2 * j) : -INFINITY;
        const float b = i + 2 * j + 1 >= 0 && i + 2 * j + 1 < V ? at(i + 2 * j + 1) : -INFINITY;
        w[j] = Elem<T>::pack(a, b);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void widen(const uint4& v, float (&x)[N]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (std::is_same<T, float>::value) {
        x[j] = __uint_as_float(w[j]);
      } else {
        const float2 f = Elem<T>::unpack(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
  }
  // f(N logits, index of the first) for this thread's share of the places [lo, hi), in ascending order, U loads under way.
  template <int U, typename F>
  __device__ __forceinline__ void each(int lo, int hi, int first, int stride, F&& f) const {
#pragma unroll 1
    for (int q = lo + first * N; q < hi; q += U * stride * N) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (q + u * stride * N < hi) v[u] = load(q + u * stride * N);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (q + u * stride * N < hi) {
          float x[N];
          widen(v[u], x);
          f(x, q + u * stride * N - off);
        }
    }
  }
};

// Inclusive sums over the block of a count and a weight; the totals in *n_all, *w_all.
__device__ __forceinline__ void block_scan(uint32_t& n, uint64_t& w, SShared& sh, uint32_t* n_all, uint64_t* w_all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t un = __shfl_up_sync(0xffffffffu, n, o);
    const uint64_t uw = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) { n += un; w += uw; }
  }
  __syncthreads();
  if (lane == 31) { sh.warp[warp] = w; sh.warp_n[warp] = n; }
  __syncthreads();
  uint32_t all_n = 0;
  uint64_t all_w = 0;
#pragma unroll
  for (int i = 0; i < kSWarps; ++i) {
    if (i == warp) { n += all_n; w += all_w; }
    all_n += sh.warp_n[i];
    all_w += sh.warp[i];
  }
  *n_all = all_n;
  *w_all = all_w;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

static_assert(kList == 2 * 2 * 32 * kSWarps, "two pairs a thread");
// Sorts list[0, n) in descending order (all values differ); list has room for the next power of two.
__device__ __forceinline__ void block_sort(uint64_t* list, int n) {
  if (n <= kShort) {  // a value's place is the number of larger ones
    uint64_t x = 0;
    int place = 0;
    if (threadIdx.x < n) {
      x = list[threadIdx.x];
#pragma unroll 8
      for (int i = 0; i < n; ++i) place += list[i] > x;
    }
    __syncthreads();
    if (threadIdx.x < n) list[place] = x;
    __syncthreads();
    return;
  }
  int size = 2 * kShort;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += kSThreads) list[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int k = 2; k <= size; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      // a warp's 64 pairs are 128 neighbouring values where j is at most 64: there it waits for nobody else
      if (j >= 64) __syncthreads(); else __syncwarp();
#pragma unroll
      for (int h = 0; h < kList / 2 / kSThreads; ++h) {
        const int i = (threadIdx.x >> 5) * 64 + h * 32 + (threadIdx.x & 31);
        if (i >= size / 2) break;
        const int a = ((i & ~(j - 1)) << 1) | (i & (j - 1)), b = a + j;
        const uint64_t x = list[a], y = list[b];
        if ((x < y) == ((a & k) == 0)) { list[a] = y; list[b] = x; }
      }
    }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Row<T>::N;
  __shared__ SShared sh;
  extern __shared__ __align__(16) unsigned char dyn[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank(), row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* bins = reinterpret_cast<uint32_t*>(dyn);                                // [4][kBins]
  uint64_t* list = reinterpret_cast<uint64_t*>(dyn);                                // [kList]
  uint64_t* bin_w = reinterpret_cast<uint64_t*>(dyn + kRegionA);                    // [kBins]
  uint32_t* bin_n = reinterpret_cast<uint32_t*>(dyn + kRegionA + kBins * 8);        // [kBins]
  uint64_t* list_w = bin_w;                                                         // [kList]
  uint64_t* tile_sum = reinterpret_cast<uint64_t*>(dyn + kRegionA + kRegionB);      // [tiles of this CTA]
  pdl_trigger();
  if (tid < 64) sh.table[tid] = kExp2[tid];
  if (tid < 8) sh.listed[tid] = 0;
  if (tid == 0) sh.mine = 0;
  int lists = 0;  // gathered so far
  auto clear = [&] {
    for (int i = tid; i < kBins * 4; i += kSThreads) bins[i] = 0;
    if (rank == 0)
      for (int i = tid; i < kBins; i += kSThreads) { bin_w[i] = 0; bin_n[i] = 0; }
  };
  clear();
  // Another CTA's shared memory may be written only once that CTA is known to run and has cleared it: all have arrived here.
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  pdl_wait();
  Row<T> logits;
  logits.p = static_cast<const T*>(a.logits) + row * a.ld;
  logits.V = a.V;
  logits.off = static_cast<int>(reinterpret_cast<uintptr_t>(logits.p) / sizeof(T) % N);
  const int tiles = (a.V + logits.off + kSTile - 1) / kSTile, per = (tiles + C - 1) / C;
  const int tile0 = min(tiles, rank * per), my_tiles = min(tiles, tile0 + per) - tile0;
  const int lo = tile0 * kSTile, hi = min((a.V + logits.off + N - 1) / N * N, (tile0 + my_tiles) * kSTile);  // places
  const float temperature = a.temperature ? a.temperature[row] : 1.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const float coin = a.coins ? a.coins[row] : 0.f;
  float* probs = a.probs ? a.probs + row * a.probs_ld : nullptr;
  const bool wide_probs = probs && (reinterpret_cast<uintptr_t>(probs) / 4 + 4 - logits.off % 4) % 4 == 0;

  // ---- the largest logit
  float top = -INFINITY;
  logits.template each<4>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int) {
#pragma unroll
    for (int j = 0; j < N; ++j) top = fmaxf(top, x[j]);  // (NaN is passed over)
  });
  const float own_top = top;
  top = warp_max(top);
  if (lane == 0) sh.warp_n[warp] = __float_as_uint(top);
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (tid < C) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) m = fmaxf(m, __uint_as_float(sh.warp_n[w]));
    cluster.map_shared_rank(&sh, tid)->best[rank] = m;
  }
  cluster.sync();
  top = -INFINITY;
  for (int r = 0; r < C; ++r) top = fmaxf(top, sh.best[r]);
  // This CTA's part of the probabilities: f(two logits, index of the first, two results)
  auto fill = [&](auto&& f) {
    logits.template each<1>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i) {
      float y[N];
#pragma unroll
      for (int j = 0; j < N; j += 2) f(x[j], x[j + 1], i + j, y[j], y[j + 1]);
      if (wide_probs && i >= 0 && i + N <= a.V) {
#pragma unroll
        for (int j = 0; j < N; j += 4) *reinterpret_cast<float4*>(probs + i + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (i + j >= 0 && i + j < a.V) probs[i + j] = y[j];
      }
    });
  };
  if (top == -INFINITY || !(temperature > 0.f)) {  // nothing to choose from, or the best token
    uint32_t at = 0xffffffffu;
    if (top > -INFINITY)
      logits.template each<2>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i) {
#pragma unroll
        for (int j = N - 1; j >= 0; --j)
          if (x[j] == top) at = min(at, static_cast<uint32_t>(i + j));
      });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) sh.warp_n[warp] = at;
    __syncthreads();
    if (tid < C) {
      for (int w = 0; w < kSWarps; ++w) at = min(w ? at : 0xffffffffu, sh.warp_n[w]);
      cluster.map_shared_rank(&sh, tid)->best_at[rank] = at;
    }
    cluster.sync();
    at = 0xffffffffu;
    for (int r = 0; r < C; ++r) at = min(at, sh.best_at[r]);
    if (rank == 0 && tid == 0 && a.tokens) a.tokens[row] = static_cast<int>(at);  // (-1 where there is none)
    if (probs)
      fill([&](float, float, int i, float& y0, float& y1) {
        y0 = static_cast<uint32_t>(i) == at ? 1.f : 0.f;
        y1 = static_cast<uint32_t>(i + 1) == at ? 1.f : 0.f;
      });
    return;
  }
  const double rate = fmin(1.4426950408889634074 / static_cast<double>(temperature), 3.0e38);
  Weigher wt;
  wt.top = top;
  wt.hi = static_cast<float>(rate);
  wt.lo = static_cast<float>(rate - static_cast<double>(wt.hi));
  wt.table = sh.table;
  uint64_t least = 0;  // min_p, rounded up
  const bool only_top = min_p >= 1.f;  // the tokens of the largest logit alone: weights do not tell them from those within 2^-28
  if (only_top) least = 1ull << kUnit;
  else if (min_p > 0.f) least = (unit_fraction(min_p) + ((1ull << (64 - kUnit)) - 1)) >> (64 - kUnit);
  const bool by_count = top_k > 0 && top_k < a.V, by_share = top_p < 1.f;

  // The cut as a logit and an index: kept are larger logits, and equal ones up to the index.
  uint64_t cut = 0;
  float cut_l = -INFINITY;
  int cut_i = a.V;
  auto set_cut = [&](uint64_t c) {
    cut = c;
    cut_l = float_of(static_cast<uint32_t>(c >> 32));
    cut_i = static_cast<int>(0xffffffffu - static_cast<uint32_t>(c));
  };
  auto kept = [&](float l, int i) { return l > cut_l || (l == cut_l && i <= cut_i); };
  auto bin_of = [&](float l) {  // kBins: no weight
    const float p = wt.distance(l);
    return p < kFar ? static_cast<uint32_t>(p * 32.f) : static_cast<uint32_t>(kBins);
  };

  // ---- counts in bins of the distance, over the cluster, in the leader's bin_n
  auto push_bins = [&] {
    __syncthreads();
    uint32_t* to = cluster.map_shared_rank(bin_n, 0);
    for (int b = tid; b < kBins; b += kSThreads)
      if (bins[b]) atomicAdd(to + b, bins[b]);
  };
  // of every thread's largest logit
  auto count_largest = [&] {
    const uint32_t b = bin_of(own_top);
    if (b < kBins) atomicAdd(&bins[b], 1u);
    push_bins();
    cluster.sync();
  };
  // of the kept tokens
  auto count_all = [&] {
    logits.template each<4>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t b = bin_of(x[j]);
        if (b < kBins && kept(x[j], i + j)) atomicAdd(&bins[b], 1u);
      }
    });
    push_bins();
    cluster.sync();
  };
  // of the kept tokens, and the sums of their weights in the leader's sums
  auto count_and_sum = [&] {
    uint64_t mine = 0;
    logits.template each<2>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i) {
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        uint64_t w[2];
        float p[2];
        wt.weights(x[j], x[j + 1], w[0], w[1], p[0], p[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (p[c] < kFar && (cut == 0 || kept(x[j + c], i + j + c))) {
            mine += w[c];
            atomicAdd(&bins[static_cast<uint32_t>(p[c] * 32.f)], 1u);
          }
      }
    });
    mine = warp_sum(mine);
    if (lane == 0) sh.warp[warp] = mine;
    push_bins();
    if (tid == 0) {
      uint64_t all = 0;
      for (int w = 0; w < kSWarps; ++w) all += sh.warp[w];
      cluster.map_shared_rank(&sh, 0)->sums[rank] = all;
    }
    cluster.sync();
  };
  auto tell = [&] {  // the leader's decision to all
    __syncthreads();
    if (tid > 0 && tid < C) cluster.map_shared_rank(&sh, tid)->dec = sh.dec;
  };
  // The leader: the bins that may hold the cut.  A token of bin b weighs between 2^-((b + 1) / 32) and 2^-(b / 32): with the
  // lower bound the cut lies at the latest in the first bin where the running weight reaches `need`.  With the mean of tokens that
  // lie evenly in their bins, brought to the known total, it lies within 2^-9 of where the running weight says so; that is
  // looked at afterwards.  By count the bin is known.
  auto choose_bins = [&](bool share) {
    if (rank == 0) {
      constexpr int Q = (kBins + kSThreads - 1) / kSThreads;
      uint64_t total = 0, need = 0;
      if (share) {
        for (int r = 0; r < C; ++r) total += sh.sums[r];
        need = share_of(top_p, total);
        if (need == 0) need = 1;  // (the first token stays)
      }
      uint32_t n[Q], run_n = 0, none = 0;
      uint64_t lower[Q], about[Q], run_lo = 0, run_ab = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int b = tid * Q + q;
        n[q] = b < kBins ? bin_n[b] : 0;
        run_n += n[q];
        lower[q] = about[q] = 0;
        if (share && n[q]) {  // (a token's bin goes by d to 2^-17)
          const float e = exp2f(static_cast<float>(kUnit) - static_cast<float>(b) * 0.03125f);
          about[q] = static_cast<uint64_t>(n[q]) * (static_cast<uint64_t>(e * 0.989247f) + 1);                              // (1 - 2^(-1/32)) * 32 / ln 2
          lower[q] = static_cast<uint64_t>(n[q]) * static_cast<uint64_t>(e * (0x1.f50764p-1f * (1.f - 0x1p-16f)));  // 2^(-1/32)
          run_lo += lower[q];
          run_ab += about[q];
        }
      }
      uint32_t own_n = run_n, all_n;
      uint64_t own_lo = run_lo, own_ab = run_ab, all_lo, all_ab = 1;
      block_scan(run_n, run_lo, sh, &all_n, &all_lo);
      if (share) block_scan(none, run_ab, sh, &none, &all_ab);
      run_n -= own_n;
      run_lo -= own_lo;
      run_ab -= own_ab;
      const float ratio = __ull2float_rn(total) / __ull2float_rn(all_ab), goal = __ull2float_rn(need);
      if (tid == 0) {
        sh.dec.found = share || static_cast<uint32_t>(top_k) <= all_n;
        sh.dec.total = total;
        sh.dec.need = need;
        sh.dec.bin0 = 0;
        sh.dec.bin1 = sh.dec.last = kBins - 1;
        sh.dec.before = 0;
        sh.dec.count = all_n;
        sh.dec.ilo = 0;
        sh.dec.ihi = static_cast<uint32_t>(a.V - 1);
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint32_t b = tid * Q + q;
        const uint32_t to_n = run_n + n[q];
        const uint64_t to_lo = run_lo + lower[q], to_ab = run_ab + about[q];
        if (b < kBins && n[q]) {
          if (share) {
            const float from = __ull2float_rn(run_ab) * ratio, to = __ull2float_rn(to_ab) * ratio;
            if (from * (1.f + 0x1p-9f) < goal && to * (1.f + 0x1p-9f) >= goal) sh.dec.bin0 = b;
            if (from * (1.f - 0x1p-9f) < goal && to * (1.f - 0x1p-9f) >= goal) sh.dec.bin1 = b;
            if (run_lo < need && to_lo >= need) { sh.dec.last = b; sh.dec.count = to_n; }
          } else if (run_n < static_cast<uint32_t>(top_k) && to_n >= static_cast<uint32_t>(top_k)) {
            sh.dec.bin0 = sh.dec.bin1 = sh.dec.last = b;
            sh.dec.before = run_n;
            sh.dec.count = to_n;
          }
        }
        run_n = to_n;
        run_lo = to_lo;
        run_ab = to_ab;
      }
      tell();
    }
    cluster.sync();
    return sh.dec;
  };
  // A logit at or below those of bins up to b, and one above those of bins from b on.
  auto below_bin = [&](uint32_t b) { return b + 1 >= kBins || wt.hi == 0.f || top == INFINITY ? -INFINITY : top - ((b + 1) * 0.03125f * (1.f + 0x1p-18f)) / wt.hi - fabsf(top) * 0x1p-22f; };
  auto above_bin = [&](uint32_t b) { return b == 0 || top == INFINITY || wt.hi == 0.f ? INFINITY : top - (b * 0.03125f * (1.f - 0x1p-18f)) / wt.hi + fabsf(top) * 0x1p-22f; };
  // A CTA's tokens of a list go to a list of its own first (in region B, free by then), since thousands of additions to one
  // counter of another CTA take longer than all else.
  auto take = [&](float l, int i) {
    const uint32_t place = atomicAdd(&sh.mine, 1u);
    if (place < kList) bin_w[place] = rank_of(l, i);
  };
  auto deliver = [&] {  // to the leader's; true where there was room for all
    uint32_t* at = &cluster.map_shared_rank(&sh, 0)->listed[lists++];
    __syncthreads();
    if (tid == 0) sh.base = atomicAdd(at, sh.mine);
    __syncthreads();
    const uint32_t n = min(sh.mine, static_cast<uint32_t>(kList)), base = sh.base;
    uint64_t* to = cluster.map_shared_rank(list, 0);
    for (uint32_t i = tid; i < n; i += kSThreads)
      if (base + i < kList) to[base + i] = bin_w[i];
    __syncthreads();
    if (tid == 0) sh.mine = 0;
    cluster.sync();
    return *at <= kList;
  };
  // Kept tokens of at least `least_l` to the leader's list.
  auto gather = [&](float least_l) {
    logits.template each<4>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (x[j] >= least_l && x[j] > -INFINITY && kept(x[j], i + j)) take(x[j], i + j);
    });
    return deliver();
  };
  // The same for those not above `ahead_l`; of the others the number and the sum of the weights (and that of every tile) in the
  // leader's counts and sums.  A warp's tokens ahead wait until there are two a lane: as a rule they are few among the others.
  auto gather_between = [&](float least_l, float ahead_l, bool weigh) {
    uint64_t mine = 0;
    uint32_t ahead_n = 0;
    float* wait = sh.wait[warp];
    for (int t = warp; t < my_tiles; t += kSWarps) {
      uint64_t sum = 0;
      int waiting = 0;
      auto weigh_two = [&](float l0, float l1) {
        uint64_t w0, w1;
        wt.weights(l0, l1, w0, w1);
        sum += w0 + w1;
      };
#pragma unroll 1
      for (int r = 0; r < kSTile / 32 / N; ++r) {
        const int place = lo + t * kSTile + (r * 32 + lane) * N, i = place - logits.off;
        float x[N];
        Row<T>::widen(logits.load(place), x);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t ahead = __ballot_sync(0xffffffffu, x[j] > ahead_l);
          if (ahead) {
            ahead_n += __popc(ahead);
            if (weigh) {
              if (x[j] > ahead_l) wait[waiting + __popc(ahead & ((1u << lane) - 1))] = x[j];
              waiting += __popc(ahead);
              if (waiting >= 64) {
                __syncwarp();
                waiting -= 64;
                weigh_two(wait[waiting + lane], wait[waiting + 32 + lane]);
                __syncwarp();
              }
            }
          }
          if (!(x[j] > ahead_l) && x[j] >= least_l && x[j] > -INFINITY && kept(x[j], i + j)) take(x[j], i + j);
        }
      }
      if (waiting) {
        __syncwarp();
        weigh_two(lane < waiting ? wait[lane] : -INFINITY, 32 + lane < waiting ? wait[32 + lane] : -INFINITY);
        __syncwarp();
      }
      sum = warp_sum(sum);
      if (lane == 0) tile_sum[t] = sum;
      mine += sum;
    }
    if (lane == 0) { sh.warp[warp] = mine; sh.warp_n[warp] = ahead_n; }
    __syncthreads();
    if (tid == 0) {
      uint64_t all = 0;
      uint32_t all_n = 0;
      for (int w = 0; w < kSWarps; ++w) { all += sh.warp[w]; all_n += sh.warp_n[w]; }
      cluster.map_shared_rank(&sh, 0)->sums[rank] = all;
      cluster.map_shared_rank(&sh, 0)->counts[rank] = all_n;
    }
    return deliver();
  };

  // ---- where a few bins of the distance hold too many tokens: bins with exact weights, of the distance (first), of keys, or of
  // indices where all keys are the same
  auto bin_shift = [&](uint32_t span) {  // span >> shift < kBins
    int s = 0;
    while ((span >> s) >= kBins) ++s;
    return s;
  };
  auto exact_bins = [&](bool first, const Decision& d) {
    const bool ties = d.klo == d.khi;
    const int shift = first ? 0 : bin_shift(ties ? d.ihi - d.ilo : d.khi - d.klo);
    clear();
    cluster.sync();
    logits.template each<1>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i0) {
#pragma unroll 1
      for (int j = 0; j < N; ++j) {
        float l = x[0];
#pragma unroll
        for (int c = 1; c < N; ++c) l = j == c ? x[c] : l;
        const uint32_t i = static_cast<uint32_t>(i0 + j);
        uint32_t bin = bin_of(l);
        if (bin >= kBins || !kept(l, i0 + j)) continue;
        if (!first) {
          const uint32_t k = key_of(l);
          if (k < d.klo || k > d.khi || i < d.ilo || i > d.ihi) continue;
          bin = (ties ? i - d.ilo : d.khi - k) >> shift;
        }
        const uint64_t w = wt.weight(l);
        // (w is at most 2^44 + 1, and 65 tiles at most: no piece of 15 bits overflows its sum)
        atomicAdd(&bins[bin], 1u);
        atomicAdd(&bins[kBins + bin], static_cast<uint32_t>(w) & 0x7fffu);
        atomicAdd(&bins[2 * kBins + bin], static_cast<uint32_t>(w >> 15) & 0x7fffu);
        atomicAdd(&bins[3 * kBins + bin], static_cast<uint32_t>(w >> 30));
      }
    });
    __syncthreads();
    unsigned long long* to_w = reinterpret_cast<unsigned long long*>(cluster.map_shared_rank(bin_w, 0));
    uint32_t* to_n = cluster.map_shared_rank(bin_n, 0);
    for (int b = tid; b < kBins; b += kSThreads)
      if (bins[b]) {
        atomicAdd(to_n + b, bins[b]);
        atomicAdd(to_w + b, static_cast<uint64_t>(bins[kBins + b]) + (static_cast<uint64_t>(bins[2 * kBins + b]) << 15) +
                                (static_cast<uint64_t>(bins[3 * kBins + b]) << 30));
      }
    cluster.sync();
  };
  // The leader: the first of these bins in which the running count reaches top_k, or the running weight d.need.
  auto choose_exact = [&](bool first, bool share, const Decision& d) {
    if (rank == 0) {
      constexpr int Q = (kBins + kSThreads - 1) / kSThreads;
      uint32_t n = 0;
      uint64_t w = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int b = tid * Q + q;
        if (b < kBins) { n += bin_n[b]; w += bin_w[b]; }
      }
      uint32_t all_n, own_n = n;
      uint64_t all_w, own_w = w;
      block_scan(n, w, sh, &all_n, &all_w);
      n += (first ? 0 : d.before) - own_n;
      w += (first ? 0 : d.before_w) - own_w;  // ahead of this thread's bins
      const bool ties = d.klo == d.khi;
      const int shift = first ? 0 : bin_shift(ties ? d.ihi - d.ilo : d.khi - d.klo);
      if (tid == 0) { sh.dec.total = d.total; sh.dec.need = d.need; }
#pragma unroll 1
      for (int q = 0; q < Q; ++q) {
        const int b = tid * Q + q;
        if (b >= kBins) break;
        const uint32_t bn = bin_n[b];
        const uint64_t bw = bin_w[b];
        if (share ? w < d.need && w + bw >= d.need : n < static_cast<uint32_t>(top_k) && n + bn >= static_cast<uint32_t>(top_k)) {
          Decision& o = sh.dec;
          o.count = bn;
          o.before = n;
          o.before_w = w;
          o.ilo = d.ilo;
          o.ihi = d.ihi;
          o.klo = d.klo;
          o.khi = d.khi;
          if (first) {  // the keys of the bin: bins ascend as keys fall
            uint32_t x = key_of(-INFINITY), y = key_of(top);
            while (x < y) {  // the largest key with a bin of b or more
              const uint32_t mid = x + (y - x + 1) / 2;
              if (bin_of(float_of(mid)) >= static_cast<uint32_t>(b)) x = mid; else y = mid - 1;
            }
            o.khi = x;
            x = key_of(-INFINITY);
            y = key_of(top);
            while (x < y) {  // the smallest key with a bin of b or less
              const uint32_t mid = x + (y - x) / 2;
              if (bin_of(float_of(mid)) <= static_cast<uint32_t>(b)) y = mid; else x = mid + 1;
            }
            o.klo = y;
          } else if (ties) {
            o.ilo = d.ilo + (static_cast<uint32_t>(b) << shift);
            o.ihi = min(d.ihi, o.ilo + (1u << shift) - 1);
          } else {
            o.khi = d.khi - (static_cast<uint32_t>(b) << shift);
            o.klo = max(d.klo, o.khi - ((1u << shift) - 1));
          }
        }
        n += bn;
        w += bw;
      }
      tell();
    }
    cluster.sync();
    return sh.dec;
  };
  auto gather_range = [&](const Decision& d) {
    logits.template each<1>(lo, hi, tid, kSThreads, [&](const float (&x)[N], int i) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t k = key_of(x[j]), at_i = static_cast<uint32_t>(i + j);
        if (k >= d.klo && k <= d.khi && at_i >= d.ilo && at_i <= d.ihi && kept(x[j], i + j)) take(x[j], i + j);
      }
    });
    deliver();
  };

  // ---- the leader's list
  constexpr int L = kList / kSThreads;
  auto logit_at = [&](int i) { return float_of(static_cast<uint32_t>(list[i] >> 32)); };
  auto weight_at = [&](int i) { return wt.weight(logit_at(i)); };
  // The list in order; the number of its tokens.
  auto sorted = [&] {
    const int n = min(sh.listed[lists - 1], static_cast<uint32_t>(kList));
    __syncthreads();
    block_sort(list, n);
    return n;
  };
  // The same cut of a list of many, without its order: exact bins of the list's distances in region B, and of the bin that holds
  // the cut every token's place.  `found` is the cut's rank; false where the bin has too many tokens.
  constexpr int kFine = 1024;  // bins: kFine * 16 bytes
  static_assert(kFine * 16 <= kRegionB && kFine == 2 * kSThreads, "two bins a thread");
  uint32_t* fine = reinterpret_cast<uint32_t*>(bin_w);  // [4][kFine]: counts, three pieces of weights
  auto put_weight = [&](uint32_t* at, int stride, uint64_t w) {  // (pieces of 15 bits, at most 2048 of them)
    atomicAdd(at, static_cast<uint32_t>(w) & 0x7fffu);
    atomicAdd(at + stride, static_cast<uint32_t>(w >> 15) & 0x7fffu);
    atomicAdd(at + 2 * stride, static_cast<uint32_t>(w >> 30));
  };
  auto weight_of = [&](const uint32_t* at, int stride) {
    return static_cast<uint64_t>(at[0]) + (static_cast<uint64_t>(at[stride]) << 15) + (static_cast<uint64_t>(at[2 * stride]) << 30);
  };
  // w[i]: weight of this thread's tokens tid + i * kSThreads, 0 for those that are out of it.  share_all: `need` is top_p of
  // their weight.
  auto border_cut = [&](int n, const uint64_t (&w)[L], bool share, bool share_all, uint32_t before, uint64_t before_w, uint64_t need,
                        float scale, float offset, uint64_t& found) {
    auto fine_of = [&](int x) {
      const float d = wt.distance(float_of(static_cast<uint32_t>(list[x] >> 32)));
      return min(kFine - 1, max(0, static_cast<int>((d - offset) * scale)));
    };
    __syncthreads();
    for (int i = tid; i < 4 * kFine; i += kSThreads) fine[i] = 0;
    if (tid == 0) { sh.border_n = 0; sh.border_bin = -1; }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (tid + i * kSThreads < n && w[i]) {
        const int b = fine_of(tid + i * kSThreads);
        atomicAdd(fine + b, 1u);
        if (share) put_weight(fine + kFine + b, kFine, w[i]);
      }
    __syncthreads();
    uint32_t c[2], run_n = 0, none;
    uint64_t s[2], run_w = 0, all;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = fine[2 * tid + i];
      s[i] = weight_of(fine + kFine + 2 * tid + i, kFine);
      run_n += c[i];
      run_w += s[i];
    }
    uint32_t at_n = before - run_n;
    uint64_t at_w = before_w - run_w;
    block_scan(run_n, run_w, sh, &none, &all);
    at_n += run_n;
    at_w += run_w;
    if (share_all) need = share_of(top_p, all);
    if (need == 0) need = 1;  // (the first token stays)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (share ? at_w < need && at_w + s[i] >= need : at_n < static_cast<uint32_t>(top_k) && at_n + c[i] >= static_cast<uint32_t>(top_k)) {
        sh.border_bin = 2 * tid + i;
        sh.border_before = at_n;
        sh.border_before_w = at_w;
      }
      at_n += c[i];
      at_w += s[i];
    }
    __syncthreads();
    const int bin = sh.border_bin;
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (tid + i * kSThreads < n && w[i] && fine_of(tid + i * kSThreads) == bin) {
        const uint32_t place = atomicAdd(&sh.border_n, 1u);
        if (place < kShort) {
          sh.border[place] = list[tid + i * kSThreads];
          sh.border_w[place] = w[i];
        }
      }
    __syncthreads();
    const int m = static_cast<int>(sh.border_n);
    if (bin < 0 || m > kShort) return false;
    if (tid < m) {
      const uint64_t own = sh.border[tid];
      uint32_t place = sh.border_before + 1;
      uint64_t ahead = sh.border_before_w;
#pragma unroll 4
      for (int i = 0; i < m; ++i) {
        const bool larger = sh.border[i] > own;
        place += larger;
        ahead += larger ? sh.border_w[i] : 0;
      }
      if (share ? ahead < need && ahead + sh.border_w[tid] >= need : place == static_cast<uint32_t>(top_k)) sh.dec.cut = own;
    }
    __syncthreads();
    found = sh.dec.cut;
    return true;
  };

  // Everything from a list that holds all that the first filter keeps (and more); its distances are below `far`.
  auto finish_from_list = [&](bool count_first, uint64_t need, float far) {
    int n = min(sh.listed[lists - 1], static_cast<uint32_t>(kList));
    uint64_t w[L], run = 0, all, unused = 0, total = 0;
    uint32_t one = 0, none;
    bool ordered = n <= kShort;
    if (!ordered) {
#pragma unroll
      for (int i = 0; i < L; ++i) w[i] = tid + i * kSThreads < n ? weight_at(tid + i * kSThreads) : 0;
      const float scale = kFine / far;
      uint64_t last = 0;
      auto drop = [&] {
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (tid + i * kSThreads < n && list[tid + i * kSThreads] < last) w[i] = 0;
      };
      if (count_first) {
        ordered = !border_cut(n, w, false, false, 0, 0, 0, scale, 0.f, last);
        if (!ordered) drop();
      }
      if (!ordered && by_share) {
        ordered = !border_cut(n, w, true, count_first, 0, 0, need, scale, 0.f, last);
        if (!ordered) drop();
      }
      if (!ordered) {
        // ---- the weight of every run of indices, then of every index of the run that holds the coin
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (w[i] < least || (only_top && w[i] && logit_at(tid + i * kSThreads) != top)) w[i] = 0;
        const int width = (a.V + kSThreads - 1) / kSThreads;  // at most 1024
        uint32_t* runs = fine;                                // [3][kSThreads]
        auto index_of = [&](int i) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(list[tid + i * kSThreads])); };
        __syncthreads();
        for (int i = tid; i < 3 * kSThreads; i += kSThreads) runs[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (w[i]) put_weight(runs + index_of(i) / width, kSThreads, w[i]);
        __syncthreads();
        const uint64_t own = weight_of(runs + tid, kSThreads);
        run = own;
        block_scan(one, run, sh, &none, &total);
        const uint64_t level = __umul64hi(unit_fraction(coin), total);
        if (tid == 0) { sh.dec.cut = last; sh.dec.total = total; }
        if (run - own <= level && run > level) { sh.border_bin = tid; sh.border_before_w = run - own; }
        __syncthreads();
        if (probs) tell();
        if (a.tokens) {
          const int start = sh.border_bin * width;
          uint64_t* slots = bin_w;  // [kFine]
          for (int i = tid; i < kFine; i += kSThreads) slots[i] = 0;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < L; ++i)
            if (w[i] && index_of(i) >= start && index_of(i) < start + width) slots[index_of(i) - start] = w[i];
          __syncthreads();
          const uint64_t s0 = slots[2 * tid], s1 = slots[2 * tid + 1];
          run = s0 + s1;
          one = 0;
          block_scan(one, run, sh, &none, &all);
          const uint64_t before = sh.border_before_w + run - s0 - s1;
          if (before <= level && before + s0 > level) a.tokens[row] = start + 2 * tid;
          if (before + s0 <= level && before + s0 + s1 > level) a.tokens[row] = start + 2 * tid + 1;
        }
        return;
      }
    }
    n = sorted();
    const int limit = count_first ? min(n, top_k) : n;
    one = 0;
    run = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int x = tid * L + i;
      w[i] = x < limit ? weight_at(x) : 0;
      run += w[i];
    }
    uint64_t before = 0 - run;
    block_scan(one, run, sh, &none, &all);
    before += run;
    if (count_first) need = by_share ? share_of(top_p, all) : ~0ull;
    uint32_t left = 0;
    const uint64_t ahead = before;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int x = tid * L + i;
      if (x < limit && (x == 0 || before < need) && w[i] >= least && (!only_top || logit_at(x) == top)) ++left;
      before += w[i];
    }
    block_scan(left, unused, sh, &left, &unused);  // (the total to all)
    const int count = static_cast<int>(left);
    // the kept weight: what stands ahead of the first one that is cut, which the thread that has the last kept one knows
    before = ahead;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      before += w[i];
      if (tid * L + i == count - 1) {
        sh.dec.cut = list[count - 1];
        sh.dec.total = before;
      }
      if (tid * L + i < count) list_w[tid * L + i] = w[i];
    }
    __syncthreads();
    total = sh.dec.total;
    if (probs) tell();
    if (a.tokens) {
      const uint64_t level = __umul64hi(unit_fraction(coin), total);
      // a token's running weight: of all with an index up to its own
      for (int x = tid; x < count; x += kSThreads) {
        const uint32_t own = static_cast<uint32_t>(list[x]);  // 0xffffffff - index
        uint64_t ahead_w = 0;
#pragma unroll 4
        for (int i = 0; i < count; ++i) ahead_w += static_cast<uint32_t>(list[i]) > own ? list_w[i] : 0;
        if (ahead_w <= level && ahead_w + list_w[x] > level) a.tokens[row] = static_cast<int>(0xffffffffu - own);
      }
    }
  };
  // The cut from a list of the tokens of a range with distances from `near` to `far`, of which `before` tokens and `before_w`
  // weight stand ahead; with `add` the kept ones of the list go to the weights of their tiles.
  auto cut_from_list = [&](bool share, uint32_t before, uint64_t before_w, uint64_t need, bool add, float near, float far) {
    int n = min(sh.listed[lists - 1], static_cast<uint32_t>(kList));
    uint64_t w[L], last = 0;
    if (tid == 0) sh.dec.found = 0;
    bool ordered = n <= kShort;
    if (!ordered) {
#pragma unroll
      for (int i = 0; i < L; ++i) w[i] = tid + i * kSThreads < n ? (share ? weight_at(tid + i * kSThreads) : 1) : 0;
      ordered = !border_cut(n, w, share, false, before, before_w, need, kFine / (far - near), near, last);
    }
    if (ordered) {
      n = sorted();
      uint64_t run = 0;
      uint32_t one = 0, none;
      uint64_t all;
#pragma unroll
      for (int i = 0; i < L; ++i) { w[i] = tid * L + i < n && share ? weight_at(tid * L + i) : 0; run += w[i]; }
      before_w -= run;
      block_scan(one, run, sh, &none, &all);
      before_w += run;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int x = tid * L + i;
        if (x < n && (share ? before_w < need && before_w + w[i] >= need : before + x + 1 == static_cast<uint32_t>(top_k))) {
          sh.dec.cut = list[x];
          sh.dec.found = 1;
        }
        before_w += w[i];
      }
      __syncthreads();
      last = sh.dec.cut;
    } else if (tid == 0) {
      sh.dec.found = 1;
    }
    __syncthreads();
    if (add && sh.dec.found)
      for (int x = tid; x < n; x += kSThreads)
        if (list[x] >= last) {
          const int tile = (static_cast<int>(0xffffffffu - static_cast<uint32_t>(list[x])) + logits.off) / kSTile, owner = tile / per;
          atomicAdd(reinterpret_cast<unsigned long long*>(cluster.map_shared_rank(tile_sum, owner) + (tile - owner * per)), weight_at(x));
        }
    __syncthreads();
    clear();  // for the next count: all of the list has been read, and the other CTAs are past their bins
    tell();
  };

  // ---- the cuts
  bool done = false, tiles_known = false;
  uint64_t total = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2 && !done; ++pass) {
    const bool share = pass == 1;
    if (!(share ? by_share : by_count)) continue;
    // by count: from the threads' largest if these can tell and the list has room, else from all tokens
    bool few = !share && top_k <= C * kSThreads / 2;
    Decision d;
    if (few) {
      count_largest();
      d = choose_bins(false);
      few = d.found && gather(below_bin(d.last));
      if (!few) {
        clear();
        cluster.sync();
      }
    }
    if (!few) {
      if (share) count_and_sum();
      else count_all();
      d = choose_bins(share);
      few = d.found && cut == 0 && d.count <= kList - 64 && gather(below_bin(d.last));
    }
    if (few) {
      // (the others have read the leader's count: it may not go before that)
      if (!probs) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
      if (rank == 0) finish_from_list(!share, d.need, (d.last + 1) * 0.03125f);
      if (!probs) {
        if (rank == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        return;
      }
      cluster.sync();
      set_cut(sh.dec.cut);
      total = sh.dec.total;
      done = true;
      break;
    }
    if (!d.found) {  // (top_k reaches into what has no weight)
      clear();
      cluster.sync();
      continue;
    }
    cluster.sync();
    const float ahead_l = above_bin(d.bin0);
    // the last filter's tile sums are what the sample goes by
    const bool last = share || !by_share;
    bool settled = false;
    if (gather_between(below_bin(d.bin1), ahead_l, last)) {
      if (rank == 0) {
        uint64_t ahead = 0;
        uint32_t ahead_n = 0;
        for (int r = 0; r < C; ++r) { ahead += sh.sums[r]; ahead_n += sh.counts[r]; }
        cut_from_list(share, ahead_n, ahead, d.need, last && least == 0, d.bin0 * 0.03125f, (d.bin1 + 1) * 0.03125f);
      } else {
        clear();
      }
      cluster.sync();
      settled = sh.dec.found;
      tiles_known = settled && last && least == 0;
    }
    if (!settled) {
      // (a bin of d, up to four levels of keys where the temperature is infinite, two of indices: every level divides its range by
      // 720 and more)
      int level = 0;
      do {
        const Decision range = d;
        exact_bins(level == 0, range);
        d = choose_exact(level == 0, share, range);
      } while (d.count > kList && ++level < 8);
      gather_range(d);
      if (rank == 0) cut_from_list(share, d.before, d.before_w, d.need, false, 0.f, kFar);
      else clear();
      cluster.sync();
    }
    if (sh.dec.found) set_cut(sh.dec.cut);
  }

  if (only_top && cut_l < top) {  // (nothing before cuts between the tokens of the largest logit)
    cut_l = top;
    cut_i = a.V;
  }
  const bool all = cut == 0 && least == 0;
  auto kept_weights = [&](float l0, float l1, int i, uint64_t& w0, uint64_t& w1) {
    w0 = w1 = 0;
    if (!all && !(l0 >= cut_l) && !(l1 >= cut_l)) return;
    wt.weights(l0, l1, w0, w1);
    if (all) return;
    if (!kept(l0, i) || w0 < least) w0 = 0;
    if (!kept(l1, i + 1) || w1 < least) w1 = 0;
  };
  if (!done) {
    // ---- the weight of every tile, then the token
    uint64_t mine = 0;
    for (int t = warp; t < my_tiles; t += kSWarps) {
      const int at = lo + t * kSTile;
      uint64_t sum = 0;
      if (tiles_known) {
        sum = tile_sum[t];
      } else {
        auto add = [&](auto whole) {
          logits.template each<2>(at, min(hi, at + kSTile), lane, 32, [&](const float (&x)[N], int i) {
#pragma unroll
            for (int j = 0; j < N; j += 2) {
              uint64_t w0, w1;
              if constexpr (decltype(whole)::value) wt.weights(x[j], x[j + 1], w0, w1);
              else kept_weights(x[j], x[j + 1], i + j, w0, w1);
              sum += w0 + w1;
            }
          });
        };
        if (all) add(std::true_type());
        else add(std::false_type());
        sum = warp_sum(sum);
        if (lane == 0) tile_sum[t] = sum;
      }
      mine += sum;
    }
    __syncthreads();
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    if (tid < C) {
      uint64_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSWarps; ++w) sum += sh.warp[w];
      cluster.map_shared_rank(&sh, tid)->sums[rank] = sum;
    }
    cluster.sync();
    uint64_t before = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += sh.sums[r];
      total += sh.sums[r];
    }
    if (a.tokens && warp == 0) {
      const uint64_t level = __umul64hi(unit_fraction(coin), total);
      if (level >= before && level < before + sh.sums[rank]) {  // in this CTA's part
        int t = 0;
        for (int t0 = 0; t0 < my_tiles; t0 += 32) {
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
        // the tile in rounds of 32 vectors: the round, the lane, the token
        constexpr int Rounds = kSTile / 32 / N;
        uint4 v[Rounds];
#pragma unroll
        for (int r = 0; r < Rounds; ++r) v[r] = logits.load(lo + t * kSTile + (r * 32 + lane) * N);
        bool open = true;
#pragma unroll
        for (int r = 0; r < Rounds; ++r) {
          if (!open) continue;
          const int i = lo + t * kSTile + (r * 32 + lane) * N - logits.off;
          float x[N];
          Row<T>::widen(v[r], x);
          uint64_t w[N], run = 0;
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            kept_weights(x[j], x[j + 1], i + j, w[j], w[j + 1]);
            run += w[j] + w[j + 1];
          }
          uint64_t sum = before - run;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
          }
          sum += run;
          const uint64_t end = before + __shfl_sync(0xffffffffu, run, 31);
          if (end > level) {
            open = false;
            bool mine_here = sum <= level;
#pragma unroll
            for (int j = 0; j < N; ++j) {
              sum += w[j];
              if (mine_here && sum > level) {
                a.tokens[row] = i + j;
                mine_here = false;
              }
            }
          }
          before = end;
        }
      }
    }
  }
  if (probs) {
    const float whole = __ull2float_rn(total);
    fill([&](float l0, float l1, int i, float& y0, float& y1) {
      uint64_t w0, w1;
      kept_weights(l0, l1, i, w0, w1);
      y0 = w0 ? __fdiv_rn(__ull2float_rn(w0), whole) : 0.f;
      y1 = w1 ? __fdiv_rn(__ull2float_rn(w1), whole) : 0.f;
    });
  }
}

template <typename T>
cudaError_t launch_sample(const SampleArgs& a, int rows, int sms, cudaStream_t s) {
  // CTAs a row: as many as stay within the SMs with more than 2 tiles each.  Measured with 129,280 words in bf16 and 2, 4, 8
  // CTAs a row, us: top_k 50 and top_p 0.9, 8 rows 23, 18, 15; 64 rows 30, 23, 35; 128 rows 32, 42, 64.
  // Uncut 64 rows 46, 31, 38; 128 rows 50, 57, 70.  Settings of their own: 32 rows 112, 74, 56; 64 rows 125, 84, 72; 128 rows 136,
  // 103, 111.  (So rows of unequal cost would gain by more CTAs than the rule gives from 64 rows on, the others lose.)
  const int tiles = (a.V + 16 / static_cast<int>(sizeof(T)) - 1 + kSTile - 1) / kSTile;  // (of a row that starts anywhere)
  int C = 1;
  while (C < kSCluster && (static_cast<long long>(kSSlice / kSTile) * C < tiles || (2LL * C * rows <= 2 * sms && tiles > C * kSWarps / 4))) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * C);
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = kRegionA + kRegionB + static_cast<size_t>((tiles + C - 1) / C) * 8;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(sample_kernel<T>), kRegionA + kRegionB + (kSSlice / kSTile + 1) * 8);
  return err != cudaSuccess ? err : cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace
}  // namespace gbmoe

extern "C" moe_status_t moe_sample(const moe_sample_args_t* r, moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_sample", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_sample: ") + m); };
    if (!r) return bad("NULL arguments");
    if (r->dtype != MOE_DTYPE_BF16 && r->dtype != MOE_DTYPE_FP16 && r->dtype != MOE_DTYPE_FP32) return bad("unknown dtype");
    if (r->rows < 0 || r->vocab <= 0) return bad("sizes must be positive");
    if (r->vocab > kSVocab || r->rows > (1 << 20))
      return report_error(MOE_ERR_UNSUPPORTED, "moe_sample: more than 524288 tokens in the vocabulary or 2^20 rows");
    if (r->rows == 0 || (!r->tokens && !r->probs)) return MOE_OK;
    if (!r->logits || (r->tokens && !r->coins)) return bad("NULL pointer");
    if (r->logits_stride < r->vocab && r->rows > 1) return bad("a row stride of the logits is shorter than its row");
    if (r->probs && r->probs_stride < r->vocab && r->rows > 1) return bad("a row stride of the probabilities is shorter than its row");
    const size_t es = r->dtype == MOE_DTYPE_FP32 ? 4 : 2;
    if (!aligned(r->logits, es) || !aligned(r->temperature, 4) || !aligned(r->top_k, 4) || !aligned(r->top_p, 4) ||
        !aligned(r->min_p, 4) || !aligned(r->coins, 4) || !aligned(r->tokens, 4) || !aligned(r->probs, 4))
      return bad("unaligned tensors");
    SampleArgs a{r->logits, r->logits_stride, r->temperature, r->top_k, r->top_p, r->min_p, r->coins,
                 r->tokens, r->probs, r->probs_stride, r->vocab};
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_sample: no CUDA device");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched("moe_sample", r->dtype == MOE_DTYPE_FP32   ? launch_sample<float>(a, r->rows, sms, s)
                                  : r->dtype == MOE_DTYPE_FP16 ? launch_sample<__half>(a, r->rows, sms, s)
                                                               : launch_sample<__nv_bfloat16>(a, r->rows, sms, s));
  });
}
