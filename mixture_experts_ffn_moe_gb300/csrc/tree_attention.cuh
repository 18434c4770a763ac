// Shared parts of the tree attention kernels: arguments, the line of tiles, small wrappers.
#pragma once

#include "sm100_ptx.cuh"
#include "step_ops.cuh"

namespace gbmoe {
namespace tree {

constexpr int kMaxBatch = 1024;
constexpr int kMaxTreeCtas = 320;    // CTAs that the workspace has room for
constexpr int kWideTile = 128;       // slots of a tile and rows of a product of the tcgen05 kernel
constexpr int kWideRows = 256;       // rows of its row tile
constexpr float kLazy = 8.f;         // growth of a row's maximum (in powers of two) that moves its reference
// Powers of two by which all of a row's weights (those of P, of its sum l and of O alike) stand above 2^(s - m).  fp16 holds
// 2^15, and a weight of at most 2^kLazy leaves 7 of them: so weights down to 2^-21 of the reference keep fp16's full precision
// in the product with V and those down to 2^-32 do not vanish, instead of 2^-14 and 2^-25.  bf16 has fp32's range.
template <typename T> constexpr float kHeadroom = 0.f;
template <> constexpr float kHeadroom<__half> = 15.f - kLazy;

struct TreeArgs {
  const void* q;
  const void* kc;
  const void* vc;
  void* out;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* offs;
  const unsigned long long* mask;  // null: a chain
  long long q_t, q_h, o_t, o_h;
  long long k_page, k_slot, k_head, v_page, v_slot, v_head;
  long long table_ld;
  int N, B, Hq, Hkv, pages, table_w;
  int tile, rows, ranks;  // slots of a tile, rows of a CTA's row tile, CTAs that work on one range side by side
  int setup;              // places on the line before a unit's first tile: what starting one costs, in tiles
  FastDiv page, group;
  int box;                // slots of a page that one TMA copy brings (0: cp.async)
  float scale_log2;
  int32_t* header;    // workspace: [0] CTAs, [1] bad lengths, offsets or counts, then for every CTA its bad pages
                      // (negative: one of its waits gave up)
  long long* prefix;  // [B + 1] first place of every sequence on the line, [B + 1] = places a group of CTAs
  float* part_o;      // [CTAs * 2][rows][D]
  float* part_ml;     // [CTAs * 2][rows][2]
};

__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Words of two 16-bit elements: does either hold an infinity or NaN?
__device__ __forceinline__ bool nonfinite2(__nv_bfloat16, uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool nonfinite2(__half, uint32_t w) {
  return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

// Committed slots and nodes of sequence b, brought into range (bad counts what had to be).
__device__ __forceinline__ void seq_sizes(const TreeArgs& a, int b, int& ctx, int& n, int& bad) {
  const int lo = a.offs[b], hi = a.offs[b + 1];
  ctx = a.ctx[b];
  n = hi - lo;
  bad = 0;
  const long long room = static_cast<long long>(a.table_w) * a.page.d;
  if (lo < 0 || hi < lo || hi > a.N || n > MOE_MAX_TREE_NODES || n > room) { n = 0; bad = 1; }
  if (ctx < 0) { ctx = 0; bad = 1; }
  if (ctx > room - n) { ctx = static_cast<int>(room - n); bad = 1; }
}

// prefix[b] = first place of sequence b on the line: `setup` places and its tiles for every unit.  sizes[b] = (committed
// slots, nodes).
template <int THREADS>
__device__ __forceinline__ void plan_line(const TreeArgs& a, long long* prefix, int2* sizes, long long* scratch, int* bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long base = 0;
  int nbad = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    long long tiles = 0;
    if (b < a.B) {
      int ctx, n, bd;
      seq_sizes(a, b, ctx, n, bd);
      nbad += bd;
      sizes[b] = make_int2(ctx, n);
      if (n > 0) {
        const int per = a.rows * a.ranks, rt = (n * static_cast<int>(a.group.d) + per - 1) / per;
        tiles = static_cast<long long>(a.Hkv) * rt * (a.setup + (static_cast<long long>(ctx) + n + a.tile - 1) / a.tile);
      }
    }
    long long incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = base, all = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += scratch[w];
      all += scratch[w];
    }
    if (b < a.B) prefix[b] = before + incl - tiles;
    base += all;
    __syncthreads();
  }
  if (tid == 0) prefix[a.B] = base;
  *bad = nbad;
  __syncthreads();
}

// A CTA group's piece of one unit: sequence, KV head, row tile, and the tiles [k0, k1) of the unit's kt (none where the
// piece ends within the unit's setup); `places` is its length on the line.
struct Piece {
  int b, ctx, n, head, row0, rows, node0, k0, k1, kt;
  long long places;
};
__device__ __forceinline__ Piece piece_at(const TreeArgs& a, const long long* prefix, const int2* sizes, long long pos, long long end,
                                          int rank) {
  Piece u;
  int lo = 0, hi = a.B;  // prefix[lo] <= pos < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= pos) lo = mid; else hi = mid;
  }
  u.b = lo;
  u.ctx = sizes[u.b].x;
  u.n = sizes[u.b].y;
  u.kt = (u.ctx + u.n + a.tile - 1) / a.tile;
  const int span = u.kt + a.setup;
  const int group = a.group.d, per = a.rows * a.ranks, rt_n = (u.n * group + per - 1) / per;
  const long long rel = pos - prefix[u.b];
  const int unit = static_cast<int>(rel / span), p0 = static_cast<int>(rel - static_cast<long long>(unit) * span);
  u.places = min(end - pos, static_cast<long long>(span - p0));
  u.k0 = max(0, p0 - a.setup);
  u.k1 = max(0, p0 + static_cast<int>(u.places) - a.setup);
  u.head = unit / rt_n;
  u.row0 = (unit - u.head * rt_n) * per + rank * a.rows;
  u.rows = u.k1 > u.k0 ? max(0, min(a.rows, u.n * group - u.row0)) : 0;  // no rows: nothing to do
  u.node0 = a.offs[u.b];
  return u;
}

// Tensor maps of the caches with boxes of a.box slots: the longest run, up to `most`, that lies in one page and stands
// on 8-row groups of the swizzled tile.  a.box = 0 where there is none (or the strides do not fit a tensor map).
inline void tree_boxes(TreeArgs& a, int D, int most, CUtensorMap* mk, CUtensorMap* mv) {
  a.box = most;
  while (a.box > 1 && a.page.d % a.box) a.box /= 2;
  if (a.box < 8 || !encode_tmap_cache(mk, a.kc, D, a.page.d, a.Hkv, a.pages, a.k_slot, a.k_head, a.k_page, 64, a.box) ||
      !encode_tmap_cache(mv, a.vc, D, a.page.d, a.Hkv, a.pages, a.v_slot, a.v_head, a.v_page, 64, a.box))
    a.box = 0;
}

// Launches the tcgen05 kernel (tree_attention_wide.cu) on `ctas` CTAs, one an SM.
cudaError_t launch_tree_wide(const TreeArgs& a, bool bf16, int D, int ctas, cudaStream_t s);

}  // namespace tree
}  // namespace gbmoe
