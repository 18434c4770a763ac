// Attention of drafted tokens over a paged cache: every node of a sequence's draft tree attends to all of the
// sequence's committed slots and to those drafted slots whose bits its mask has (its ancestors and itself).
//
// Mathematics.  For node j and query head h of KV head h / (Hq / Hkv):
//   out = sum_k softmax_k(scale * q . K_k) V_k  over the visible slots k, in one pass over the cache: a running
// reference m, the sum l of 2^(s - m) and the unnormalised output are kept in fp32, and partial results over
// different slots are joined as (m, l, O).  The reference is moved (and O rescaled) only when a row's maximum has
// grown by more than 2^8; that leaves the result the same and keeps 2^(s - m) at most 2^8.  A row that sees
// nothing gives zeros.  P is rounded to the cache's type for the product with V, l is the sum of the unrounded weights: half a
// step of that type a term, as the output is itself rounded to it.  In fp16 the weights stand 2^7 higher (kHeadroom), since
// fp16 has few bits for small ones: a slot 2^25 below a row's largest still counts.
//
// Bound: K and V are read once: 4 * L * Hkv * D bytes.  The nodes of a tree and the query heads of a KV head
// are rows of one matrix product, so a cache line serves all of them.
//
// Work split.  A unit is (sequence, KV head, tile of rows); its cache is cut in tiles of 64 slots.  The tiles of all
// units form one line that is divided evenly over the CTAs, whatever the lengths; where a unit is cut, the parts
// go to the workspace as fp32 (m, l, O) and a second kernel joins them in order, so results do not depend on
// scheduling.  Inside a CTA each warp owns 16 slots of every tile with a ring of stages of its own, so warps never
// wait for each other inside a unit.  Where pages hold a multiple of 8 slots a stage is brought by 2 or 4 TMA boxes
// (128-byte swizzle), else slot by slot with cp.async; the next stage's block table entry is read a tile ahead.
//
// Measured: 32 sequences of 300 to 4100 slots, chains of 4 nodes, 32 / 8 heads of 128 (261 MB): 51.8 us = 5.0 TB/s, of which
// planning and the first loads take about 3 us and the join of the parts 3; 5 nodes over 37 slots: 7.8 us, a chain of launch,
// lengths, table, cache, and the join's launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include "tree_attention.cuh"

namespace gbmoe {
namespace {

using namespace tree;

constexpr int kAWarps = 4;
constexpr int kAThreads = kAWarps * 32;
constexpr int kTile = kAWarps * 16;  // cache slots a tile

template <int D> struct TreeCfg {
  static constexpr int kRow = D * 2;                     // bytes of a cache row
  static constexpr int kHalf = 16 * 128;                 // 64 columns of 16 slots
  static constexpr int kStage = 16 * kRow * 2;           // K and V of 16 slots
  static constexpr int S = D == 128 ? 3 : 6;             // stages a warp
  static constexpr int kRing = S * kStage;               // 24 KB a warp
};

template <int D, int RT> constexpr size_t tree_smem(int B) {
  return static_cast<size_t>(kAWarps) * (TreeCfg<D>::kRing > RT * 16 * D * 4 ? TreeCfg<D>::kRing : RT * 16 * D * 4) +
         RT * 16 * D * 2 + (2 * B + 1 + kAWarps) * 8 + kAWarps * (8 * 4 + 8 * 8 + RT * 16 * 8) + 16 + 1024;
}

constexpr long long kLimit = 4000000000LL;  // about 2 s of SM clocks a wait

template <typename T, int D, int RT, bool TMA>
__global__ void __launch_bounds__(kAThreads, 2)
    tree_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = TreeCfg<D>;
  constexpr int R = RT * 16, KS = D / 16, CH = D / 8;  // rows, K steps, 16-byte chunks a row
  constexpr int kWarpBytes = C::kRing > R * D * 4 ? C::kRing : R * D * 4;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
  unsigned char* ring = smem + (threadIdx.x >> 5) * kWarpBytes;
  unsigned char* qs = smem + kAWarps * kWarpBytes;                                       // [R][D]
  long long* prefix = reinterpret_cast<long long*>(qs + R * D * 2);                      // [B + 1], then scan scratch
  int2* sizes = reinterpret_cast<int2*>(prefix + a.B + 1 + kAWarps);                     // [B]
  uint64_t* full = reinterpret_cast<uint64_t*>(sizes + a.B) + (threadIdx.x >> 5) * 8;    // [S] a warp (TMA)
  float* ml = reinterpret_cast<float*>(reinterpret_cast<uint64_t*>(sizes + a.B) + kAWarps * 8);  // [warps][R][2]
  uint32_t* okmask = reinterpret_cast<uint32_t*>(ml + kAWarps * R * 2) + (threadIdx.x >> 5) * 8;  // [S] a warp
  int* abort_s = reinterpret_cast<int*>(ml + kAWarps * R * 2) + kAWarps * 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring_s = sm100::smem_addr(ring), q_s = sm100::smem_addr(qs);
  // offset of chunk ch of slot `key` in a stage's K or V: halves of 64 columns, 128-byte rows, swizzled
  auto chunk_at = [](int key, int ch) { return (ch >> 3) * C::kHalf + key * 128 + (((ch & 7) ^ (key & 7)) << 4); };

  pdl_trigger();
  if constexpr (TMA) {
    if (lane == 0)
      for (int i = 0; i < C::S; ++i) sm100::mbar_init(&full[i], 1);
    if (tid == 0) *abort_s = 0;
    sm100::fence_barrier_init();
  }
  pdl_wait();
  int bad_plan;
  plan_line<kAThreads>(a, prefix, sizes, prefix + a.B + 1, &bad_plan);
  const long long total = prefix[a.B];
  const long long chunk = (total + gridDim.x - 1) / gridDim.x;
  if (blockIdx.x == 0) {
    bad_plan = __syncthreads_count(bad_plan);
    if (tid == 0) { a.header[0] = gridDim.x; a.header[1] = bad_plan; a.prefix[a.B + 1] = chunk; }
    for (int b = tid; b <= a.B; b += kAThreads) a.prefix[b] = prefix[b];
  }
  int bad_pages = 0;
  int used = 0;  // stages this warp has used (TMA): stage used % S, phase used / S
  auto stage_of = [&](int ahead) { return (used + ahead) % C::S; };
  bool fine = true;
  long long pos = blockIdx.x * chunk;
  const long long end = pos + chunk < total ? pos + chunk : total;
  while (pos < end) {
    const Piece u = piece_at(a, prefix, sizes, pos, end, 0);
    pos += u.places;
    if (u.rows == 0) continue;
    const int b = u.b, ctx = u.ctx, L = u.ctx + u.n, kt = u.kt, k0 = u.k0, k1 = u.k1, head = u.head, row0 = u.row0;
    const int rows = u.rows, node0 = u.node0;
    const T* kbase = static_cast<const T*>(a.kc) + head * a.k_head;
    const T* vbase = static_cast<const T*>(a.vc) + head * a.v_head;
    const int32_t* table = a.table + b * a.table_ld;

    // The block table entry of this lane's slot of tile `it` (TMA: of its box, lane = box), before its use.
    struct Place { int page, at; };
    auto look_up = [&](int it) {
      const int slot = it * kTile + warp * 16 + (TMA ? lane * a.box : lane);
      Place p{-1, 0};
      if (it < k1 && lane < (TMA ? (a.box == 16 ? 1 : 2) : 16) && slot < L) {
        const int pi = div_by(slot, a.page);
        p.at = slot - pi * a.page.d;
        p.page = __ldg(table + pi);
      }
      return p;
    };
    // this warp's 16 slots of tile `it`, which lie at `place`, into stage `st`
    auto issue = [&](int it, int st, Place place) {
      const int at = place.at;
      int page = place.page;
      if (page < 0 || page >= a.pages) {
        const int slot = it * kTile + warp * 16 + (TMA ? lane * a.box : lane);
        if (lane < (TMA ? (a.box == 16 ? 1 : 2) : 16) && slot < L) bad_pages += TMA ? min(a.box, L - slot) : 1;
        page = -1;
      }
      if constexpr (TMA) {
        const int pg = __shfl_sync(0xffffffffu, page, (lane & 15) >> (a.box == 16 ? 4 : 3)), sl = __shfl_sync(0xffffffffu, at, (lane & 15) >> (a.box == 16 ? 4 : 3));
        const uint32_t ok = __ballot_sync(0xffffffffu, lane < 16 && pg >= 0 && it * kTile + warp * 16 + lane < L);
        if (lane == 0) {
          okmask[st] = ok;
          sm100::mbar_arrive_expect_tx(&full[st], C::kStage);
        }
        __syncwarp();
        // lanes on the first slot of a box: K and V of each half.  Page -1 is outside the tensor: zeros.
        if (lane < 16 && (lane & (a.box - 1)) == 0) {
          const uint32_t dst = ring_s + st * C::kStage + lane * 128;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            sm100::tma_load_4d(dst + h * C::kHalf, &mk, &full[st], h * 64, sl, head, pg);
            sm100::tma_load_4d(dst + 16 * C::kRow + h * C::kHalf, &mv, &full[st], h * 64, sl, head, pg);
          }
        }
      } else {
        const uint32_t ok = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) okmask[st] = ok;
        const uint32_t base = ring_s + st * C::kStage;
#pragma unroll
        for (int i = 0; i < 16 * CH / 32; ++i) {
          const int c = i * 32 + lane, r = c / CH, ch = c % CH;
          const int pg = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, at, r);
          const bool live = pg >= 0;
          const long long p = live ? pg : 0;
          const uint32_t dst = base + chunk_at(r, ch);
          cp_async16(dst, kbase + p * a.k_page + sl * a.k_slot + ch * 8, live);
          cp_async16(dst + 16 * C::kRow, vbase + p * a.v_page + sl * a.v_slot + ch * 8, live);
        }
      }
    };
    // A unit starts with all of its loads under way at once: places of the first tiles, queries and masks (rows past
    // the last one repeat it, without a branch around the loads: nothing is taken from them).
    __syncwarp();
    Place first[C::S - 1];
#pragma unroll
    for (int s = 0; s < C::S - 1; ++s) first[s] = look_up(k0 + s);
    Place next = look_up(k0 + C::S - 1);
    // row r of the unit is node r / group, head r % group of the KV head's queries
    uint4 qv[R * CH / kAThreads];
#pragma unroll
    for (int k = 0; k < R * CH / kAThreads; ++k) {
      const int i = tid + k * kAThreads, r = row0 + min(i / CH, rows - 1), node = div_by(r, a.group);
      const int hq = head * a.group.d + (r - node * a.group.d);
      qv[k] = ld_v4(static_cast<const T*>(a.q) + (node0 + node) * a.q_t + hq * a.q_h + i % CH * 8);
    }
    unsigned long long bits[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int node = div_by(row0 + min(r * 16 + h * 8 + g, rows - 1), a.group);
        bits[r][h] = (2ull << node) - 1;
        if (a.mask) bits[r][h] = a.mask[node0 + node];
      }
    int sent = 0;  // tiles of this unit
#pragma unroll
    for (int s = 0; s < C::S - 1; ++s) {
      if (k0 + s < k1) { issue(k0 + s, TMA ? stage_of(s) : s, first[s]); ++sent; }
      if constexpr (!TMA) cp_commit();
    }
#pragma unroll
    for (int k = 0; k < R * CH / kAThreads; ++k) {
      const int i = tid + k * kAThreads, r = i / CH, ch = i % CH;
      *reinterpret_cast<uint4*>(qs + r * C::kRow + ((ch ^ (r & 7)) << 4)) = qv[k];
    }
    __syncthreads();

    float o[RT][CH][4], m[RT][2], l[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int d = 0; d < CH; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[r][d][i] = 0.f;
      m[r][0] = m[r][1] = -INFINITY;
      l[r][0] = l[r][1] = 0.f;
    }

    int st = TMA ? stage_of(0) : 0;
    for (int it = k0; it < k1; ++it) {
      if constexpr (TMA) {
        fine = __all_sync(0xffffffffu, sm100::mbar_wait(&full[st], (used / C::S) & 1, abort_s, nullptr, kLimit)) != 0;
        if (!fine) break;
      } else {
        cp_wait<C::S - 2>();
        __syncwarp();
      }
      const uint32_t kst = ring_s + st * C::kStage, vst = kst + 16 * C::kRow;
      const uint32_t ok = okmask[st];
      const int slot0 = it * kTile + warp * 16;
      float s[RT][2][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[r][i >> 2][i & 3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t kb[4];
        const int key = ((lane >> 4) << 3) + (lane & 7), ch = ks * 2 + ((lane >> 3) & 1);
        ldm4(kst + chunk_at(key, ch), kb);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t qa[4];
          const int qr = r * 16 + (lane & 15), qc = ks * 2 + (lane >> 4);
          ldm4(q_s + qr * C::kRow + ((qc ^ (qr & 7)) << 4), qa);
          mma_16816(T(), s[r][0], qa, kb[0], kb[1]);
          mma_16816(T(), s[r][1], qa, kb[2], kb[3]);
        }
      }
      const bool edge = ok != 0xffffu || slot0 + 16 > ctx;
      uint32_t p[RT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[4] = {s[r][0][2 * h], s[r][0][2 * h + 1], s[r][1][2 * h], s[r][1][2 * h + 1]};
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] *= a.scale_log2;
          if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = (i >> 1) * 8 + 2 * t + (i & 1), node = slot0 + key - ctx;
              const bool sees = ((ok >> key) & 1) && (node < 0 || ((bits[r][h] >> (node & 63)) & 1));
              if (!sees) v[i] = -INFINITY;
            }
          }
          float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const bool grow = mx > m[r][h] + kLazy || (m[r][h] == -INFINITY && mx > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float nm = grow ? mx : m[r][h];
            const float f = grow ? ex2(m[r][h] - nm) : 1.f;  // 0 for the first reference
            m[r][h] = nm;
            l[r][h] *= f;
#pragma unroll
            for (int d = 0; d < CH; ++d) { o[r][d][2 * h] *= f; o[r][d][2 * h + 1] *= f; }
          }
          const float ref = (m[r][h] == -INFINITY ? 0.f : m[r][h]) - kHeadroom<T>;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = ex2(v[i] - ref);
          l[r][h] += (v[0] + v[1]) + (v[2] + v[3]);
          p[r][h] = Elem<T>::pack(v[0], v[1]);
          p[r][2 + h] = Elem<T>::pack(v[2], v[3]);
        }
      }
      unsigned char* vrows = ring + st * C::kStage + 16 * C::kRow;
      if constexpr (TMA) {
        if (ok != 0xffffu) {  // rows of the last page past the sequence's end hold anything
#pragma unroll
          for (int i = 0; i < 16 * CH / 32; ++i) {
            const int c = i * 32 + lane, r = c / CH, ch = c % CH;
            if (!((ok >> r) & 1)) *reinterpret_cast<uint4*>(vrows + chunk_at(r, ch)) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
      }
      if (slot0 + 16 > ctx) {
        // Drafted slots are hidden from some rows: an infinity or NaN of a hidden value would come through as
        // 0 * inf.  Such slots (rare) are added to the rows that see them one by one and cleared for the rest.
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < 16 * CH / 32; ++i) {
          const int c = i * 32 + lane, r = c / CH, ch = c % CH;
          const uint4 v = *reinterpret_cast<const uint4*>(vrows + chunk_at(r, ch));
          const bool nf = nonfinite2(T(), v.x) || nonfinite2(T(), v.y) || nonfinite2(T(), v.z) || nonfinite2(T(), v.w);
          if (nf && slot0 + r >= ctx) odd |= 1u << r;
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
        while (odd) {
          const int key = __ffs(odd) - 1;
          odd &= odd - 1;
          const int node = slot0 + key - ctx;
          const int src = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = __shfl_sync(0xffffffffu, key < 8 ? p[r][h] : p[r][2 + h], src);
              const float2 pp = Elem<T>::unpack(w);
              const float pk = (key & 1) ? pp.y : pp.x;
              if ((bits[r][h] >> node) & 1) {
#pragma unroll
                for (int d = 0; d < CH; ++d) {
                  const float2 vv = Elem<T>::unpack(*reinterpret_cast<const uint32_t*>(vrows + chunk_at(key, d) + t * 4));
                  o[r][d][2 * h] += pk * vv.x;
                  o[r][d][2 * h + 1] += pk * vv.y;
                }
              }
            }
          __syncwarp();
          if (lane < CH) *reinterpret_cast<uint4*>(vrows + chunk_at(key, lane)) = make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
      }
#pragma unroll
      for (int db = 0; db < KS; ++db) {
        uint32_t vb[4];
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7), ch = db * 2 + (lane >> 4);
        ldm4t(vst + chunk_at(key, ch), vb);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          mma_16816(T(), o[r][2 * db], p[r], vb[0], vb[1]);
          mma_16816(T(), o[r][2 * db + 1], p[r], vb[2], vb[3]);
        }
      }
      if constexpr (TMA) {
        if (ok != 0xffffu || slot0 + 16 > ctx) sm100::fence_proxy_async_smem();  // (rows were cleared)
      }
      __syncwarp();
      const int nx = it + C::S - 1;
      if (nx < k1) {
        issue(nx, st == 0 ? C::S - 1 : st - 1, next);
        next = look_up(nx + 1);
        ++sent;
      }
      if constexpr (!TMA) cp_commit();
      st = st + 1 == C::S ? 0 : st + 1;
      ++used;
    }
    if constexpr (TMA) {
      if (!__syncthreads_and(fine)) {  // a wait gave up: what is on its way lands before the CTA goes
        int none = 0;
        const int done = used;  // of this unit: sent - (stages used in it) are in flight
        for (int i = 0; i < C::S - 1; ++i)
          if (lane == 0 && i < sent) sm100::mbar_wait(&full[(done + i) % C::S], ((done + i) / C::S) & 1, &none, nullptr, kLimit / 4);
        fine = false;
        break;
      }
    } else {
      cp_wait<0>();
      __syncwarp();
    }

    // join the warps' slots: m, l and O of every row
    float* mine = reinterpret_cast<float*>(ring);  // [R][D]
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[r][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int row = r * 16 + h * 8 + g;
        if (t == 0) { ml[(warp * R + row) * 2] = m[r][h]; ml[(warp * R + row) * 2 + 1] = sum; }
#pragma unroll
        for (int d = 0; d < CH; ++d)
          *reinterpret_cast<float2*>(mine + row * D + ((d * 8 + 2 * t) ^ ((row & 3) << 3))) =
              make_float2(o[r][d][2 * h], o[r][d][2 * h + 1]);
      }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == kt;
    const long long slot = static_cast<long long>(blockIdx.x) * 2 + (k0 == 0 ? 1 : 0);
    for (int i = tid; i < rows * (D / 4); i += kAThreads) {
      const int row = i / (D / 4), c = (i % (D / 4)) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAWarps; ++w) mm = fmaxf(mm, ml[(w * R + row) * 2]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kAWarps; ++w) {
        const float f = ex2(ml[(w * R + row) * 2] - ref);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * kWarpBytes) + row * D +
                                                          (c ^ ((row & 3) << 3)));
        sum += f * ml[(w * R + row) * 2 + 1];
        acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int node = div_by(row0 + row, a.group), hq = head * a.group.d + (row0 + row - node * a.group.d);
        T* dst = static_cast<T*>(a.out) + (node0 + node) * a.o_t + hq * a.o_h + c;
        *reinterpret_cast<uint2*>(dst) = make_uint2(Elem<T>::pack(acc.x * inv, acc.y * inv), Elem<T>::pack(acc.z * inv, acc.w * inv));
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * R + row) * D + c) = acc;
        if (c == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * R + row) * 2) = make_float2(mm, sum);
      }
    }
    if constexpr (TMA) sm100::fence_proxy_async_smem();  // the sums stood where the next unit's stages go
    __syncthreads();
  }
  bad_pages = __reduce_add_sync(0xffffffffu, bad_pages);
  __syncthreads();
  if (lane == 0) okmask[0] = bad_pages;
  __syncthreads();
  if (tid == 0) {
    int all = 0;
    for (int w = 0; w < kAWarps; ++w) all += okmask[w * 8];
    a.header[2 + blockIdx.x] = fine ? all : -1;
  }
}

// Joins the parts of units that were cut; one warp a row (node, query head).
template <typename T, int D>
__global__ void __launch_bounds__(128) tree_join_kernel(TreeArgs a) {
  pdl_trigger();
  pdl_wait();
  const long long row_id = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row_id >= static_cast<long long>(a.N) * a.Hq) return;
  const int i = static_cast<int>(row_id / a.Hq), hq = static_cast<int>(row_id - static_cast<long long>(i) * a.Hq);
  // The sequence of node i: the last one that starts at or before it where all offsets ascend.  Beside offsets that do not,
  // that can be a sequence without the node (or none); then all of them are asked.
  static_assert(kMaxBatch <= 32 * 32, "two steps");
  int ctx, n, bd, j;
  auto owner = [&](int s) {
    seq_sizes(a, s, ctx, n, bd);
    j = i - a.offs[s];
    return j >= 0 && j < n;
  };
  const int step = (a.B + 31) / 32;
  int b = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {  // every step-th sequence, then those in between
    const int at = b + lane * (s ? 1 : step);
    const uint32_t before = __ballot_sync(0xffffffffu, (s == 0 || lane < step) && at < a.B && a.offs[min(at, a.B - 1)] <= i);
    b += before ? (31 - __clz(before)) * (s ? 1 : step) : 0;
  }
  if (!owner(b)) {
    uint32_t who = 0;
    int first = 0;
    for (; first < a.B; first += 32) {
      const int s = first + lane;
      who = __ballot_sync(0xffffffffu, s < a.B && owner(min(s, a.B - 1)));
      if (who) break;
    }
    if (!who) return;
    b = first + __ffs(who) - 1;
    owner(b);
  }
  const int group = a.group.d, head = hq / group, r = j * group + (hq - head * group);
  const int kt = (ctx + n + a.tile - 1) / a.tile, per = a.rows * a.ranks, rt_n = (n * group + per - 1) / per;
  const long long chunk = a.prefix[a.B + 1];
  const long long s = a.prefix[b] + (static_cast<long long>(head) * rt_n + r / per) * (kt + a.setup), e = s + a.setup + kt;
  const long long c0 = (s + a.setup) / chunk, c1 = (e - 1) / chunk;  // from the CTA with the unit's first tile
  if (c0 == c1) return;
  const int rank = r % per / a.rows, row = r % a.rows, parts = static_cast<int>(c1 - c0 + 1);
  auto at = [&](int p) {
    const long long c = c0 + p;
    return ((c * a.ranks + rank) * 2 + (p == 0 ? 1 : 0)) * a.rows + row;
  };
  float mm = -INFINITY;
  for (int p = lane; p < parts; p += 32) mm = fmaxf(mm, a.part_ml[at(p) * 2]);
  mm = warp_max(mm);
  const float ref = mm == -INFINITY ? 0.f : mm;
  constexpr int E = D / 32;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int k = 0; k < E; ++k) acc[k] = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const long long x = at(p);
    const float2 v = *reinterpret_cast<const float2*>(a.part_ml + x * 2);
    const float f = ex2(v.x - ref);
    sum += f * v.y;
#pragma unroll
    for (int k = 0; k < E; ++k) acc[k] += f * a.part_o[x * D + lane * E + k];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* dst = static_cast<T*>(a.out) + i * a.o_t + hq * a.o_h + lane * E;
#pragma unroll
  for (int k = 0; k < E; k += 2) *reinterpret_cast<uint32_t*>(dst + k) = Elem<T>::pack(acc[k] * inv, acc[k + 1] * inv);
}

struct TreeLayout {
  size_t header = 0, prefix = 0, ml = 0, o = 0, total = 0;
};
TreeLayout tree_layout(int B, int ctas, int rows, int D) {
  TreeLayout l;
  size_t at = 0;
  auto take = [&](size_t n) { const size_t r = at; at = (at + n + 255) / 256 * 256; return r; };
  l.header = take((2 + static_cast<size_t>(kMaxTreeCtas)) * 4);
  l.prefix = take((static_cast<size_t>(B) + 2) * 8);
  l.ml = take(static_cast<size_t>(ctas) * 2 * rows * 8);
  l.o = take(static_cast<size_t>(ctas) * 2 * rows * D * 4);
  l.total = at;
  return l;
}

// How a call is cut, from the host's sizes: the average tree's rows a KV head.  Measured with 16 sequences of 2000 slots, 8 KV
// heads of 128: up to 16 rows 33.0 us in tiles of 16 and 39.4 in tiles of 32; about 30 rows 43.1 and 41.3, on tcgen05 45;
// about 38 rows 53.7, 52.2 and 46.5.  CTAs side by side on one range (ranks), rows over 256: 4 sequences of 16,000 slots,
// 512 rows: 2 CTAs 175 us, 1 CTA 177, 4 (two of them idle) 296.
struct TreePlan { int rows, ranks; bool wide; };
TreePlan tree_plan(int N, int B, int Hq, int Hkv) {
  const long long avg = (static_cast<long long>(N) + B - 1) / B * (Hq / Hkv);
  if (avg <= 16) return {16, 1, false};
  if (avg <= 32) return {32, 1, false};
  return {kWideRows, avg <= kWideRows ? 1 : avg <= 2 * kWideRows ? 2 : 4, true};
}

template <typename T, int D, int RT>
cudaError_t launch_narrow(TreeArgs& a, int ctas, cudaStream_t s) {
  CUtensorMap mk{}, mv{};
  tree_boxes(a, D, 16, &mk, &mv);
  auto kern = a.box ? tree_kernel<T, D, RT, true> : tree_kernel<T, D, RT, false>;
  cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(tree_smem<D, RT>(kMaxBatch)));
  if (err != cudaSuccess) return err;
  return launch_kernel(kern, dim3(ctas), dim3(kAThreads), tree_smem<D, RT>(a.B), s, true, a, mk, mv);
}

template <typename T>
cudaError_t launch_tree(TreeArgs& a, int D, const TreePlan& p, int sms, bool bounded_to_one_tile, cudaStream_t s) {
  cudaError_t err;
  if (p.wide) {
    const int ctas = sms / p.ranks * p.ranks;
    err = launch_tree_wide(a, std::is_same<T, __nv_bfloat16>::value, D, ctas < kMaxTreeCtas / 2 ? ctas : kMaxTreeCtas / 2 / p.ranks * p.ranks, s);
  } else {
    const int ctas = 2 * sms < kMaxTreeCtas ? 2 * sms : kMaxTreeCtas;
    if (D == 128) err = p.rows == 16 ? launch_narrow<T, 128, 1>(a, ctas, s) : launch_narrow<T, 128, 2>(a, ctas, s);
    else err = p.rows == 16 ? launch_narrow<T, 64, 1>(a, ctas, s) : launch_narrow<T, 64, 2>(a, ctas, s);
  }
  if (err != cudaSuccess || bounded_to_one_tile) return err;  // a unit of one tile is never cut
  const long long rows = static_cast<long long>(a.N) * a.Hq;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  return D == 128 ? launch_kernel(tree_join_kernel<T, 128>, grid, dim3(128), 0, s, true, a)
                  : launch_kernel(tree_join_kernel<T, 64>, grid, dim3(128), 0, s, true, a);
}

// CTAs that the workspace of a call has partial results for.
int tree_part_ctas(const TreePlan& p) { return p.wide ? kMaxTreeCtas / 2 : kMaxTreeCtas; }

}  // namespace
}  // namespace gbmoe

extern "C" size_t moe_tree_attention_workspace_size(int nodes, int batch, int q_heads, int k_heads, int dim) {
  using namespace gbmoe;
  if (nodes < 0 || batch <= 0 || batch > kMaxBatch || q_heads <= 0 || k_heads <= 0 || q_heads % k_heads ||
      (dim != 64 && dim != 128))
    return 0;
  const TreePlan p = tree_plan(nodes, batch, q_heads, k_heads);
  return tree_layout(batch, tree_part_ctas(p), p.rows, dim).total;
}

extern "C" moe_status_t moe_tree_attention(const moe_tree_attention_args_t* r, void* workspace, size_t workspace_bytes,
                                           moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_tree_attention", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_tree_attention: ") + m); };
    auto not_built = [](const char* m) { return report_error(MOE_ERR_UNSUPPORTED, std::string("moe_tree_attention: ") + m); };
    if (!r) return bad("NULL arguments");
    if (r->dtype != MOE_DTYPE_BF16 && r->dtype != MOE_DTYPE_FP16) return bad("dtype must be bf16 or fp16");
    if (r->nodes < 0 || r->batch < 0 || r->q_heads <= 0 || r->k_heads <= 0 || r->page_size <= 0 || r->num_pages < 0 ||
        r->table_width < 0)
      return bad("sizes must be positive");
    if (r->q_heads % r->k_heads) return bad("q_heads must be a multiple of k_heads");
    if (r->dim != 64 && r->dim != 128) return not_built("head dimension must be 64 or 128");
    if (r->batch > kMaxBatch) return not_built("more than 1024 sequences");
    if (r->q_heads / r->k_heads > 1024 || r->k_heads > 65536 || r->nodes > (1 << 20))
      return not_built("problem too large");
    if (static_cast<long long>(r->table_width) * r->page_size > 0x7fffff00LL)
      return not_built("more than 2^31 - 256 slots a sequence");
    if (!(r->scale > -INFINITY && r->scale < INFINITY)) return bad("scale must be finite");
    if (r->nodes == 0 || r->batch == 0) return MOE_OK;
    if (!r->q || !r->k_cache || !r->v_cache || !r->block_table || !r->context_lens || !r->node_offsets || !r->out)
      return bad("NULL pointer");
    const long long strides[] = {r->q_stride_t, r->q_stride_h, r->k_page_stride, r->k_slot_stride, r->k_head_stride,
                                 r->v_page_stride, r->v_slot_stride, r->v_head_stride};
    for (long long s : strides)
      if (s % 8) return bad("strides must be multiples of 8 elements (16 bytes)");
    if (r->out_stride_t % 4 || r->out_stride_h % 4) return bad("output strides must be multiples of 4 elements");
    if (!aligned(r->q, 16) || !aligned(r->k_cache, 16) || !aligned(r->v_cache, 16)) return bad("q and the caches must be 16-byte aligned");
    if (!aligned(r->out, 8) || !aligned(r->tree_mask, 8)) return bad("out and tree_mask must be 8-byte aligned");
    const TreePlan p = tree_plan(r->nodes, r->batch, r->q_heads, r->k_heads);
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_tree_attention: no CUDA device");
    const TreeLayout l = tree_layout(r->batch, tree_part_ctas(p), p.rows, r->dim);
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256))
      return report_error(MOE_ERR_WORKSPACE, "moe_tree_attention: workspace NULL, misaligned or too small");
    TreeArgs a{};
    a.q = r->q; a.kc = r->k_cache; a.vc = r->v_cache; a.out = r->out;
    a.table = r->block_table; a.ctx = r->context_lens; a.offs = r->node_offsets;
    a.mask = reinterpret_cast<const unsigned long long*>(r->tree_mask);
    a.q_t = r->q_stride_t; a.q_h = r->q_stride_h; a.o_t = r->out_stride_t; a.o_h = r->out_stride_h;
    a.k_page = r->k_page_stride; a.k_slot = r->k_slot_stride; a.k_head = r->k_head_stride;
    a.v_page = r->v_page_stride; a.v_slot = r->v_slot_stride; a.v_head = r->v_head_stride;
    a.table_ld = r->table_stride;
    a.N = r->nodes; a.B = r->batch; a.Hq = r->q_heads; a.Hkv = r->k_heads; a.pages = r->num_pages; a.table_w = r->table_width;
    a.page = fast_div(r->page_size);
    a.group = fast_div(r->q_heads / r->k_heads);
    a.scale_log2 = r->scale * 1.4426950408889634f;
    char* ws = static_cast<char*>(workspace);
    a.header = reinterpret_cast<int32_t*>(ws + l.header);
    a.prefix = reinterpret_cast<long long*>(ws + l.prefix);
    a.part_ml = reinterpret_cast<float*>(ws + l.ml);
    a.part_o = reinterpret_cast<float*>(ws + l.o);
    a.tile = p.wide ? kWideTile : kTile;
    a.rows = p.rows;
    a.ranks = p.ranks;
    a.setup = 4;  // measured 1, 2, 3, 4: 57.5, 54.6, 52.2, 52.0 us for ragged short units (6, 9: slower again), 463 to 459 us for long ones
    const bool one_tile = static_cast<long long>(r->table_width) * r->page_size <= a.tile;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched("moe_tree_attention", r->dtype == MOE_DTYPE_FP16 ? launch_tree<__half>(a, r->dim, p, sms, one_tile, s)
                                                                     : launch_tree<__nv_bfloat16>(a, r->dim, p, sms, one_tile, s));
  });
}

extern "C" moe_status_t moe_read_tree_status(const void* workspace, int32_t status_out[2], moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_read_tree_status", [&]() -> moe_status_t {
    if (!workspace || !status_out) return report_error(MOE_ERR_INVALID_ARG, "moe_read_tree_status: NULL pointer");
    int32_t host[2 + kMaxTreeCtas];
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = cudaMemcpyAsync(host, workspace, sizeof(host), cudaMemcpyDeviceToHost, s);
    if (err == cudaSuccess) err = cudaStreamSynchronize(s);
    if (err != cudaSuccess) return launched("moe_read_tree_status", err);
    int pages = 0;
    bool gave_up = false;
    for (int c = 0; c < host[0] && c < kMaxTreeCtas; ++c) {
      if (host[2 + c] < 0) gave_up = true; else pages += host[2 + c];
    }
    status_out[0] = host[1];
    status_out[1] = pages;
    if (gave_up) return report_error(MOE_ERR_TIMEOUT, "moe_read_tree_status: a bounded device wait gave up");
    if (host[1] || pages)
      return report_error(MOE_ERR_BAD_IDS, "moe_read_tree_status: lengths, node offsets or cache pages out of range");
    return MOE_OK;
  });
}
