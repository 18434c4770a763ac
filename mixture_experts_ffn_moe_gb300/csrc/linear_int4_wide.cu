// 4-bit linear layer for more rows than linear_int4.cu takes in one launch, on the 5th-generation tensor cores.
//
// The weights stay the 128-row operand: a tile is 128 weight rows (gated: 64 gate rows and their 64 up rows), a block
// 128 columns of it, 8 KB of codes.  Per block
//   D = U x^T  (tcgen05.mma, U from tensor memory, x from shared memory, fp32 in tensor memory)
//   acc[row, token] += s[row, group] * 2^e[token] * (D[row, token] - 8 sum x[token])
// where U holds the biased codes as fp16 subnormals and x is kept in fp16 frames in the codes' order, as in
// linear_int4.cu (the same first kernel writes it).  A thread owns a weight row: it reads the row's 64 bytes
// of a block, expands them (5 integer instructions for 8 codes) into tensor memory, and takes the block's sums back
// into fp32 registers.  Three warpgroups take blocks in turn, so that one expands while another's product runs.
//
// What bounds it is a block's way through the roles.  A warpgroup takes about 3,200 cycles for one: 870 until its codes are
// there, 590 to expand them, 1,500 for its product in a queue of three, 225 to take the sums; so with three of them one leaves
// every 1,060.  The products alone take 48 cycles each back to back whatever the tokens up to 64 (64 at 128), 57 to 64 with a
// commit a block and the warpgroups' traffic to tensor memory beside them: about 500 a block, where HBM would deliver its 8 KB
// of codes in 340.  Around it stand the launches: the first kernel takes about 3 us, the join of cut tiles 4.
//
// More tokens than a product has are further parts, on CTAs of their own, that expand and multiply all of the weights
// again: 64 tokens a part in groups of 128, 32 in groups of 64, 16 in groups of 32, where every group of a block has sums of
// its own in tensor memory, for three warpgroups.
//
// Measured, 7168 x 7168: groups of 128, 16, 32, 64, 65, 128, 256 rows: 20.4, 22.9, 28.2, 41, 42, 73 us; groups of 64, 16, 32,
// 33, 64, 128, 256 rows: 21.4, 24.6, 39, 39, 68, 120; groups of 32, 16, 17, 32, 64, 128, 256 rows: 26.4, 42, 43, 76, 139, 286.
// 64 rows, 32,768 x 2048 in groups of 128: 33 us.
//
// The blocks of all tiles form one line, divided evenly over the CTAs where that is faster than whole tiles; a tile
// that is cut leaves fp32 parts in the workspace that a last kernel adds up in order.  Every wait is bounded.
#include <cuda.h>
#include <cuda_runtime.h>

#include "linear_int4.cuh"
#include "sm100_ptx.cuh"

namespace gbmoe {
namespace linear {
namespace {

using namespace sm100;

constexpr int kGroupsOfWarps = 3;                   // warpgroups that expand
constexpr int kThreads = kGroupsOfWarps * 128 + 64;  // then the TMA warp and the product warp
constexpr int kRows = 128;
constexpr int kCodeBytes = kRows * 64;
constexpr long long kLimit = 4000000000LL;          // about 2 s of SM clocks a wait

template <int G, int MT> struct Cfg {
  static constexpr int P = 128 / G;
  static constexpr int kX = MT * 256;                            // x of a block: two halves of 64 columns
  static constexpr int kSums = (P + 1) * MT * 4 + 16;            // group sums, factors, mark
  static constexpr int kStage = (kCodeBytes + kX + kSums + 1023) / 1024 * 1024;
  static constexpr int kJoin = kRows * (MT + 1) * 4;             // sums of a tile, warpgroup after warpgroup
  static constexpr int NS = (208 * 1024 - kJoin) / kStage < 16 ? (208 * 1024 - kJoin) / kStage : 16;
  static constexpr int kSmem = 1024 + NS * kStage + kJoin + 512;
  static constexpr int kCols = 64 + P * MT;                      // tensor memory of a warpgroup: U, then a D a group
  static_assert(kGroupsOfWarps * kCols <= 512, "tensor memory");
};

struct Small {
  uint64_t full[16], empty[16];
  uint64_t u_full[kGroupsOfWarps], d_full[kGroupsOfWarps], turn[kGroupsOfWarps], gate, drain;
  uint32_t tmem;
  int abort;
};

// D[tmem] (+)= A[tmem] * B[smem]; one thread issues.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// Row of weights that row r of a tile stands for (past the last one where the tile is ragged).
__device__ __forceinline__ long long weight_row(const LinearArgs& a, int tile, int r) {
  return a.gated ? static_cast<long long>(r < 64 ? 0 : a.N) + tile * 64LL + (r & 63) : tile * 128LL + r;
}

__device__ __forceinline__ void store(const LinearArgs& a, int m, int n, float v) {
  const long long at = m * a.ldy + n;
  if (a.bf16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(a.y)[at] = __float2half_rn(v);
}

template <int G, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx) {
  using C = Cfg<G, MT>;
  constexpr int P = C::P, NS = C::NS;
  extern __shared__ unsigned char raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
  float* join = reinterpret_cast<float*>(base + NS * C::kStage);  // [row][MT + 1]
  Small& sm = *reinterpret_cast<Small*>(base + NS * C::kStage + C::kJoin);
  static_assert(sizeof(Small) <= 512 && C::kJoin % 16 == 0, "shared memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nblk = (a.K + 127) / 128, m0 = blockIdx.y * MT, live_m = min(MT, a.M - m0);
  const int tile_rows = a.gated ? 64 : 128;
  const long long total = static_cast<long long>((a.N + tile_rows - 1) / tile_rows) * nblk;
  const long long first = blockIdx.x * a.chunk, end = first + a.chunk < total ? first + a.chunk : total;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) { mbar_init(&sm.full[i], 1); mbar_init(&sm.empty[i], 4); }
    for (int i = 0; i < kGroupsOfWarps; ++i) { mbar_init(&sm.u_full[i], 128); mbar_init(&sm.d_full[i], 1); mbar_init(&sm.turn[i], 128); }
    mbar_init(&sm.gate, 128);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == kGroupsOfWarps * 4 + 1) tmem_alloc(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = sm.tmem;
  volatile int* abort = &sm.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort, a.status, kLimit); };

  if (warp < kGroupsOfWarps * 4) {
    // ---------------------------------------------------------------- expand, and take the sums back
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t u_tm = tmem + lanes + wg * C::kCols, d_tm = u_tm + 64;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    int n = 0, done = 0, piece = 0, wholes = 0;  // blocks of the CTA, blocks of this warpgroup, pieces, whole gated tiles
    bool fine = true;
    const int groups = a.K / G;
    for (long long pos = first; pos < end && fine; ++piece) {
      const int tile = static_cast<int>(pos / nblk), b0 = static_cast<int>(pos - static_cast<long long>(tile) * nblk);
      const int b1 = static_cast<int>(end - pos < nblk - b0 ? b0 + (end - pos) : nblk);
      pos += b1 - b0;
      const long long wr = min(weight_row(a, tile, row), (a.gated ? 2LL : 1LL) * a.N - 1);
      const float* scale = a.scale + wr * groups;
      float acc[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = 0.f;
      for (int b = b0; b < b1; ++b, ++n) {
        if (n % kGroupsOfWarps != wg) continue;
        float s[P];
#pragma unroll
        for (int p = 0; p < P; ++p) s[p] = b * P + p < groups ? __ldg(scale + b * P + p) : 0.f;
        const int st = n % NS;
        if (!(fine = warp_wait(&sm.full[st], (n / NS) & 1))) break;
        const unsigned char* stage = base + st * C::kStage;
        const float* sums = reinterpret_cast<const float*>(stage + kCodeBytes + C::kX);
        bool odd = false;
#pragma unroll
        for (int i = 0; i < MT / 16; ++i) odd |= i * 16 < live_m && sums[(P + 1) * MT + i] != 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 bytes, 32 codes, 16 columns of U
          const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t u[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t q[4];
            expand8(w[j], q);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[j * 4 + i] = q[i];
          }
          if (odd) {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = unbias2(u[i], i & 1 ? 0x00800080u : 0x00080008u);
          }
          tmem_st16(u_tm + c * 16, u);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.u_full[wg]);
        if (!(fine = warp_wait(&sm.d_full[wg], done & 1))) break;
        ++done;
        tc_fence_after();
        // (the stage is the warpgroup's until it says so: its sums are still to be read)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int c = 0; c < MT; c += 16) {
            uint32_t d[16];
            tmem_ld16(d_tm + p * MT + c, d);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 f = *reinterpret_cast<const float4*>(sums + P * MT + c + i);
              float4 k = *reinterpret_cast<const float4*>(sums + p * MT + c + i);
              if (odd) k = make_float4(0.f, 0.f, 0.f, 0.f);
              acc[c + i] = fmaf(s[p], (__uint_as_float(d[i]) + k.x) * f.x, acc[c + i]);
              acc[c + i + 1] = fmaf(s[p], (__uint_as_float(d[i + 1]) + k.y) * f.y, acc[c + i + 1]);
              acc[c + i + 2] = fmaf(s[p], (__uint_as_float(d[i + 2]) + k.z) * f.z, acc[c + i + 2]);
              acc[c + i + 3] = fmaf(s[p], (__uint_as_float(d[i + 3]) + k.w) * f.w, acc[c + i + 3]);
            }
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);
      }
      if (!fine) break;
      // ---- the warpgroups' sums in turn: 0 writes, 1 adds, 2 adds and writes the result
      float* mine = join + row * (MT + 1);
      if (wg == 0) {
        if (piece > 0 && !(fine = warp_wait(&sm.turn[kGroupsOfWarps - 1], (piece - 1) & 1))) break;
#pragma unroll
        for (int i = 0; i < MT; ++i) mine[i] = acc[i];
      } else {
        if (!(fine = warp_wait(&sm.turn[wg - 1], piece & 1))) break;
#pragma unroll
        for (int i = 0; i < MT; ++i) mine[i] += acc[i];
      }
      if (wg < kGroupsOfWarps - 1) {
        mbar_arrive(&sm.turn[wg]);
        continue;
      }
      const bool whole = b0 == 0 && b1 == nblk;
      if (whole && !a.gated) {
        const int nrow = tile * 128 + row;
        if (nrow < a.N)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (m < live_m) store(a, m0 + m, nrow, mine[m] * 4096.f);
      } else if (whole) {
        // gate and up rows meet: the last warpgroup's rows are complete once all of its threads have added
        mbar_arrive(&sm.gate);
        if (!(fine = warp_wait(&sm.gate, wholes++ & 1))) break;
        const int nrow = tile * 64 + (row & 63);
        if (nrow < a.N) {
          const float* gate = join + (row & 63) * (MT + 1);
          const float* up = gate + 64 * (MT + 1);
          for (int m = row >> 6; m < live_m; m += 2) store(a, m0 + m, nrow, silu_f32(gate[m] * 4096.f) * (up[m] * 4096.f));
        }
      } else {
        const long long slot = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 + (b0 == 0 ? 1 : 0);
        float* dst = a.part + slot * (kRows * MT) + row;
#pragma unroll
        for (int m = 0; m < MT; ++m) dst[m * kRows] = mine[m];
      }
      mbar_arrive(&sm.turn[wg]);
    }
  } else if (warp == kGroupsOfWarps * 4) {
    // ---------------------------------------------------------------- loads
    {
      int n = 0;
      bool fine = true;
      int tile = static_cast<int>(first / nblk), b = static_cast<int>(first - static_cast<long long>(tile) * nblk);
      for (long long pos = first; pos < end; ++pos, ++n) {
        const int st = n % NS;
        if (!(fine = __all_sync(0xffffffffu, wait(&sm.empty[st], ((n / NS) & 1) ^ 1)) != 0)) break;
        unsigned char* stage = base + st * C::kStage;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], kCodeBytes + C::kX + C::kSums);
        __syncwarp();
        if (lane < 2) {  // 64 rows each
          const int row = a.gated ? lane * a.N + tile * 64 : tile * 128 + lane * 64;
          tma_load_2d(stage + lane * 64 * 64, &mw, &sm.full[st], b * 64, row);
        } else if (lane == 2) {
          tma_load_3d(smem_addr(stage + kCodeBytes), &mx, &sm.full[st], 0, m0, b * 2);
        } else if (lane == 3) {
          bulk_load(smem_addr(stage + kCodeBytes + C::kX),
                    a.sums + (static_cast<long long>(b) * gridDim.y + blockIdx.y) * ((P + 1) * MT + 4), C::kSums, &sm.full[st]);
        }
        if (++b == nblk) { b = 0; ++tile; }
      }
      if (!fine && lane == 0) {  // copies on their way land before the CTA goes
        int none = 0;
        for (int t = max(0, n - NS); t < n; ++t) mbar_wait(&sm.full[t % NS], (t / NS) & 1, &none, nullptr, kLimit);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t id = idesc_f16_f32(128, MT);
      const int count = static_cast<int>(end > first ? end - first : 0);
      bool fine = true;
      for (int n = 0; n < count; ++n) {
        const int wg = n % kGroupsOfWarps, st = n % NS;
        if (!(fine = wait(&sm.u_full[wg], (n / kGroupsOfWarps) & 1) && wait(&sm.full[st], (n / NS) & 1))) break;
        tc_fence_after();
        const uint32_t x = smem_addr(base + st * C::kStage + kCodeBytes), u = tmem + wg * C::kCols;
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 columns: 8 of U, 32 bytes of x's rows
          umma_f16_ts(u + 64 + (k * 16 / G) * MT, u + k * 8, sw128_kmajor_desc(x + (k >> 2) * (C::kX / 2) + (k & 3) * 32), id,
                      k * 16 % G != 0);
        umma_commit(&sm.d_full[wg]);
      }
      if (!fine) {
        int none = 0;
        umma_commit(&sm.drain);
        mbar_wait(&sm.drain, 0, &none, nullptr, kLimit);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kGroupsOfWarps * 4 + 1) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the parts of the tiles that were cut, in order: four neighbouring rows of a token a thread.
template <int MT>
__global__ void __launch_bounds__(128) linear_join_kernel(const __grid_constant__ LinearArgs a, int ctas) {
  pdl_trigger();
  pdl_wait();
  const int nblk = (a.K + 127) / 128, tile = blockIdx.x, m0 = blockIdx.y * MT, live_m = min(MT, a.M - m0);
  const long long s = static_cast<long long>(tile) * nblk, e = s + nblk;
  const int c0 = static_cast<int>(s / a.chunk), c1 = static_cast<int>((e - 1) / a.chunk);
  if (c0 == c1) return;
  const int quads = a.gated ? 16 : 32, i = blockIdx.z * 128 + threadIdx.x;
  const int row = i % quads * 4, m = i / quads;
  if (m >= live_m) return;
  auto sum = [&](int r) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const long long slot = (static_cast<long long>(blockIdx.y) * ctas + c) * 2 + (c > c0 ? 0 : 1);
      const float4 p = *reinterpret_cast<const float4*>(a.part + slot * (kRows * MT) + m * kRows + r);
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    return v;
  };
  const float4 v = sum(row);
  const float y[4] = {v.x * 4096.f, v.y * 4096.f, v.z * 4096.f, v.w * 4096.f};
  float up[4] = {};
  if (a.gated) {
    const float4 u = sum(row + 64);
    up[0] = u.x * 4096.f; up[1] = u.y * 4096.f; up[2] = u.z * 4096.f; up[3] = u.w * 4096.f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = tile * quads * 4 + row + j;
    if (n < a.N) store(a, m0 + m, n, a.gated ? silu_f32(y[j]) * up[j] : y[j]);
  }
}

template <int G, int MT>
cudaError_t launch(LinearArgs a, const WidePlan& p, cudaStream_t s) {
  using C = Cfg<G, MT>;
  CUtensorMap mw, mx;
  const int nblk = (a.K + 127) / 128;
  if (!encode_tmap_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w, static_cast<uint64_t>(a.K) / 2, static_cast<uint64_t>(a.N) * (a.gated ? 2 : 1),
                      64, 64, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_tmap_halves(&mx, a.xf, nblk * 2, a.tokens, MT))
    return cudaErrorInvalidValue;
  a.chunk = p.chunk;
  auto kern = linear_tc_kernel<G, MT>;
  cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), C::kSmem);
  if (err != cudaSuccess) return err;
  err = launch_kernel(kern, dim3(p.ctas, p.parts), dim3(kThreads), C::kSmem, s, true, a, mw, mx);
  if (err != cudaSuccess || !p.cut) return err;
  const int tiles = (a.N + (a.gated ? 63 : 127)) / (a.gated ? 64 : 128);
  const int z = (a.M < MT ? a.M : MT) * (a.gated ? 16 : 32);
  return launch_kernel(linear_join_kernel<MT>, dim3(tiles, p.parts, (z + 127) / 128), dim3(128), 0, s, true, a, p.ctas);
}

}  // namespace

WidePlan wide_plan(int M, int N, int K, int group, int gated, int sms) {
  WidePlan p;
  // tokens of a product: what 512 columns of tensor memory hold for three warpgroups
  const int most = group == 128 ? 64 : group == 64 ? 32 : 16;
  p.mt = M <= 16 || most == 16 ? 16 : M <= 32 || most == 32 ? 32 : 64;
  p.parts = (M + p.mt - 1) / p.mt;
  const long long tiles = (N + (gated ? 63LL : 127LL)) / (gated ? 64 : 128), nblk = (K + 127) / 128, total = tiles * nblk;
  const int per = sms / p.parts > 0 ? sms / p.parts : 1;  // CTAs of one part of the tokens
  // whole tiles, or the line divided evenly (a last kernel then joins the cut tiles: about 8 blocks' time)
  const long long whole = (tiles + per - 1) / per * nblk, even = (total + per - 1) / per;
  p.cut = even + 8 < whole;
  p.chunk = p.cut ? even : whole;
  p.ctas = static_cast<int>((total + p.chunk - 1) / p.chunk);
  p.part_bytes = p.cut ? static_cast<size_t>(p.parts) * p.ctas * 2 * kRows * p.mt * 4 : 0;
  return p;
}

cudaError_t launch_wide_tc(const LinearArgs& a, int group, const WidePlan& p, cudaStream_t s) {
  if (group == 128) return p.mt == 16 ? launch<128, 16>(a, p, s) : p.mt == 32 ? launch<128, 32>(a, p, s) : launch<128, 64>(a, p, s);
  if (group == 64) return p.mt == 16 ? launch<64, 16>(a, p, s) : launch<64, 32>(a, p, s);
  return launch<32, 16>(a, p, s);
}

}  // namespace linear
}  // namespace gbmoe
