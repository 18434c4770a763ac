// Tree attention for wide trees: the same sums as tree_attention.cu on the 5th-generation tensor cores.
//
// A tree of many nodes times the query heads of a KV head gives more rows than warp MMA keeps up with: at
// 64 nodes and 16 heads a cache slot of one KV head takes part in 1024 products, and the tensor cores bound the call
// (4 * rows * D operations per slot and KV head against 4 * D bytes).
//
// A CTA owns 256 rows as two products of 128 rows, i = 0 and 1, and walks over its range of 128-slot tiles:
//   S_i = Q_i K^T (tcgen05.mma, both operands in shared memory, fp32 in tensor memory)
//   P_i = 2^(S_i * scale - m_i), one thread a row, written back over S_i as 16-bit values
//   O_i += P_i V (P_i from tensor memory, V from shared memory with its rows as the K dimension)
// The products of one i run while the other's softmax does.  Tensor memory holds S_0, S_1, O_0, O_1 (4 x 128
// columns for D = 128).  Roles: 2 x 4 softmax warps, one thread that issues the products, and the loaders: where pages
// hold a multiple of 8 slots one warp whose lanes each bring a page's part of a tile by TMA, else 4 warps with
// cp.async, slot by slot (any page size and stride).  The latter spend about 4,600 cycles on the instructions of a
// tile, twice what its products take; the TMA loader is not seen.
//
// Over a cache of 8-bit codes (tree_attention_fp8.cu has the mathematics) the loaders' warps bring codes by cp.async to the
// rows of a tile where they are needed, a tile ahead, and turn them into fp16 in place, which is exact; the products are those
// of fp16.  The softmax takes three numbers a slot from shared memory: the key's scale, log2 of the value's, and the power of
// two that takes that off again.  Two documents of 50,003 to 65,536 slots, 64 nodes, 64 / 4 heads of 128: 390 us = 622 TFLOP/s.
// There a chain bounds it, not a number of instructions (40% of the issue slots are used): a tile's softmax, the whole of its P,
// the second product, and the next S, which takes P's place.  With a quarter of the softmax left out the time falls by 46 us, with
// three quarters by 139, without the loaders' conversions not at all.  Reading the codes back (61 us) and attending to them in
// 16 bits (246) would take 305 us.  Lanes with four rows and a quarter of the slots each, which read a quarter of the scales, take 411 us; two numbers a
// slot, with the largest weight looked at after the exponentials, 557, and once a tile instead of every 32 slots 445.
//
// CTAs whose row tiles belong to the same cache range (up to 4) walk over it side by side, so that HBM delivers it
// once and L2 the rest.  Every wait is bounded: a role that gives up marks the CTA and all leave.
//
// Measured: two documents of 100,003 to 131,072 slots, 64 nodes, 64 / 4 heads of 128: 451 us = 1074 TFLOP/s; 16 sequences of
// 2000 slots, 64 nodes, 64 / 8 heads: 126 us (pages of 12 slots, by cp.async: 159).  A tile of 128 slots takes about 4,300
// cycles.  Its 32 products take 2,048 of them (the products' pipe is active for 47%) and a softmax of 128 rows 1,400, but the
// thread that issues the products is inside their instructions for 3,450.  The products' form is not why: by themselves, back
// to back, those of 128 x 128 x 16 take 64 cycles each, with the first operand in shared memory or in tensor memory, into one
// accumulator or two, in this kernel's order or in turn, and with the softmax warps' traffic to tensor memory beside them.
// Shared memory is at 34% of its rate.  What keeps them apart in here has not been found.
#include <cuda.h>
#include <cuda_runtime.h>

#include "tree_attention.cuh"

namespace gbmoe {
namespace tree {
namespace {

using namespace sm100;

// 8 softmax warps, the loaders (4 warps; over codes 4 for the keys and 4 for the values), and the warp that issues products
// among 4
template <bool Q8> constexpr int kThreads = Q8 ? 640 : 512;
constexpr long long kLimit = 4000000000LL;  // about 2 s of SM clocks a wait

template <int D> struct WideCfg {
  static constexpr int NS = D == 128 ? 2 : 4;          // stages of K and of V
  static constexpr int LAG = D == 128 ? 2 : 4;         // loads in flight behind the newest
  static constexpr int kTileBytes = 128 * D * 2;       // Q_i, K or V of 128 rows
  static constexpr int kData = (2 + 2 * NS) * kTileBytes;
  static constexpr int kSmall = 1024;                  // barriers, masks, marks
};
// What the softmax takes of the slots of 2 NS tiles, and of its rows (caches of codes).
template <int D> struct Scales {
  float key[2 * WideCfg<D>::NS][128], value[2 * WideCfg<D>::NS][128], back[2 * WideCfg<D>::NS][128];
  float frame[kWideRows];
};
template <int D, bool Q8> size_t wide_smem(int B) {
  return 1024 + WideCfg<D>::kData + WideCfg<D>::kSmall + (Q8 ? sizeof(Scales<D>) : 0) + (2 * static_cast<size_t>(B) + 1 + kThreads<Q8> / 32) * 8;
}

struct Small {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], q_full, o_full, drain;
  unsigned long long odd[2];
  alignas(16) uint32_t ok[8][4];  // visible slots of a tile, 32 a word
  uint32_t tmem;
  int abort, bad_pages;
  DeviceStatus status;
};
static_assert(sizeof(Small) <= 1024, "small area");

// Descriptor of a K = 16 step of V: slots are the K dimension, elements of D contiguous (64 of them a 128-byte
// swizzled row, the next 64 one half tile further).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(half_bytes >> 4) << 16;  // next 64 elements
  d |= static_cast<uint64_t>(1024 >> 4) << 32;        // next 8 slots
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;                // 128-byte swizzle
  return d;
}
// Instruction descriptor of kind::f16: fp32 D, A and B both bf16 or both fp16, A K-major.
__device__ __forceinline__ uint32_t idesc_16(bool bf16, bool b_mn, int M, int N) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]; one thread issues.
__device__ __forceinline__ void umma_16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two floats in one register pair: GB300's fp32 units take two at once.
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpack2(uint64_t p, uint32_t& a, uint32_t& b) { asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Visible slots among 32 from `first` on: the loaded ones, committed or with their bit in `bits`.
__device__ __forceinline__ uint32_t visible(uint32_t ok, int first, int ctx, unsigned long long bits) {
  const int d = ctx - first;  // place of node 0
  if (d >= 32) return ok;
  if (d > 0) return ok & (((1u << d) - 1) | static_cast<uint32_t>(bits << d));
  return d <= -64 ? 0u : ok & static_cast<uint32_t>(bits >> -d);
}

// T: type of q and out.  Q8: the caches hold 8-bit codes and the products are fp16.
template <typename T, int D, bool TMA, bool Q8>
__global__ void __launch_bounds__(kThreads<Q8>, 1)
    tree_wide_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = WideCfg<D>;
  constexpr int CH = D / 8, HALF = 128 * 128;  // 16-byte chunks of a row; bytes of 64 columns of a tile
  extern __shared__ unsigned char raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
  unsigned char* qs = base;                                   // [2] tiles
  unsigned char* ks = qs + 2 * C::kTileBytes;                 // [NS]
  unsigned char* vs = ks + C::NS * C::kTileBytes;             // [NS]
  Small& sm = *reinterpret_cast<Small*>(base + C::kData);
  Scales<D>& sc = *reinterpret_cast<Scales<D>*>(base + C::kData + C::kSmall);  // (Q8)
  long long* prefix = reinterpret_cast<long long*>(base + C::kData + C::kSmall + (Q8 ? sizeof(Scales<D>) : 0));
  int2* sizes = reinterpret_cast<int2*>(prefix + a.B + 1 + kThreads<Q8> / 32);  // [B]
  constexpr int kIssuer = kThreads<Q8> / 32 - 4;  // the warp that issues products
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  using P = typename std::conditional<Q8, __half, T>::type;  // of the products' operands
  constexpr bool kBf16 = std::is_same<P, __nv_bfloat16>::value;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sm.k_full[i], TMA ? 1 : 128);
      mbar_init(&sm.v_full[i], TMA ? 1 : 128);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 2);  // the products, and the issuing thread (which has seen the loaders' masks)
      mbar_init(&sm.p_full[i], 128);
      sm.odd[i] = 0;
    }
    mbar_init(&sm.q_full, 256);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    sm.bad_pages = 0;
    sm.status.bad_ids = sm.status.flags = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) tmem_alloc(&sm.tmem, 512);
  pdl_wait();
  int bad_plan;
  plan_line<kThreads<Q8>>(a, prefix, sizes, prefix + a.B + 1, &bad_plan);  // (its barriers also publish the set-up above)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int* abort = &sm.abort;
  // a bounded wait of a whole warp: true for all of its lanes or for none
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, &sm.status, kLimit)) != 0;
  };
  const int rank = blockIdx.x % a.ranks, grp = blockIdx.x / a.ranks, groups = gridDim.x / a.ranks;
  const long long total = prefix[a.B], chunk = (total + groups - 1) / groups;
  if (blockIdx.x == 0) {
    bad_plan = __syncthreads_count(bad_plan);
    if (tid == 0) { a.header[0] = gridDim.x; a.header[1] = bad_plan; a.prefix[a.B + 1] = chunk; }
    for (int b = tid; b <= a.B; b += kThreads<Q8>) a.prefix[b] = prefix[b];
  }
  const long long first = grp * chunk, end = first + chunk < total ? first + chunk : total;
  const float scale = fmaxf(fabsf(a.scale_log2), 1e-30f);  // its sign goes into Q; 0 would make 0 * inf of hidden slots
  const bool negate = a.scale_log2 < 0.f;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax: one thread a row
    regs_inc<Q8 ? 152 : 192>();
    const int i = warp >> 2, r_in = tid & 127, row0 = warp * 32;  // row0: the warp's first row
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 * (warp % 4) in the lane field
    const uint32_t s_tm = tmem + lanes + i * 128, o_tm = tmem + lanes + 256 + i * D;
    int n = 0, piece = 0, done = 0;  // tiles of the CTA, pieces, tiles of this half
    for (long long pos = first; pos < end;) {
      const Piece u = piece_at(a, prefix, sizes, pos, end, rank);
      pos += u.places;
      if (u.rows == 0) continue;
      const int row = i * 128 + r_in;
      const bool mine = i == 0 || u.rows > 128;  // has this half any row?
      // Q_i into shared memory, every warp its own 32 rows (rows past the last one repeat it: nothing
      // is taken from them), without a branch around the loads, so that all are under way at once
      if (mine) {
        constexpr int B = 8;
#pragma unroll 1
        for (int x = 0; x < CH; x += B) {
          uint4 v[B];
#pragma unroll
          for (int k = 0; k < B; ++k) {
            const int c = (x + k) * 32 + lane, r = u.row0 + min(row0 + c / CH, u.rows - 1), ch = c % CH;
            const int node = div_by(r, a.group), hq = u.head * a.group.d + (r - node * a.group.d);
            v[k] = ld_v4(static_cast<const T*>(a.q) + (u.node0 + node) * a.q_t + hq * a.q_h + ch * 8);
          }
          if constexpr (Q8) {
#pragma unroll
            for (int k = 0; k < B; ++k) {
              const int c = (x + k) * 32 + lane;
              float mul = a.scale_log2;
              if constexpr (std::is_same<T, __nv_bfloat16>::value) {  // as fp16 in the row's frame
                uint32_t* w = reinterpret_cast<uint32_t*>(&v[k]);
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 f = Elem<T>::unpack(w[j]);
                  top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
#pragma unroll
                for (int o = CH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = x_frame_exp(top);
                const float to = exp2i(-e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 f = Elem<T>::unpack(w[j]);
                  w[j] = pack_half2(f.x * to, f.y * to);
                }
                mul *= exp2i(e);
              }
              if (c % CH == 0) sc.frame[row0 + c / CH] = mul;
            }
            __syncwarp();
          }
#pragma unroll
          for (int k = 0; k < B; ++k) {
            const int c = (x + k) * 32 + lane, r = (row0 & 127) + c / CH, ch = c % CH;
            if (!Q8 && negate) { v[k].x ^= 0x80008000u; v[k].y ^= 0x80008000u; v[k].z ^= 0x80008000u; v[k].w ^= 0x80008000u; }
            *reinterpret_cast<uint4*>(qs + i * C::kTileBytes + (ch >> 3) * HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v[k];
          }
        }
      }
      if (tid == 0) sm.odd[piece & 1] = 0;
      fence_proxy_async_smem();
      tc_fence_before();  // O_i of the last piece has been read
      mbar_arrive(&sm.q_full);
      unsigned long long bits = 0;
      if (row < u.rows) {
        const int node = div_by(u.row0 + row, a.group);
        bits = a.mask ? a.mask[u.node0 + node] : (2ull << node) - 1;
      }
      float m = -INFINITY, l = 0.f;
      const float row_mul = Q8 && mine ? sc.frame[row] : 0.f;
      bool fine = true;
      for (int it = u.k0; it < u.k1; ++it, ++n) {
        if (!mine) continue;
        if (!(fine = warp_wait(&sm.s_full[i], done & 1))) break;
        ++done;
        tc_fence_after();
        const int slot0 = it * 128;
        if constexpr (Q8) {
          // 32 slots at a time (their scales make more numbers than registers hold for 128): should the reference move, what
          // of the tile has been written before moves with O
          const int sn = n % (2 * C::NS);
          const uint4 okw = *reinterpret_cast<const uint4*>(sm.ok[n & 7]);
          const uint32_t oks[4] = {okw.x, okw.y, okw.z, okw.w};
          const uint64_t row2 = pack2(row_mul, row_mul);
          uint32_t sr[2][32];
          tmem_ld32(s_tm, sr[0]);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t (&s)[32] = sr[c & 1];
            tmem_ld_wait();
            if (c < 3) tmem_ld32(s_tm + (c + 1) * 32, sr[(c + 1) & 1]);
            uint64_t e[16];
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const ulonglong2 key = *reinterpret_cast<const ulonglong2*>(&sc.key[sn][c * 32 + k]);
              const ulonglong2 value = *reinterpret_cast<const ulonglong2*>(&sc.value[sn][c * 32 + k]);
              e[k / 2] = fma2(mul2(pack2u(s[k], s[k + 1]), key.x), row2, value.x);
              e[k / 2 + 1] = fma2(mul2(pack2u(s[k + 2], s[k + 3]), key.y), row2, value.y);
            }
            if (oks[c] != 0xffffffffu || slot0 + c * 32 + 32 > u.ctx) {
              const uint32_t vis = visible(oks[c], slot0 + c * 32, u.ctx, bits);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                uint32_t x, y;
                unpack2(e[k], x, y);
                e[k] = pack2u((vis >> (2 * k)) & 1 ? x : 0xff800000u, (vis >> (2 * k + 1)) & 1 ? y : 0xff800000u);
              }
            }
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              uint32_t x, y;
              unpack2(e[k], x, y);
              top = max3(top, __uint_as_float(x), __uint_as_float(y));
            }
            const bool grow = top > m + kLazy;  // (from -infinity: any number is)
            if (__any_sync(0xffffffffu, grow)) {
              const float nm = grow ? top : m, f = grow ? ex2(m - nm) : 1.f;
              m = nm;
              l *= f;
              const uint64_t f2 = pack2(f, f);
              sum[0] = mul2(sum[0], f2);
              sum[1] = mul2(sum[1], f2);
              if (c > 0) tmem_st_wait();
#pragma unroll 1
              for (int z = 0; z < c; ++z) {
                uint32_t p[16];
                tmem_ld16(s_tm + z * 16, p);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const float2 x = Elem<__half>::unpack(p[k]);
                  p[k] = pack_half2(x.x * f, x.y * f);
                }
                tmem_st16(s_tm + z * 16, p);
              }
              if (it > u.k0) {  // O_i holds something: all products up to S_i have completed
#pragma unroll 1
                for (int z = 0; z < D / 16; ++z) {
                  uint32_t o[16];
                  tmem_ld16(o_tm + z * 16, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st16(o_tm + z * 16, o);
                }
              }
            }
            const float ref = (m == -INFINITY ? 0.f : m) - kHeadroom<__half>;
            const uint64_t ref2 = pack2(-ref, -ref);
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const ulonglong2 back = *reinterpret_cast<const ulonglong2*>(&sc.back[sn][c * 32 + 2 * k]);
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                uint32_t x, y;
                unpack2(add2(e[k + z], ref2), x, y);
                const float wx = ex2(__uint_as_float(x)), wy = ex2(__uint_as_float(y));
                sum[z] = fma2(pack2(wx, wy), z ? back.y : back.x, sum[z]);
                p[k + z] = pack_half2(wx, wy);
              }
            }
            tmem_st16(s_tm + c * 16, p);
          }
          uint32_t x[4];
          unpack2(sum[0], x[0], x[1]);
          unpack2(sum[1], x[2], x[3]);
          l += (__uint_as_float(x[0]) + __uint_as_float(x[1])) + (__uint_as_float(x[2]) + __uint_as_float(x[3]));
        }
        if constexpr (!Q8) {
          uint32_t sr[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + c * 32, sr[c]);
          tmem_ld_wait();
          const uint4 okw = *reinterpret_cast<const uint4*>(sm.ok[n & 7]);
          const uint32_t oks[4] = {okw.x, okw.y, okw.z, okw.w};
          if ((okw.x & okw.y & okw.z & okw.w) != 0xffffffffu || slot0 + 128 > u.ctx) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t vis = visible(oks[c], slot0 + c * 32, u.ctx, bits);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1)) sr[c][e] = 0xff800000u;  // -inf
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = __uint_as_float(sr[c][0]);
#pragma unroll
            for (int e = 1; e < 32; ++e) mx[c] = fmaxf(mx[c], __uint_as_float(sr[c][e]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
          const bool grow = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float nm = grow ? top : m, f = grow ? ex2(m - nm) : 1.f;
            m = nm;
            l *= f;
            if (it > u.k0) {  // O_i holds something: all products up to S_i have completed
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(o_tm + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(o_tm + c * 32, o);
              }
            }
          }
          const float ref = (m == -INFINITY ? 0.f : m) - kHeadroom<T>;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int c = h * 2 + (e >> 4), k = (e & 15) * 2;
              const float x = ex2(fmaf(__uint_as_float(sr[c][k]), scale, -ref)), y = ex2(fmaf(__uint_as_float(sr[c][k + 1]), scale, -ref));
              sum[e & 3] += x + y;
              p[e] = Elem<T>::pack(x, y);
            }
            tmem_st32(s_tm + h * 32, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          if (i == 0 && slot0 + 128 > u.ctx) {
            // Drafted slots are hidden from some rows: V rows with infinities or NaN are cleared here (0 * inf) and added
            // to the rows that see them at the end.
            if (!(fine = warp_wait(&sm.v_full[n % C::NS], (n / C::NS) & 1))) break;
            unsigned char* v = vs + (n % C::NS) * C::kTileBytes;
            const int lo = max(u.ctx - slot0, 0), hi = min(u.ctx + u.n - slot0, 128);
            for (int c = lo * CH + r_in; c < hi * CH; c += 128) {
              const int r = c / CH, ch = c % CH;
              const uint4 w = *reinterpret_cast<const uint4*>(v + (ch >> 3) * HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
              if (nonfinite2(T(), w.x) || nonfinite2(T(), w.y) || nonfinite2(T(), w.z) || nonfinite2(T(), w.w)) {
                atomicOr(&sm.odd[piece & 1], 1ull << (slot0 + r - u.ctx));
                for (int z = 0; z < CH; ++z)
                  *reinterpret_cast<uint4*>(v + (z >> 3) * HALF + r * 128 + ((z & 7) << 4)) = make_uint4(0, 0, 0, 0);
              }
            }
            if constexpr (TMA) {  // rows of the last page past the sequence's end hold anything
              for (int c = hi * CH + r_in; c < 128 * CH; c += 128) {
                const int r = c / CH, ch = c % CH;
                *reinterpret_cast<uint4*>(v + (ch >> 3) * HALF + r * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[i]);
      }
      if (!fine) break;
      if (!warp_wait(&sm.o_full, piece & 1)) break;
      tc_fence_after();
      if (mine) {
        // ---- the row's result
        const bool live = row < u.rows, whole = u.k0 == 0 && u.k1 == u.kt;
        const int node = div_by(u.row0 + (live ? row : 0), a.group);
        const int hq = u.head * a.group.d + (u.row0 + (live ? row : 0) - node * a.group.d);
        const long long slot = static_cast<long long>(blockIdx.x) * 2 + (u.k0 == 0 ? 1 : 0);
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const unsigned long long odd = !Q8 && live ? sm.odd[piece & 1] & bits : 0;
        const T* qr = static_cast<const T*>(a.q) + (u.node0 + node) * a.q_t + hq * a.q_h;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_tm + c * 32, o);
          tmem_ld_wait();
          if (odd) {  // rare: the cleared rows of V, from the cache
            for (unsigned long long rest = odd; rest; rest &= rest - 1) {
              const int s = u.ctx + __ffsll(static_cast<long long>(rest)) - 1, pi = div_by(s, a.page), at = s - pi * a.page.d;
              const long long page = a.table[u.b * a.table_ld + pi];
              const T* kr = static_cast<const T*>(a.kc) + page * a.k_page + at * a.k_slot + u.head * a.k_head;
              const T* vr = static_cast<const T*>(a.vc) + page * a.v_page + at * a.v_slot + u.head * a.v_head;
              float dot = 0.f;
              for (int d = 0; d < D; ++d) dot = fmaf(Elem<T>::to_float(qr[d]), Elem<T>::to_float(kr[d]), dot);
              const float pk = ex2(fmaf(negate ? -dot : dot, scale, kHeadroom<T> - (m == -INFINITY ? 0.f : m)));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(fmaf(pk, Elem<T>::to_float(vr[c * 32 + e]), __uint_as_float(o[e])));
            }
          }
          if (whole) {
            if (live) {
              T* dst = static_cast<T*>(a.out) + (u.node0 + node) * a.o_t + hq * a.o_h + c * 32;
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint2*>(dst + e) = make_uint2(Elem<T>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                                                                Elem<T>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv));
            }
          } else {  // parts leave in whole lines, through the 4 KB of the warp's rows of Q_i
            unsigned char* turn = qs + i * C::kTileBytes + (row0 & 127) * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(turn + lane * 128 + ((e ^ (lane & 7)) << 4)) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = k * 4 + (lane >> 3), e = lane & 7;
              if (row0 + r < u.rows)
                *reinterpret_cast<uint4*>(a.part_o + (slot * a.rows + row0 + r) * D + c * 32 + e * 4) =
                    *reinterpret_cast<const uint4*>(turn + r * 128 + ((e ^ (r & 7)) << 4));
            }
            __syncwarp();
          }
        }
        if (live && !whole) *reinterpret_cast<float2*>(a.part_ml + (slot * a.rows + row) * 2) = make_float2(m, l);
      }
      ++piece;
    }
  } else if (warp < kIssuer) {
    // ---------------------------------------------------------------- loaders
    regs_dec<64>();
    if constexpr (Q8) {
      // A warp's 32 slots of the keys, or of the values, of a tile: codes by cp.async into their own rows of the tile (a tile
      // ahead), from there through registers, and back as fp16.  Codes of row r stand in the upper half of the columns (D = 64:
      // in the half of the row that r & 1 says).
      constexpr int LPR = D / 16, X = LPR, RPX = 32 / LPR;  // chunks of a row; a lane's chunks; rows that are RPX apart
      const bool values = warp >= 12;
      const int lw = warp & 3, ch = lane % LPR, x0 = lane / LPR;
      unsigned char* const tiles = (values ? vs : ks) + lw * 32 * 128;  // (this warp's rows)
      uint64_t* const full = values ? sm.v_full : sm.k_full;
      uint64_t* const empty = values ? sm.v_empty : sm.k_empty;
      // where the lane's i-th chunk stands: of row i RPX + x0, whose place in a group of 8 rows is x0 (+ 4 for odd i at D = 128)
      auto code_at = [&](int i) {
        const int r = i * RPX + x0;
        return D == 128 ? HALF + r * 128 + ((ch ^ (x0 + (i & 1) * 4)) << 4) : r * 128 + ((x0 & 1) << 6) + (ch << 4);
      };
      auto to_fp16 = [&](unsigned char* tile) {
        uint4 x[X];
#pragma unroll
        for (int i = 0; i < X; ++i) x[i] = *reinterpret_cast<const uint4*>(tile + code_at(i));
        __syncwarp();
        // chunks 2 ch and 2 ch + 1; lanes whose chunks lie in the other half of the columns write them in the other order: no bank
        // conflicts
        const int swap = ch >> 2, c0 = ch * 2 + swap, half = (ch >> 2) * HALF;
#pragma unroll
        for (int i = 0; i < X; ++i) {
          const int r = i * RPX + x0, low = D == 128 ? x0 + (i & 1) * 4 : x0;
          uint4 v[2];
          e4m3x4_to_f16x4(x[i].x, v[0].x, v[0].y);
          e4m3x4_to_f16x4(x[i].y, v[0].z, v[0].w);
          e4m3x4_to_f16x4(x[i].z, v[1].x, v[1].y);
          e4m3x4_to_f16x4(x[i].w, v[1].z, v[1].w);
          unsigned char* row = tile + half + r * 128;
          *reinterpret_cast<uint4*>(row + (((c0 & 7) ^ low) << 4)) = swap ? v[1] : v[0];
          *reinterpret_cast<uint4*>(row + (((c0 & 7) ^ 1 ^ low) << 4)) = swap ? v[0] : v[1];
        }
        fence_proxy_async_smem();
      };
      // scales of slot lw * 32 + lane of the tile that is on its way, its loaded slots, and its first drafted one (keys' warps)
      float key = 0.f, value = 0.f;
      uint32_t ok = 0;
      int draft = 0, n = 0, bad = 0;
      bool fine = true, pending = false;
      const unsigned char* value_row = nullptr;  // the lane's slot's value codes
      auto finish = [&] {  // tile n - 1
        const int t = n - 1;
        if (!values) {
          bool nan = value != value;
          if (draft < 32) {
            // Drafted slots are hidden from some rows, where a NaN of a hidden value would come through as 0 * NaN: the scale of
            // such a slot, which only those rows take that see it, becomes NaN (and the values' warps clear its codes).
            if (lane >= draft && value_row)
              for (int c = 0; c < LPR; ++c) nan = nan || has_nan(__ldg(reinterpret_cast<const uint4*>(value_row) + c));
          }
          float log_v = lg2(fminf(fmaxf(value, 0x1p-64f), 0x1p64f));
          // a slot of zero values?  (as a rule the first 16 codes tell; for all slots by loads of whole rows: 454 us for 390)
          if (value == kZeroScale && value_row) {
            bool some = false;
#pragma unroll 1
            for (int c = 0; c < LPR && !some; ++c) some = not_zero(__ldg(reinterpret_cast<const uint4*>(value_row) + c));
            if (!some) log_v = kZeroCounts;
          }
          __syncwarp();
          const int sn = t % (2 * C::NS);
          sc.key[sn][lw * 32 + lane] = key;
          sc.value[sn][lw * 32 + lane] = nan ? __int_as_float(0x7fffffff) : log_v;
          sc.back[sn][lw * 32 + lane] = ex2(-log_v);
          if (lane == 0) sm.ok[t & 7][lw] = ok;
        }
        cp_wait<0>();
        __syncwarp();
        unsigned char* tile = tiles + (t % C::NS) * C::kTileBytes;
        if (values && draft < 32) {
#pragma unroll
          for (int i = 0; i < X; ++i) {
            const uint32_t odd = __ballot_sync(0xffffffffu, has_nan(*reinterpret_cast<const uint4*>(tile + code_at(i))) && i * RPX + x0 >= draft);
            if ((odd >> (x0 * LPR)) & ((1u << LPR) - 1)) *reinterpret_cast<uint4*>(tile + code_at(i)) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        to_fp16(tile);
        mbar_arrive(&full[t % C::NS]);
      };
      for (long long pos = first; pos < end && fine;) {
        const Piece u = piece_at(a, prefix, sizes, pos, end, rank);
        pos += u.places;
        if (u.rows == 0) continue;
        const int32_t* table = a.table + u.b * a.table_ld;
        const unsigned char* base_of = static_cast<const unsigned char*>(values ? a.vc : a.kc) + u.head * (values ? a.v_head : a.k_head) + ch * 16;
        const long long page_stride = values ? a.v_page : a.k_page, slot_stride = values ? a.v_slot : a.k_slot;
        const int L = u.ctx + u.n;
        int page = -1, at = 0;
        auto look_up = [&](int it) {
          const int slot = it * 128 + lw * 32 + lane;
          page = -1;
          at = 0;
          if (it < u.k1 && slot < L) {
            const int pi = div_by(slot, a.page);
            at = slot - pi * a.page.d;
            page = __ldg(table + pi);
          }
        };
        look_up(u.k0);
        for (int it = u.k0; it < u.k1; ++it) {
          const int st = n % C::NS;
          if (pending) finish();
          // this tile's place
          const bool in = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
          if (!values && !in && it * 128 + lw * 32 + lane < L) ++bad;
          const uint64_t pg = in ? static_cast<uint32_t>(page) : 0, row = static_cast<uint32_t>(at);
          const uint64_t off = pg * page_stride + row * slot_stride;
          ok = __ballot_sync(0xffffffffu, in);
          draft = u.ctx - it * 128 - lw * 32;
          if (!values) {
            key = in ? __ldg(a.ks + u.head * a.ks_head + pg * a.ks_page + row * a.ks_slot) : 0.f;
            value = in ? __ldg(a.vs + u.head * a.vs_head + pg * a.vs_page + row * a.vs_slot) : 1.f;
            value_row = in ? static_cast<const unsigned char*>(a.vc) + u.head * a.v_head + pg * a.v_page + row * a.v_slot : nullptr;
          }
          look_up(it + 1);
          if (!(fine = warp_wait(&empty[st], ((n / C::NS) & 1) ^ 1))) break;
          const uint32_t dst = smem_addr(tiles + st * C::kTileBytes);
#pragma unroll
          for (int i = 0; i < X; ++i) {
            const int r = i * RPX + x0;
            cp_async16(dst + code_at(i), base_of + __shfl_sync(0xffffffffu, off, r), (ok >> r) & 1);
          }
          cp_commit();
          pending = true;
          ++n;
        }
        if (fine && pending) finish();  // the next piece's first tile waits for all of this piece's products
        pending = false;
      }
      cp_wait<0>();
      bad = __reduce_add_sync(0xffffffffu, bad);
      if (lane == 0 && bad) atomicAdd(&sm.bad_pages, bad);
    } else if constexpr (TMA) {
      if (warp == 8) {  // lane j: the part of a tile in its j-th run of `box` slots
        int n = 0, bad = 0, k_sent = 0, v_sent = 0;
        bool fine = true;
        const int boxes = 128 / a.box;
        for (long long pos = first; pos < end && fine;) {
          const Piece u = piece_at(a, prefix, sizes, pos, end, rank);
          pos += u.places;
          if (u.rows == 0) continue;
          const int32_t* table = a.table + u.b * a.table_ld;
          const int L = u.ctx + u.n;
          for (int it = u.k0; it < u.k1 && fine; ++it, ++n) {
            int page = -1, at = 0;  // page -1 is outside the tensor: zeros
            const int slot = it * 128 + lane * a.box;
            if (lane < boxes && slot < L) {
              const int pi = div_by(slot, a.page);
              at = slot - pi * a.page.d;
              page = __ldg(table + pi);
              if (page < 0 || page >= a.pages) { page = -1; bad += min(a.box, L - slot); }
            }
            uint32_t ok[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int s = w * 32 + lane;
              ok[w] = __ballot_sync(0xffffffffu, __shfl_sync(0xffffffffu, page, s / a.box) >= 0 && it * 128 + s < L);
            }
            const int st = n % C::NS;
            const uint32_t parity = ((n / C::NS) & 1) ^ 1;
#pragma unroll
            for (int kv = 0; kv < 2 && fine; ++kv) {
              if (!(fine = warp_wait(kv ? &sm.v_empty[st] : &sm.k_empty[st], parity))) break;
              uint64_t* full = kv ? &sm.v_full[st] : &sm.k_full[st];
              if (lane == 0) {
                if (kv == 0) *reinterpret_cast<uint4*>(sm.ok[n & 7]) = make_uint4(ok[0], ok[1], ok[2], ok[3]);
                mbar_arrive_expect_tx(full, C::kTileBytes);
              }
              if (kv) ++v_sent; else ++k_sent;
              __syncwarp();
              const uint32_t dst = smem_addr((kv ? vs : ks) + st * C::kTileBytes) + lane * a.box * 128;
              if (lane < boxes)
#pragma unroll
                for (int h = 0; h < D / 64; ++h) tma_load_4d(dst + h * HALF, kv ? &mv : &mk, full, h * 64, at, u.head, page);
            }
          }
        }
        if (!fine && lane == 0) {  // copies on their way land before the CTA goes
          int none = 0;
          for (int t = max(0, k_sent - C::NS); t < k_sent; ++t) mbar_wait(&sm.k_full[t % C::NS], (t / C::NS) & 1, &none, nullptr, kLimit);
          for (int t = max(0, v_sent - C::NS); t < v_sent; ++t) mbar_wait(&sm.v_full[t % C::NS], (t / C::NS) & 1, &none, nullptr, kLimit);
        }
        bad = __reduce_add_sync(0xffffffffu, bad);
        if (lane == 0 && bad) atomicAdd(&sm.bad_pages, bad);
      }
    } else {
    const int lw = warp - 8;
    int n = 0, bad = 0, sent = 0;  // loads announced so far
    bool fine = true;
    auto arrive_load = [&](int q) {  // load q: K of tile q / 2, or its V
      fence_proxy_async_smem();
      const int t = q >> 1;
      mbar_arrive(q & 1 ? &sm.v_full[t % C::NS] : &sm.k_full[t % C::NS]);
    };
    for (long long pos = first; pos < end && fine;) {
      const Piece u = piece_at(a, prefix, sizes, pos, end, rank);
      pos += u.places;
      if (u.rows == 0) continue;
      const int32_t* table = a.table + u.b * a.table_ld;
      const T* kbase = static_cast<const T*>(a.kc) + u.head * a.k_head;
      const T* vbase = static_cast<const T*>(a.vc) + u.head * a.v_head;
      const int L = u.ctx + u.n;
      for (int it = u.k0; it < u.k1 && fine; ++it, ++n) {
        int page = -1, at = 0;
        const int slot = it * 128 + lw * 32 + lane;
        if (slot < L) {
          const int pi = div_by(slot, a.page);
          at = slot - pi * a.page.d;
          page = __ldg(table + pi);
          if (page < 0 || page >= a.pages) { page = -1; ++bad; }
        }
        const uint32_t ok = __ballot_sync(0xffffffffu, page >= 0);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t* empty = kv ? &sm.v_empty[n % C::NS] : &sm.k_empty[n % C::NS];
          const uint32_t parity = ((n / C::NS) & 1) ^ 1;
          if (!__all_sync(0xffffffffu, mbar_try_wait(empty, parity))) {
            // no room: announce all that is on its way before waiting, since the room may depend on it
            cp_wait<0>();
            for (; sent < 2 * n + kv; ++sent) arrive_load(sent);
            fine = warp_wait(empty, parity);
          }
          if (!fine) break;
          if (kv == 0 && lane == 0) sm.ok[n & 7][lw] = ok;
          const uint32_t dst = smem_addr((kv ? vs : ks) + (n % C::NS) * C::kTileBytes);
          const T* src = kv ? vbase : kbase;
          const long long ps = kv ? a.v_page : a.k_page, ss = kv ? a.v_slot : a.k_slot;
#pragma unroll 4
          for (int x = 0; x < CH; ++x) {  // 32 slots x CH chunks, 32 chunks at a time
            const int c = x * 32 + lane, r = c / CH, ch = c % CH;
            const int pg = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, at, r);
            const bool live = pg >= 0;
            const int rr = lw * 32 + r;
            cp_async16(dst + (ch >> 3) * HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                       src + (live ? pg : 0) * ps + sl * ss + ch * 8, live);
          }
          cp_commit();
          const int q = 2 * n + kv;
          if (sent <= q - C::LAG) {
            cp_wait<C::LAG>();
            for (; sent <= q - C::LAG; ++sent) arrive_load(sent);
          }
        }
      }
    }
    cp_wait<0>();
    if (fine)
      for (; sent < 2 * n; ++sent) arrive_load(sent);
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0 && bad) atomicAdd(&sm.bad_pages, bad);
    }
  } else {
    // ---------------------------------------------------------------- products: one thread issues
    regs_dec<Q8 ? 48 : 64>();  // (96 a thread at launch over codes: 61,440 = 256 * 152 + 256 * 64 + 128 * 48)
    if (warp == kIssuer && lane == 0) {
      const uint32_t id_s = idesc_16(kBf16, false, 128, 128), id_o = idesc_16(kBf16, true, 128, D);
      const uint32_t q_s = smem_addr(qs), k_s = smem_addr(ks), v_s = smem_addr(vs);
      int n = 0, piece = 0, done[2] = {0, 0};
      bool fine = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort, &sm.status, kLimit); };
      auto score = [&](int i, int t) {  // S_i of tile t (its K has arrived)
        const uint32_t kb = k_s + (t % C::NS) * C::kTileBytes, qb = q_s + i * C::kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * HALF + (k & 3) * 32;
          umma_f16(tmem + i * 128, sw128_kmajor_desc(qb + off), sw128_kmajor_desc(kb + off), id_s, k > 0);
        }
        umma_commit(&sm.s_full[i]);
        mbar_arrive(&sm.s_full[i]);
      };
      for (long long pos = first; pos < end && fine;) {
        const Piece u = piece_at(a, prefix, sizes, pos, end, rank);
        pos += u.places;
        if (u.rows == 0) continue;
        const int nq = u.rows > 128 ? 2 : 1, T0 = n, T1 = n + (u.k1 - u.k0);
        fine = wait(&sm.q_full, piece & 1) && wait(&sm.k_full[n % C::NS], (n / C::NS) & 1);
        if (!fine) break;
        tc_fence_after();
        for (int i = 0; i < nq; ++i) score(i, n);
        umma_commit(&sm.k_empty[n % C::NS]);
        for (; n < T1; ++n) {
          if (!(fine = wait(&sm.v_full[n % C::NS], (n / C::NS) & 1))) break;
          const bool more = n + 1 < T1;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i >= nq || !fine) break;
            if (!(fine = wait(&sm.p_full[i], done[i]++ & 1))) break;
            tc_fence_after();
            const uint32_t vb = v_s + (n % C::NS) * C::kTileBytes;
#pragma unroll
            for (int k = 0; k < 8; ++k)  // 16 slots a product: 8 columns of P, 16 rows of V
              umma_16_ts(tmem + 256 + i * D, tmem + i * 128 + k * 8, sw128_mnmajor_desc(vb + k * 2048, HALF), id_o, n > T0 || k > 0);
            if (i == nq - 1) umma_commit(&sm.v_empty[n % C::NS]);
            if (more) {
              if (i == 0 && !(fine = wait(&sm.k_full[(n + 1) % C::NS], ((n + 1) / C::NS) & 1))) break;
              tc_fence_after();
              score(i, n + 1);
              if (i == nq - 1) umma_commit(&sm.k_empty[(n + 1) % C::NS]);
            }
          }
          if (!fine) break;
        }
        if (!fine) break;
        umma_commit(&sm.o_full);
        ++piece;
      }
      if (!fine) {  // what has been issued ends before the memory it works on goes
        int none = 0;
        umma_commit(&sm.drain);
        mbar_wait(&sm.drain, 0, &none, nullptr, kLimit);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) a.header[2 + blockIdx.x] = sm.abort ? -1 : sm.bad_pages;
}

template <typename T, int D>
cudaError_t launch(TreeArgs a, int ctas, cudaStream_t s) {
  CUtensorMap mk{}, mv{};
  tree_boxes(a, D, 128, &mk, &mv);
  auto kern = a.box ? tree_wide_kernel<T, D, true, false> : tree_wide_kernel<T, D, false, false>;
  cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(wide_smem<D, false>(kMaxBatch)));
  if (err != cudaSuccess) return err;
  return launch_kernel(kern, dim3(ctas), dim3(kThreads<false>), wide_smem<D, false>(a.B), s, true, a, mk, mv);
}
template <typename T, int D>
cudaError_t launch_codes(const TreeArgs& a, int ctas, cudaStream_t s) {
  auto kern = tree_wide_kernel<T, D, false, true>;
  cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(wide_smem<D, true>(kMaxBatch)));
  if (err != cudaSuccess) return err;
  return launch_kernel(kern, dim3(ctas), dim3(kThreads<true>), wide_smem<D, true>(a.B), s, true, a, CUtensorMap{}, CUtensorMap{});
}

}  // namespace

cudaError_t launch_tree_wide(const TreeArgs& a, bool bf16, int D, int ctas, cudaStream_t s) {
  if (D == 128) return bf16 ? launch<__nv_bfloat16, 128>(a, ctas, s) : launch<__half, 128>(a, ctas, s);
  return bf16 ? launch<__nv_bfloat16, 64>(a, ctas, s) : launch<__half, 64>(a, ctas, s);
}

cudaError_t launch_tree_wide_fp8(const TreeArgs& a, bool bf16, int D, int ctas, cudaStream_t s) {
  if (D == 128) return bf16 ? launch_codes<__nv_bfloat16, 128>(a, ctas, s) : launch_codes<__half, 128>(a, ctas, s);
  return bf16 ? launch_codes<__nv_bfloat16, 64>(a, ctas, s) : launch_codes<__half, 64>(a, ctas, s);
}

}  // namespace tree
}  // namespace gbmoe
