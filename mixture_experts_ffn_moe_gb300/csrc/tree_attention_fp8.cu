// Attention of drafted tokens (or of single ones) over a paged cache of 8-bit codes.
//
// Mathematics.  As in tree_attention.cu, with K_s = code * ks_s and V_s = code * vs_s, one scale a slot and KV head.  The
// codes enter both products as they are, as fp16 (exact); the key's scale multiplies its scores.  The value's scale goes
// into the exponent of the weights:
//   w_s = 2^(x_s + log2 vs_s - m),  O = sum w_s code_s,  l = sum w_s / vs_s,  out = O / l,
// x_s = score * log2 e, m a running reference of x_s + log2 vs_s.  So what is rounded to fp16 for the second product is a
// weight together with its slot's scale: slots of small values lose their bits only where they lose them in the result.  As
// there, a row's reference moves when its maximum has grown by more than 2^8 and the weights stand 2^7 higher.  A slot of zero
// values has a scale of 1, as the append writes it, and beside it values far below 1 would lose their bits to a slot that adds
// nothing: any scale is right for it, so it counts with 2^-40.  Only slots with a scale of 1 are looked at (all of them: 32
// sequences of 300 to 4,100 slots, 32 rows, 71.2 us; none 68.9; so 69.3, and 72.2 where all scales are 1).  bf16 queries become
// fp16 in a power-of-two frame a row.
//
// Bound: codes and scales are read once: (2 D + 8) bytes a slot and KV head.  Work split and join are tree_attention.cu's.
//
// Layout.  A warp owns 16 slots of one KV head a step, with a ring of stages of its own.  Its loads are pieces of D bytes, a
// slot each: at D = 64 half lines, so there the warps of a CTA take two KV heads that stand side by side (64 sequences of 300
// to 8,100 slots, 8 KV heads of 64: 88 us with one head a CTA; at D = 128 two heads take 131 us instead of 110).
// The cache is the first operand (16 slots, or 16 elements of D, by 16) and the queries, or the weights turned by movmatrix,
// are the second (8 rows): a decode step has the few query heads of a KV head as its rows, and rows of 16 would leave half of
// the products and of the softmax idle (64 sequences of 300 to 8,100 slots, 8 KV heads of 128, 4 rows: 136 us so, 110 now).
// A product sums over its K index in any order, so that index is chosen such that a lane finds its operands side by side: 16
// neighbouring codes of a key are its operands of four steps, and 16 (8) neighbouring codes of four values those of 8 (4)
// blocks of D.  That takes 8 16-byte loads from shared memory and 64 conversions a stage.  The 16-byte chunks of a row are
// permuted (code_at) such that both patterns are free of bank conflicts.
//
// Measured: those 64 sequences (579 MB) in 110 us = 5.3 TB/s; the loads alone, without any product, take 101 to 104 of them,
// planning, the first loads and the join 8.  One sequence of 65,536 slots 36 us (floor 20); one of 37 slots 5.1 us.  8 KV heads
// of 64, 64 sequences of those lengths: 64 us (floor 44).
#include <cuda_runtime.h>

#include "tree_attention.cuh"

namespace gbmoe {
namespace {

using namespace tree;

constexpr int kFWarps = 4;
constexpr int kFThreads = kFWarps * 32;

// RN: 8-row tiles of a CTA's rows.
template <int D, int RN> struct F8Cfg {
  static constexpr int kSides = D == 64 ? 2 : 1;   // KV heads that the warps of a CTA share at most
  static constexpr int kSide = 16 * D;             // codes of 16 keys or values
  static constexpr int kStage = 2 * kSide + 128;   // and their 2 x 16 scales
  static constexpr int S = D == 128 ? 4 : 8;       // stages a warp
  static constexpr int kCtas = RN <= 2 ? 3 : 2;    // an SM: 12 warps with 3 stages under way (16 with 2: the same within 1%)
  static constexpr int kJoin = RN * 8 * D * 4;     // a warp's rows of O
  static constexpr int kWarp = S * kStage > kJoin ? S * kStage : kJoin;
};

template <int D, int RN> constexpr size_t f8_smem(int B) {
  return static_cast<size_t>(kFWarps) * F8Cfg<D, RN>::kWarp + (2 * static_cast<size_t>(B) + 1 + kFWarps) * 8 +
         kFWarps * (8 * 4 + RN * 8 * 8) + F8Cfg<D, RN>::kSides * RN * 8 * (D * 2 + 4) + 128;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
  return r;
}
// An 8 x 8 block of 16-bit elements, two neighbours of row lane / 4 a lane: its transpose, held alike.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Byte offset of chunk ch (16 codes) of slot r of a stage's keys or values.  D = 128: rows of 8 chunks; D = 64: rows r and
// r + 4 share a line of 8.  Conflict-free for lanes that read chunks 0..3 of slots r and r + 4, and for lanes that read a
// pair of chunks of slots 0..3 or 4..7.
template <int D> __device__ __forceinline__ int code_at(int r, int ch) {
  if constexpr (D == 128) return r * 128 + ((ch ^ (((r & 3) ^ ((r & 4) >> 1)) << 1)) << 4);
  else return ((r & 3) + ((r >> 3) << 2)) * 128 + (((((r >> 2) & 1) * 4 + ch) ^ ((r & 3) << 1)) << 4);
}
// The slot (of 8) that is row n of a score block: rows 2t and 2t + 1 are slots t and t + 4.
__device__ __forceinline__ int slot_of(int n) { return ((n & 1) << 2) | (n >> 1); }

// UNI: a page holds a multiple of 16 slots, so that a warp's 16 slots lie in one.
template <typename T, int D, int RN, bool UNI>
__global__ void __launch_bounds__(kFThreads, F8Cfg<D, RN>::kCtas) tree_fp8_kernel(const __grid_constant__ TreeArgs a) {
  using C = F8Cfg<D, RN>;
  constexpr int R = RN * 8, CH = D / 8, E = D / 8;  // rows; 16-byte chunks of a query; codes of a value that a lane takes
  constexpr int LPR = D / 16;           // chunks of a code row
  extern __shared__ unsigned char raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 127) / 128 * 128);
  unsigned char* ring = smem + (threadIdx.x >> 5) * C::kWarp;
  unsigned char* qs = smem + kFWarps * C::kWarp;                                         // [sides][R][D] fp16
  long long* prefix = reinterpret_cast<long long*>(qs + C::kSides * R * D * 2);             // [B + 1], then scan scratch
  int2* sizes = reinterpret_cast<int2*>(prefix + a.B + 1 + kFWarps);                     // [B]
  float* ml = reinterpret_cast<float*>(sizes + a.B);                                     // [warps][R][2]
  float* frame = ml + kFWarps * R * 2;                                                   // [sides][R]
  uint32_t* okmask = reinterpret_cast<uint32_t*>(frame + C::kSides * R) + (threadIdx.x >> 5) * 8;  // [S] a warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int side = warp & (a.sides - 1), run = warp / a.sides;  // of the CTA's a.sides KV heads, and runs of 16 slots
  const uint32_t ring_s = sm100::smem_addr(ring), q_s = sm100::smem_addr(qs) + side * (R * D * 2);

  pdl_trigger();
  pdl_wait();
  int bad_plan;
  plan_line<kFThreads>(a, prefix, sizes, prefix + a.B + 1, &bad_plan);
  const long long total = prefix[a.B];
  const long long chunk = (total + gridDim.x - 1) / gridDim.x;
  if (blockIdx.x == 0) {
    bad_plan = __syncthreads_count(bad_plan);
    if (tid == 0) { a.header[0] = gridDim.x; a.header[1] = bad_plan; a.prefix[a.B + 1] = chunk; }
    for (int b = tid; b <= a.B; b += kFThreads) a.prefix[b] = prefix[b];
  }
  int bad_pages = 0;
  long long pos = blockIdx.x * chunk;
  const long long end = pos + chunk < total ? pos + chunk : total;
  while (pos < end) {
    const Piece u = piece_at(a, prefix, sizes, pos, end, 0);
    pos += u.places;
    if (u.rows == 0) continue;
    const int b = u.b, ctx = u.ctx, L = u.ctx + u.n, kt = u.kt, k0 = u.k0, k1 = u.k1, row0 = u.row0;
    const int head = u.head * a.sides + side, rows = u.rows, node0 = u.node0;
    const int sl = lane & 15, ch16 = lane % LPR, r16 = lane / LPR;  // of the copies: the lane's scale, chunk and first row
    const unsigned char* kbase = static_cast<const unsigned char*>(a.kc) + head * a.k_head + ch16 * 16 + (UNI ? r16 * a.k_slot : 0);
    const unsigned char* vbase = static_cast<const unsigned char*>(a.vc) + head * a.v_head + ch16 * 16 + (UNI ? r16 * a.v_slot : 0);
    // lanes 0..15 bring the keys' scales, 16..31 the values'
    const float* sbase = lane < 16 ? a.ks + head * a.ks_head + (UNI ? sl * a.ks_slot : 0) : a.vs + head * a.vs_head + (UNI ? sl * a.vs_slot : 0);
    const long long s_page = lane < 16 ? a.ks_page : a.vs_page, s_slot = lane < 16 ? a.ks_slot : a.vs_slot;
    const int32_t* table = a.table + b * a.table_ld;

    // Block table entries before their use.  UNI: lane i has that of the warp's 16 slots of tile `from` + i, 32 tiles at once;
    // else that of this lane's slot of one tile.
    struct Place { int page, at; };
    auto look_up = [&](int it) {
      const int slot = it * a.tile + run * 16 + (UNI ? 0 : sl);
      Place p{-1, 0};
      if (it < k1 && slot < L) {
        const int pi = div_by(slot, a.page);
        p.at = slot - pi * a.page.d;
        p.page = __ldg(table + pi);
      }
      return p;
    };
    // this warp's 16 slots of tile `it`, which lie at `place`, into stage `st`
    auto issue = [&](int it, int st, Place place) {
      const int left = L - it * a.tile - run * 16;
      const uint32_t base = ring_s + st * C::kStage;
      const bool in = static_cast<uint32_t>(place.page) < static_cast<uint32_t>(a.pages);
      const uint64_t pg = in ? static_cast<uint32_t>(place.page) : 0, at = static_cast<uint32_t>(place.at);
      const uint64_t ko = pg * a.k_page + at * a.k_slot, vo = pg * a.v_page + at * a.v_slot;
      const float* sp = sbase + (pg * s_page + at * s_slot);
      uint32_t ok;
      if constexpr (UNI) {
        ok = !in || left <= 0 ? 0u : left >= 16 ? 0xffffu : (1u << left) - 1;
        if (!in && lane == 0 && left > 0) bad_pages += min(16, left);
      } else {
        ok = __ballot_sync(0xffffffffu, in && sl < left) & 0xffffu;
        if (!in && lane < 16 && sl < left) ++bad_pages;
      }
      const unsigned char *kp = kbase + ko, *vp = vbase + vo;
      auto copy = [&](auto all) {
#pragma unroll
        for (int i = 0; i < 16 * LPR / 32; ++i) {
          const int r = r16 + i * (32 / LPR);
          const uint32_t dst = base + code_at<D>(r, ch16);
          const bool live = decltype(all)::value || ((ok >> r) & 1);
          if constexpr (!UNI) {
            kp = kbase + __shfl_sync(0xffffffffu, ko, r);
            vp = vbase + __shfl_sync(0xffffffffu, vo, r);
          }
          cp_async16(dst, kp, live);
          cp_async16(dst + C::kSide, vp, live);
          if constexpr (UNI) {
            kp += (32 / LPR) * a.k_slot;
            vp += (32 / LPR) * a.v_slot;
          }
        }
        cp_async4(base + 2 * C::kSide + lane * 4, sp, decltype(all)::value || ((ok >> sl) & 1));
      };
      if (ok == 0xffffu) copy(std::true_type());
      else copy(std::false_type());
      if (lane == 0) okmask[st] = ok;
    };
    // A unit starts with all of its loads under way at once: places of the first tiles, queries and masks (rows past the
    // last one repeat it, without a branch around the loads: nothing is taken from them).
    __syncwarp();
    Place first[UNI ? 1 : C::S - 1], next;
    int from = k0;
    if constexpr (UNI) {
      next = look_up(k0 + lane);
    } else {
#pragma unroll
      for (int s = 0; s < C::S - 1; ++s) first[s] = look_up(k0 + s);
      next = look_up(k0 + C::S - 1);
    }
    auto of_tile = [&](int it) {  // (UNI)
      return Place{__shfl_sync(0xffffffffu, next.page, it - from), __shfl_sync(0xffffffffu, next.at, it - from)};
    };
    // queries of the CTA's KV heads
    constexpr int QV = (C::kSides * R * CH + kFThreads - 1) / kFThreads;
    uint4 qv[QV];
#pragma unroll
    for (int k = 0; k < QV; ++k) {
      const int i = tid + k * kFThreads, x = i / (R * CH), r = row0 + min(i / CH - x * R, rows - 1), node = div_by(r, a.group);
      const int hq = (u.head * a.sides + x) * a.group.d + (r - node * a.group.d);
      qv[k] = make_uint4(0, 0, 0, 0);
      if (x < a.sides) qv[k] = ld_v4(static_cast<const T*>(a.q) + (node0 + node) * a.q_t + hq * a.q_h + i % CH * 8);
    }
    // this lane's rows: 8n + 2t and 8n + 2t + 1
    unsigned long long bits[RN][2];
#pragma unroll
    for (int n = 0; n < RN; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int node = div_by(row0 + min(n * 8 + 2 * t + c, rows - 1), a.group);
        bits[n][c] = (2ull << node) - 1;
        if (a.mask) bits[n][c] = a.mask[node0 + node];
      }
#pragma unroll
    for (int s = 0; s < C::S - 1; ++s) {
      if (k0 + s < k1) issue(k0 + s, s, UNI ? of_tile(k0 + s) : first[UNI ? 0 : s]);
      cp_commit();
    }
    // as fp16; chunk ch of row r stands at ch ^ (r & 1)
#pragma unroll
    for (int k = 0; k < QV; ++k) {
      const int i = tid + k * kFThreads, r = i / CH, ch = i % CH;
      uint4 v = qv[k];
      float row_mul = a.scale_log2;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = Elem<T>::unpack(w[j]);
          top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
#pragma unroll
        for (int o = CH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = x_frame_exp(top);
        const float f = exp2i(-e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = Elem<T>::unpack(w[j]);
          w[j] = pack_half2(x.x * f, x.y * f);
        }
        row_mul *= exp2i(e);
      }
      if (i < C::kSides * R * CH) {
        if (ch == 0) frame[r] = row_mul;
        *reinterpret_cast<uint4*>(qs + r * D * 2 + ((ch ^ (r & 1)) << 4)) = v;
      }
    }
    __syncthreads();
    // second operands of the scores: of row 8n + g its elements 16t .. 16t + 15 (+ 64 hf), 4 a step
    auto q_load = [&](int n, int hf, uint32_t (&w)[8]) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int ch = hf * 8 + 2 * t + c, r = n * 8 + g;
        const uint4 x = lds128(q_s + r * D * 2 + ((ch ^ (r & 1)) << 4));
        w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
      }
    };
    constexpr bool kKeepQ = RN <= 2;
    uint32_t qw[kKeepQ ? RN : 1][kKeepQ ? D / 64 : 1][8];
    if constexpr (kKeepQ) {
#pragma unroll
      for (int n = 0; n < RN; ++n)
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) q_load(n, hf, qw[n][hf]);
    }
    float mul[RN][2];
#pragma unroll
    for (int n = 0; n < RN; ++n) {
      mul[n][0] = frame[side * R + n * 8 + 2 * t];
      mul[n][1] = frame[side * R + n * 8 + 2 * t + 1];
    }

    // o[n][j]: elements E g + 2j (0, 1) and E g + 2j + 1 (2, 3) of D, of this lane's two rows
    float o[RN][E / 2][4], m[RN][2], l[RN][2];
#pragma unroll
    for (int n = 0; n < RN; ++n) {
#pragma unroll
      for (int j = 0; j < E / 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    const int key0 = slot_of(g);  // this lane's slots: key0 and key0 + 8

    int st = 0;
    for (int it = k0; it < k1; ++it) {
      cp_wait<C::S - 2>();
      __syncwarp();
      const uint32_t kst = ring_s + st * C::kStage, vst = kst + C::kSide, sst = vst + C::kSide;
      const uint32_t ok = okmask[st];
      const int slot0 = it * a.tile + run * 16;
      const bool edge = ok != 0xffffu || slot0 + 16 > ctx;
      if (slot0 + 16 > ctx) {
        // Drafted slots are hidden from some rows: a NaN of a hidden value would come through as 0 * NaN.  The codes of such
        // a slot are cleared and its scale, which only those rows take that see it, becomes NaN.
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < 16 * LPR / 32; ++i) {
          const int r = r16 + i * (32 / LPR);
          if (has_nan(lds128(vst + code_at<D>(r, ch16))) && slot0 + r >= ctx) odd |= 1u << r;
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
        unsigned char* stage = ring + st * C::kStage;
        for (; odd; odd &= odd - 1) {
          const int r = __ffs(odd) - 1;
          if (lane < LPR) *reinterpret_cast<uint4*>(stage + C::kSide + code_at<D>(r, lane)) = make_uint4(0, 0, 0, 0);
          if (lane == 0) *reinterpret_cast<float*>(stage + 2 * C::kSide + 64 + r * 4) = __int_as_float(0x7fffffff);
        }
        __syncwarp();
      }
      // scores: row slot_of(g) (+ 8) of the block, column 2t (+ 1)
      float s[RN][4];
#pragma unroll
      for (int n = 0; n < RN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        const uint4 x = lds128(kst + code_at<D>(key0, hf * 4 + t)), y = lds128(kst + code_at<D>(8 + key0, hf * 4 + t));
        uint32_t ka[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e4m3x4_to_f16x4(reinterpret_cast<const uint32_t*>(&x)[j], ka[j][0], ka[j][2]);
          e4m3x4_to_f16x4(reinterpret_cast<const uint32_t*>(&y)[j], ka[j][1], ka[j][3]);
        }
#pragma unroll
        for (int n = 0; n < RN; ++n) {
          uint32_t tw[8];
          if constexpr (!kKeepQ) q_load(n, hf, tw);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (kKeepQ) mma_f16_16816(s[n], ka[j], qw[n][hf][2 * j], qw[n][hf][2 * j + 1]);
            else mma_f16_16816(s[n], ka[j], tw[2 * j], tw[2 * j + 1]);
          }
        }
      }
      float ks[2], lv[2], iv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ks[i] = lds_f(sst + (key0 + 8 * i) * 4);
        const float v = lds_f(sst + 64 + (key0 + 8 * i) * 4), x = lg2(fminf(fmaxf(v, 0x1p-64f), 0x1p64f));
        iv[i] = ex2(-x);
        lv[i] = v == v ? x : v;
      }
      uint32_t p[RN][2];
#pragma unroll
      for (int n = 0; n < RN; ++n) {
        float v[4];  // slot i / 2, row i % 2
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(s[n][i] * mul[n][i & 1], ks[i >> 1], lv[i >> 1]);
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 8 * (i >> 1), node = slot0 + key - ctx;
            const bool sees = ((ok >> key) & 1) && (node < 0 || ((bits[n][i & 1] >> (node & 63)) & 1));
            if (!sees) v[i] = -INFINITY;
          }
        }
        // a row's maximum has grown past its reference if any lane's has
        auto more = [&] { return fmaxf(v[0], v[2]) > m[n][0] + kLazy || fmaxf(v[1], v[3]) > m[n][1] + kLazy; };  // (from -infinity: any number is)
        const bool ones = lv[0] == 0.f || lv[1] == 0.f;  // scales of 1
        bool move = __any_sync(0xffffffffu, more() || (n == 0 && ones));
        if (n == 0 && move) {
          if (__any_sync(0xffffffffu, ones)) {  // those of zero values (the other rows' exponents come after this)
            uint32_t some = 0;
#pragma unroll
            for (int i = 0; i < 16 * LPR / 32; ++i) {
              const int r = r16 + i * (32 / LPR);
              if (not_zero(lds128(vst + code_at<D>(r, ch16)))) some |= 1u << r;
            }
            some = __reduce_or_sync(0xffffffffu, some);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (lv[i] == 0.f && !((some >> (key0 + 8 * i)) & 1)) {
                lv[i] = kZeroCounts;
                iv[i] = ex2(-kZeroCounts);
                v[2 * i] += kZeroCounts;
                v[2 * i + 1] += kZeroCounts;
              }
            move = __any_sync(0xffffffffu, more());
          }
        }
        if (move) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(v[c], v[2 + c]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const bool grow = top > m[n][c] + kLazy;
            const float nm = grow ? top : m[n][c], f = grow ? ex2(m[n][c] - nm) : 1.f;  // 0 for the first reference
            m[n][c] = nm;
            l[n][c] *= f;
#pragma unroll
            for (int j = 0; j < E / 2; ++j) { o[n][j][c] *= f; o[n][j][2 + c] *= f; }
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float ref = (m[n][c] == -INFINITY ? 0.f : m[n][c]) - kHeadroom<__half>;
          v[c] = ex2(v[c] - ref);
          v[2 + c] = ex2(v[2 + c] - ref);
          l[n][c] = fmaf(v[c], iv[0], fmaf(v[2 + c], iv[1], l[n][c]));
        }
        p[n][0] = transposed(pack_half2(v[0], v[1]));
        p[n][1] = transposed(pack_half2(v[2], v[3]));
      }
      // values of slots t, t + 4, t + 8, t + 12: codes E g .. E g + E - 1, two a block of D
      uint32_t vw[4][E / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const uint4 x = lds128(vst + code_at<D>(t + 4 * i, g));
          vw[i][0] = x.x; vw[i][1] = x.y; vw[i][2] = x.z; vw[i][3] = x.w;
        } else {
          const uint2 x = lds64(vst + code_at<D>(t + 4 * i, g >> 1) + (g & 1) * 8);
          vw[i][0] = x.x; vw[i][1] = x.y;
        }
      }
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        uint32_t va[4];
        const int sel = j & 1 ? 0x7362 : 0x5140;
        e4m3x4_to_f16x4(__byte_perm(vw[0][j / 2], vw[1][j / 2], sel), va[0], va[1]);
        e4m3x4_to_f16x4(__byte_perm(vw[2][j / 2], vw[3][j / 2], sel), va[2], va[3]);
#pragma unroll
        for (int n = 0; n < RN; ++n) mma_f16_16816(o[n][j], va, p[n][0], p[n][1]);
      }
      __syncwarp();
      const int nx = it + C::S - 1;
      if (nx < k1) {
        if constexpr (UNI) {
          if (nx - from == 32) {
            from = nx;
            next = look_up(nx + lane);
          }
          issue(nx, st == 0 ? C::S - 1 : st - 1, of_tile(nx));
        } else {
          issue(nx, st == 0 ? C::S - 1 : st - 1, next);
          next = look_up(nx + 1);
        }
      }
      cp_commit();
      st = st + 1 == C::S ? 0 : st + 1;
    }
    cp_wait<0>();
    __syncwarp();

    const bool whole = k0 == 0 && k1 == kt;
    // where the results of row `row` of the CTA's KV head x go, from element c on: four of them
    auto put = [&](int x, int row, int c, float4 v, float sum, float top) {
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int node = div_by(row0 + row, a.group), hq = (u.head * a.sides + x) * a.group.d + (row0 + row - node * a.group.d);
        T* dst = static_cast<T*>(a.out) + (node0 + node) * a.o_t + hq * a.o_h + c;
        *reinterpret_cast<uint2*>(dst) = make_uint2(Elem<T>::pack(v.x * inv, v.y * inv), Elem<T>::pack(v.z * inv, v.w * inv));
      } else {
        const long long slot = (static_cast<long long>(blockIdx.x) * a.sides + x) * 2 + (k0 == 0 ? 1 : 0);
        *reinterpret_cast<float4*>(a.part_o + (slot * R + row) * D + c) = v;
        if (c == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * R + row) * 2) = make_float2(top, sum);
      }
    };
    // join the slots of a head's warps: m, l and O of every row.  Elements 4 c4 .. 4 c4 + 3 of row r stand in group_at(r, c4).
    float* mine = reinterpret_cast<float*>(ring);  // [R][D]
    auto group_at = [](int r, int c4) {
      const int x = (r >> 1) & 3;
      return c4 ^ (D == 128 ? x : (x & 1) | ((x & 2) << 1));
    };
#pragma unroll
    for (int n = 0; n < RN; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[n][c];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int row = n * 8 + 2 * t + c;
        if (g == 0) { ml[(warp * R + row) * 2] = m[n][c]; ml[(warp * R + row) * 2 + 1] = sum; }
#pragma unroll
        for (int j = 0; j < E / 2; j += 2)
          *reinterpret_cast<float4*>(mine + row * D + group_at(row, (E * g + 2 * j) / 4) * 4) =
              make_float4(o[n][j][c], o[n][j][2 + c], o[n][j + 1][c], o[n][j + 1][2 + c]);
      }
    __syncthreads();
    for (int i = tid; i < a.sides * rows * (D / 4); i += kFThreads) {
      const int x = i / (rows * (D / 4)), row = (i - x * rows * (D / 4)) / (D / 4), c4 = i % (D / 4);
      float mm = -INFINITY;
      for (int w = x; w < kFWarps; w += a.sides) mm = fmaxf(mm, ml[(w * R + row) * 2]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      for (int w = x; w < kFWarps; w += a.sides) {
        const float f = ex2(ml[(w * R + row) * 2] - ref);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * C::kWarp) + row * D + group_at(row, c4) * 4);
        sum += f * ml[(w * R + row) * 2 + 1];
        acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
      }
      put(x, row, c4 * 4, acc, sum, mm);
    }
    __syncthreads();
  }
  bad_pages = __reduce_add_sync(0xffffffffu, bad_pages);
  __syncthreads();
  if (lane == 0) okmask[0] = bad_pages;
  __syncthreads();
  if (tid == 0) {
    int all = 0;
    for (int w = 0; w < kFWarps; ++w) all += okmask[w * 8];
    a.header[2 + blockIdx.x] = all;
  }
}

// How a call is cut, from the host's sizes: the average tree's rows a KV head; more than 64 go to the tcgen05 kernel.  Measured
// with 16 sequences of 2000 slots, 8 KV heads, in tiles of 8, 16, 32 rows and on tcgen05, us:
//   heads of 128:  8 rows 24, 29, 35, 68;  16 rows 30, 30, 37, 68;  32 rows 39, 37, 41, 69;  64 rows 66, 59, 60, 71;
//                  96 rows 94, 84, 77, 74;  128 rows 116, 101, 98, 77
//   heads of 64:   8 rows 20, 23, 26, 57;  16 rows 23, 22, 27, 58;  32 rows 30, 26, 28, 58;  64 rows 47, 38, 41, 59;
//                  96 rows 68, 56, 52, 61;  128 rows 84, 63, 64, 63
// So tiles of 32 come out level with tiles of 16 between 17 and 64 rows (1 to 9% behind in this shape), and at heads of 64 the
// border to tcgen05 could lie at 128 rows.
struct F8Plan { int rows, sides, ranks; bool wide; };
F8Plan f8_plan(int N, int B, int Hq, int Hkv, int dim, bool adjacent) {
  const long long avg = (static_cast<long long>(N) + B - 1) / B * (Hq / Hkv);
  if (avg > 64) return {kWideRows, 1, avg <= kWideRows ? 1 : avg <= 2 * kWideRows ? 2 : 4, true};
  return {avg <= 8 ? 8 : avg <= 16 ? 16 : 32, dim == 64 && adjacent && Hkv % 2 == 0 ? 2 : 1, 1, false};
}
TreeLayout f8_layout(const F8Plan& p, int B, int dim) {  // (room for two sides at 64, whatever the strides say)
  return tree_layout(B, p.wide ? kMaxTreeCtas / 2 : (p.rows == 32 ? kMaxTreeCtas : kHeaderCtas) * (dim == 64 ? 2 : 1), p.rows, dim);
}

constexpr int kSmemOfSm = 227 * 1024;

template <typename T, int D, int RN, bool UNI>
cudaError_t launch_fp8(const TreeArgs& a, int sms, cudaStream_t s) {
  auto kern = tree_fp8_kernel<T, D, RN, UNI>;
  cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(f8_smem<D, RN>(kMaxBatch)));
  if (err != cudaSuccess) return err;
  const size_t smem = f8_smem<D, RN>(a.B);
  int per = static_cast<int>(kSmemOfSm / (smem + 1024));  // (1 KB a CTA is the system's)
  per = per > F8Cfg<D, RN>::kCtas ? F8Cfg<D, RN>::kCtas : per;
  constexpr int kMost = RN == 4 ? kMaxTreeCtas : kHeaderCtas;  // (as f8_layout has it)
  const int ctas = per * sms < kMost ? per * sms : kMost;
  return launch_kernel(kern, dim3(ctas), dim3(kFThreads), smem, s, true, a);
}

template <typename T, int D, int RN>
cudaError_t launch_fp8_pages(const TreeArgs& a, int sms, cudaStream_t s) {
  return a.page.d % 16 == 0 ? launch_fp8<T, D, RN, true>(a, sms, s) : launch_fp8<T, D, RN, false>(a, sms, s);
}

template <typename T, int D>
cudaError_t launch_fp8_rows(const TreeArgs& a, int sms, cudaStream_t s) {
  return a.rows == 8    ? launch_fp8_pages<T, D, 1>(a, sms, s)
         : a.rows == 16 ? launch_fp8_pages<T, D, 2>(a, sms, s)
                        : launch_fp8_pages<T, D, 4>(a, sms, s);
}

template <typename T>
cudaError_t launch_fp8_typed(const TreeArgs& a, int D, bool wide, int sms, bool one_tile, cudaStream_t s) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  cudaError_t err;
  if (wide) {
    const int ctas = sms / a.ranks * a.ranks;
    err = launch_tree_wide_fp8(a, kBf16, D, ctas < kMaxTreeCtas / 2 ? ctas : kMaxTreeCtas / 2 / a.ranks * a.ranks, s);
  } else {
    err = D == 128 ? launch_fp8_rows<T, 128>(a, sms, s) : launch_fp8_rows<T, 64>(a, sms, s);
  }
  if (err != cudaSuccess || one_tile) return err;  // a unit of one tile is never cut
  // few rows, so long ones: 8 warps each (32 heads, one sequence of 1,000 slots 10.7 us, 12.9 with one warp; 8,000 slots 14, 23;
  // 65,536 slots 37, 49; 16 sequences of 8,000 slots 59, 61)
  return launch_tree_join(a, kBf16, D, !wide && static_cast<long long>(a.N) * a.Hq <= 4LL * sms, s);
}

}  // namespace
}  // namespace gbmoe

extern "C" size_t moe_tree_attention_fp8_workspace_size(int nodes, int batch, int q_heads, int k_heads, int dim) {
  using namespace gbmoe;
  if (nodes < 0 || batch <= 0 || batch > kMaxBatch || q_heads <= 0 || k_heads <= 0 || q_heads % k_heads ||
      (dim != 64 && dim != 128))
    return 0;
  return f8_layout(f8_plan(nodes, batch, q_heads, k_heads, dim, true), batch, dim).total;
}

extern "C" moe_status_t moe_tree_attention_fp8(const moe_tree_attention_fp8_args_t* r, void* workspace, size_t workspace_bytes,
                                               moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_tree_attention_fp8", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_tree_attention_fp8: ") + m); };
    auto not_built = [](const char* m) { return report_error(MOE_ERR_UNSUPPORTED, std::string("moe_tree_attention_fp8: ") + m); };
    if (!r) return bad("NULL arguments");
    if (r->dtype != MOE_DTYPE_BF16 && r->dtype != MOE_DTYPE_FP16) return bad("dtype must be bf16 or fp16");
    if (r->nodes < 0 || r->batch < 0 || r->q_heads <= 0 || r->k_heads <= 0 || r->page_size <= 0 || r->num_pages < 0 ||
        r->table_width < 0)
      return bad("sizes must be positive");
    if (r->q_heads % r->k_heads) return bad("q_heads must be a multiple of k_heads");
    if (r->dim != 64 && r->dim != 128) return not_built("head dimension must be 64 or 128");
    if (r->batch > kMaxBatch) return not_built("more than 1024 sequences");
    if (r->q_heads / r->k_heads > 1024 || r->k_heads > 65536 || r->nodes > (1 << 20)) return not_built("problem too large");
    if (static_cast<long long>(r->table_width) * r->page_size > 0x7fffff00LL) return not_built("more than 2^31 - 256 slots a sequence");
    if (!(r->scale > -INFINITY && r->scale < INFINITY)) return bad("scale must be finite");
    if (r->nodes == 0 || r->batch == 0) return MOE_OK;
    if (!r->q || !r->k_cache.data || !r->v_cache.data || !r->k_cache.scale || !r->v_cache.scale || !r->block_table ||
        !r->context_lens || !r->node_offsets || !r->out)
      return bad("NULL pointer");
    if (r->q_stride_t % 8 || r->q_stride_h % 8) return bad("query strides must be multiples of 8 elements (16 bytes)");
    for (const moe_cache_view_t* c : {&r->k_cache, &r->v_cache}) {
      if (c->page_stride % 16 || c->slot_stride % 16 || c->head_stride % 16) return bad("code strides must be multiples of 16 elements (16 bytes)");
      if (!aligned(c->data, 16)) return bad("the caches must be 16-byte aligned");
      if (!aligned(c->scale, 4)) return bad("scales must be 4-byte aligned");
    }
    if (r->out_stride_t % 4 || r->out_stride_h % 4) return bad("output strides must be multiples of 4 elements");
    if (!aligned(r->q, 16)) return bad("q must be 16-byte aligned");
    if (!aligned(r->out, 8) || !aligned(r->tree_mask, 8)) return bad("out and tree_mask must be 8-byte aligned");
    const F8Plan p = f8_plan(r->nodes, r->batch, r->q_heads, r->k_heads, r->dim, r->k_cache.head_stride == r->dim && r->v_cache.head_stride == r->dim);
    const TreeLayout l = f8_layout(p, r->batch, r->dim);
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256))
      return report_error(MOE_ERR_WORKSPACE, "moe_tree_attention_fp8: workspace NULL, misaligned or too small");
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_tree_attention_fp8: no CUDA device");
    TreeArgs a{};
    a.q = r->q; a.kc = r->k_cache.data; a.vc = r->v_cache.data; a.out = r->out;
    a.table = r->block_table; a.ctx = r->context_lens; a.offs = r->node_offsets;
    a.mask = reinterpret_cast<const unsigned long long*>(r->tree_mask);
    a.q_t = r->q_stride_t; a.q_h = r->q_stride_h; a.o_t = r->out_stride_t; a.o_h = r->out_stride_h;
    a.k_page = r->k_cache.page_stride; a.k_slot = r->k_cache.slot_stride; a.k_head = r->k_cache.head_stride;
    a.v_page = r->v_cache.page_stride; a.v_slot = r->v_cache.slot_stride; a.v_head = r->v_cache.head_stride;
    a.ks = r->k_cache.scale; a.vs = r->v_cache.scale;
    a.ks_page = r->k_cache.scale_page_stride; a.ks_slot = r->k_cache.scale_slot_stride; a.ks_head = r->k_cache.scale_head_stride;
    a.vs_page = r->v_cache.scale_page_stride; a.vs_slot = r->v_cache.scale_slot_stride; a.vs_head = r->v_cache.scale_head_stride;
    a.table_ld = r->table_stride;
    a.N = r->nodes; a.B = r->batch; a.Hq = r->q_heads; a.Hkv = r->k_heads / p.sides; a.pages = r->num_pages; a.table_w = r->table_width;
    a.page = fast_div(r->page_size);
    a.group = fast_div(r->q_heads / r->k_heads);
    a.scale_log2 = r->scale * 1.4426950408889634f;
    char* ws = static_cast<char*>(workspace);
    a.header = reinterpret_cast<int32_t*>(ws + l.header);
    a.prefix = reinterpret_cast<long long*>(ws + l.prefix);
    a.part_ml = reinterpret_cast<float*>(ws + l.ml);
    a.part_o = reinterpret_cast<float*>(ws + l.o);
    a.tile = p.wide ? kWideTile : 16 * (kFWarps / p.sides);
    a.rows = p.rows;
    a.ranks = p.ranks;
    a.sides = p.sides;
    a.setup = 4 * p.sides;
    const bool one_tile = static_cast<long long>(r->table_width) * r->page_size <= a.tile;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched("moe_tree_attention_fp8", r->dtype == MOE_DTYPE_FP16 ? launch_fp8_typed<__half>(a, r->dim, p.wide, sms, one_tile, s)
                                                                         : launch_fp8_typed<__nv_bfloat16>(a, r->dim, p.wide, sms, one_tile, s));
  });
}
