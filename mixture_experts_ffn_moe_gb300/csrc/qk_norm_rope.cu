// Norms of query and key heads with the rotary positions in the same pass, and the append to a paged cache of the same
// type or of 8-bit codes.
//
// Mathematics.  A head x of dim elements becomes n = x * w / sqrt(mean(x^2) + eps), whose pairs then turn as in rope.cu.
// For an 8-bit cache a head y is stored as E4M3(y / s) with s = max|y| / 448.  Norm, turn and quantisation are three
// passes over a head that all fit into the registers of a few lanes, so the head is read once and written once.
//
// Split.  A head is cut into units as in rope.cu (in the halves layout a unit inside the turning part is two vectors, one
// of each half), a unit a lane: 8 lanes for a head of 128 16-bit elements, so that a warp takes 4 heads at once and the
// sum of squares is three shuffles.  A warp stays with one token: its sines and cosines are formed once, by all lanes,
// and kept in registers, and the loads of the next heads are under way while the current ones are computed.
//
// Bound: HBM for prompts, launch latency for decode steps.  Measured: 16,384 tokens, 64 / 4 heads of 128 (571 MB) in 98 us =
// 5.8 TB/s; 4,096 tokens, 32 / 8 heads, without norms, into codes (93 MB) in 26 us; 32 tokens, 64 / 4 heads, into codes in 3.6 us.
#include <cuda_runtime.h>

#include <type_traits>

#include "rope.cuh"
#include "step_ops.cuh"

namespace gbmoe {
namespace {

constexpr int kNWarps = 4;

struct NormView {  // [token, head, dim], dim contiguous, strides in elements
  const void* in;
  void* out;
  long long in_t, in_h, out_t, out_h;
  const void* weight;  // null: no norm
};

struct NormCache {
  void* data;
  float* scale;
  long long page, slot, head, s_page, s_slot, s_head;
};

struct NormArgs {
  NormView x[3];       // q, k, v
  NormCache cache[2];  // k, v
  int tokens, dim, rot, offset;
  int hq, hk, hv;
  float scale, eps;
  const int32_t* positions;
  const double* inv_freq;
  const int32_t* slots;
  int kind, num_slots;   // MOE_CACHE_*
  FastDiv page;          // slots a page
  int units, lanes;      // units of a head, lanes that share it (a power of two)
  int items, heads_item; // pieces of work (one token and some of its heads) and their heads
  FastDiv pieces;        // pieces a token
};

template <typename T, int V> struct alignas(sizeof(T) * V) NVec { T e[V]; };

template <typename T> __device__ __forceinline__ float widen(T a) { return Elem<T>::to_float(a); }
template <> __device__ __forceinline__ float widen<float>(float a) { return a; }
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* dst, const float (&y)[V]) {
  if constexpr (std::is_same<T, float>::value) {
    NVec<float, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = y[i];
    *reinterpret_cast<NVec<float, V>*>(dst) = o;
  } else if constexpr (V % 2 == 0) {
    NVec<uint32_t, V / 2> o;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) o.e[i] = Elem<T>::pack(y[2 * i], y[2 * i + 1]);
    *reinterpret_cast<NVec<uint32_t, V / 2>*>(dst) = o;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) dst[i] = Elem<T>::from_float(y[i]);
  }
}
// V codes of y / s to dst (V bytes aligned where V is 4 or 8).
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&y)[V], float s) {
  uint32_t w[V >= 4 ? V / 4 : 1] = {};
#pragma unroll
  for (int i = 0; i < V; ++i) w[i / 4] |= e4m3_code(__fdiv_rn(y[i], s)) << (8 * (i % 4));
  if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(dst) = w[0];
  else {
#pragma unroll
    for (int i = 0; i < V; ++i) dst[i] = static_cast<uint8_t>(w[0] >> (8 * i));
  }
}

// Heads of any size and alignment: V elements a vector, NU units a lane at most.
template <typename T, int V, bool INTER, int NU>
__global__ void __launch_bounds__(kNWarps * 32) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  using W = NVec<T, V>;
  constexpr int P = INTER ? 1 : 2;  // vectors of a unit
  extern __shared__ uint64_t turns[];  // [rot / 2] turn fractions, then a table of (cos, sin) a warp
  const int half = a.rot >> 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* table = reinterpret_cast<float2*>(turns + half) + warp * half;
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < half; i += kNWarps * 32) turns[i] = turn_fraction(a.inv_freq[i]);
  __syncthreads();
  const int item = blockIdx.x * kNWarps + warp;
  if (item >= a.items) return;
  const int tok = div_by(item, a.pieces), piece = item - tok * a.pieces.d;
  const int h_lo = piece * a.heads_item, h_hi = min(h_lo + a.heads_item, a.hq + a.hk + a.hv);
  const int G = a.lanes, gl = lane & (G - 1), first = lane / G, step = 32 / G;
  const int unit0 = a.offset / V, turning = (INTER ? a.rot : half) / V;
  int slot = -1;
  if (a.kind != MOE_CACHE_NONE) {
    slot = a.slots[tok];
    if (slot >= a.num_slots) slot = -1;
  }
  const bool keep = a.kind == MOE_CACHE_NONE || slot >= 0;

  // first element of the lane's n-th unit
  auto place = [&](int u) { return INTER || u < unit0 + turning ? u * V : u * V + half; };
  auto turns_at = [&](int u) { return u >= unit0 && u < unit0 + turning; };
  struct Raw { W v[NU][P]; };
  auto source = [&](int head, int& which) {  // null: nothing to do
    which = head < a.hq ? 0 : head < a.hq + a.hk ? 1 : 2;
    const int h = head - (which == 0 ? 0 : which == 1 ? a.hq : a.hq + a.hk);
    const T* p = static_cast<const T*>(which == 0 ? a.x[0].in : which == 1 ? a.x[1].in : a.x[2].in);
    return head < h_hi && (which == 0 || keep)
               ? p + tok * (which == 0 ? a.x[0].in_t : which == 1 ? a.x[1].in_t : a.x[2].in_t) +
                     h * (which == 0 ? a.x[0].in_h : which == 1 ? a.x[1].in_h : a.x[2].in_h)
               : nullptr;
  };
  auto load = [&](const T* src, Raw& r) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const int u = gl + n * G;
      if (src && u < a.units) {
        r.v[n][0] = *reinterpret_cast<const W*>(src + place(u));
        if constexpr (P == 2)
          if (turns_at(u)) r.v[n][1] = *reinterpret_cast<const W*>(src + place(u) + half);
      }
    }
  };

  int which;
  const T* src = source(h_lo + first, which);
  Raw raw;
  load(src, raw);

  const uint64_t position = static_cast<uint64_t>(static_cast<int64_t>(a.positions[tok]));
  for (int i = lane; i < half; i += 32) {
    float cs, sn;
    turn_cos_sin(position * turns[i], cs, sn);
    table[i] = make_float2(cs * a.scale, sn * a.scale);
  }
  __syncwarp();
  constexpr int C = INTER ? V / 2 : V;  // angles of a unit

  for (int h0 = h_lo; h0 < h_hi; h0 += step) {
    const int head = h0 + first;
    const bool active = src != nullptr;
    float y[NU][P][V];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const bool in = active && gl + n * G < a.units, two = P == 2 && in && turns_at(gl + n * G);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) y[n][p][i] = (p ? two : in) ? widen<T>(raw.v[n][p].e[i]) : 0.f;
    }
    const T* wt = static_cast<const T*>(which == 0 ? a.x[0].weight : which == 1 ? a.x[1].weight : nullptr);
    if (__any_sync(0xffffffffu, active && wt != nullptr)) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i) sum = fmaf(y[n][p][i], y[n][p][i], sum);
      for (int o = G >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float r = rsqrtf(__fdividef(sum, static_cast<float>(a.dim)) + a.eps);
      if (__any_sync(0xffffffffu, sum == INFINITY)) {
        // squares past fp32's range: the sum of (x / 2^80)^2, in range for 1024 of the largest numbers; x / 2^40 and 2^40 / root
        // then are normal numbers wherever their product counts
        float small = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) small = fmaf(y[n][p][i] * 0x1p-80f, y[n][p][i] * 0x1p-80f, small);
        for (int o = G >> 1; o > 0; o >>= 1) small += __shfl_xor_sync(0xffffffffu, small, o);
        if (sum == INFINITY) {
          r = rsqrtf(__fdividef(small, static_cast<float>(a.dim))) * 0x1p-40f;
#pragma unroll
          for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
              for (int i = 0; i < V; ++i) y[n][p][i] *= 0x1p-40f;
        }
      }
      if (active && wt) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const int u = gl + n * G;
            if (u < a.units && (p == 0 || turns_at(u))) {
              const W w = *reinterpret_cast<const W*>(wt + place(u) + p * half);
#pragma unroll
              for (int i = 0; i < V; ++i) y[n][p][i] = y[n][p][i] * r * widen<T>(w.e[i]);
            }
          }
      }
    }
    if (which < 2) {
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const int u = gl + n * G;
        if (active && turns_at(u)) {
#pragma unroll
          for (int i = 0; i < C; ++i) {
            const float2 c = table[(u - unit0) * C + i];
            float& p = INTER ? y[n][0][INTER ? 2 * i : 0] : y[n][0][i];
            float& q = INTER ? y[n][0][INTER ? 2 * i + 1 : 0] : y[n][P - 1][i];
            const float x0 = p, x1 = q;
            p = x0 * c.x - x1 * c.y;
            q = x1 * c.x + x0 * c.y;
          }
        }
      }
    }
    const bool cached = a.kind != MOE_CACHE_NONE && which > 0;
    if (a.kind == MOE_CACHE_E4M3 && __any_sync(0xffffffffu, active && cached)) {
      // the largest magnitude by its bits: those of infinities and NaN are above all others
      uint32_t top = 0;
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i) top = max(top, __float_as_uint(y[n][p][i]) & 0x7fffffffu);
      for (int o = G >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (active && cached) {
        const bool fine = top < 0x7f800000u;
        float s = fine ? fminf(fmaxf(__fdiv_rn(__uint_as_float(top), 448.f), 0x1p-64f), 0x1p64f) : 1.f;
        if (top == 0) s = 1.f;
        const int h = head - a.hq - (which == 1 ? 0 : a.hk), page = div_by(slot, a.page), at = slot - page * a.page.d;
        const NormCache& c = which == 1 ? a.cache[0] : a.cache[1];
        uint8_t* dst = static_cast<uint8_t*>(c.data) + page * c.page + at * c.slot + h * c.head;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          const int u = gl + n * G;
          if (u < a.units) {
            if (!fine) {
#pragma unroll
              for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) y[n][p][i] = 0.f;
            }
            store_codes<V>(dst + place(u), y[n][0], s);
            if constexpr (P == 2)
              if (turns_at(u)) store_codes<V>(dst + place(u) + half, y[n][1], s);
          }
        }
        if (gl == 0) c.scale[page * c.s_page + at * c.s_slot + h * c.s_head] = fine ? s : __int_as_float(0x7fffffff);
      }
    }
    if (active && !(a.kind == MOE_CACHE_E4M3 && cached)) {
      T* dst;
      if (cached) {
        const int h = head - a.hq - (which == 1 ? 0 : a.hk), page = div_by(slot, a.page), at = slot - page * a.page.d;
        const NormCache& c = which == 1 ? a.cache[0] : a.cache[1];
        dst = static_cast<T*>(c.data) + page * c.page + at * c.slot + h * c.head;
      } else {
        const NormView& x = which == 0 ? a.x[0] : a.x[1];
        dst = static_cast<T*>(x.out) + tok * x.out_t + (which == 0 ? head : head - a.hq) * x.out_h;
      }
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const int u = gl + n * G;
        if (u < a.units) {
          store_vec<T, V>(dst + place(u), y[n][0]);
          if constexpr (P == 2)
            if (turns_at(u)) store_vec<T, V>(dst + place(u) + half, y[n][1]);
        }
      }
    }
    if (h0 + step < h_hi) {
      src = source(head + step, which);
      load(src, raw);
    } else {
      src = nullptr;
    }
  }
}

// ---- heads whose units fit the lanes one each, in 16-byte vectors: what decoders have

// Two floats in one register pair: GB300's fp32 units take two at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
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
// 16 bytes as 4 or 8 floats, in pairs, and back.
template <typename T, int H>
__device__ __forceinline__ void widen_vec(const uint4& v, uint64_t (&x)[H]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < H; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      x[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
      const float2 f = Elem<T>::unpack(w[i]);
      x[i] = pair(f.x, f.y);
    }
  }
}
template <typename T, int H>
__device__ __forceinline__ uint4 narrow_vec(const uint64_t (&x)[H]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const float2 f = unpair(x[i]);
    if constexpr (std::is_same<T, float>::value) {
      w[2 * i] = __float_as_uint(f.x);
      w[2 * i + 1] = __float_as_uint(f.y);
    } else {
      w[i] = Elem<T>::pack(f.x, f.y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Codes of y / s, 2H of them.  y * (1 / s) is off by at most two units of its last place; where that could matter (the bits
// that E4M3 cuts off are within them of a half, or below its normals) the quotient is formed.
template <int H>
__device__ __forceinline__ void store_codes2(uint8_t* dst, const uint64_t (&y)[H], float s, float inv) {
  float q[2 * H];
  bool near = false;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const float2 f = unpair(y[i]);
    q[2 * i] = f.x * inv;
    q[2 * i + 1] = f.y * inv;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t b = __float_as_uint(q[2 * i + c]);
      near |= ((b & 0xfffffu) - 0x7fffcu) <= 8u || (fabsf(q[2 * i + c]) < 0x1p-6f && (b << 1) != 0);
    }
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float2 f = unpair(y[i]);
      q[2 * i] = __fdiv_rn(f.x, s);
      q[2 * i + 1] = __fdiv_rn(f.y, s);
    }
  }
  uint32_t w[H / 2];
#pragma unroll
  for (int i = 0; i < H / 2; ++i)
    w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3)) |
           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3)) << 16;
  if constexpr (H == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kNWarps * 32, 5) norm_rope_vec_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = 16 / sizeof(T), H = V / 2;  // elements and pairs of a vector
  constexpr int P = INTER ? 1 : 2;              // vectors of a unit
  extern __shared__ uint64_t turns[];           // [rot / 2] turn fractions, then a table of (cos, sin) a warp
  const int half = a.rot >> 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* table = reinterpret_cast<float2*>(turns + half) + warp * half;
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < half; i += kNWarps * 32) turns[i] = turn_fraction(a.inv_freq[i]);
  const int item = blockIdx.x * kNWarps + warp;
  const bool some = item < a.items;
  const int tok = some ? div_by(item, a.pieces) : 0, piece = item - tok * a.pieces.d;
  const int G = a.lanes, gl = lane & (G - 1), first = lane / G, step = 32 / G;
  const int unit0 = a.offset / V, turning = (INTER ? a.rot : half) / V;
  const bool live = gl < a.units, turn = gl >= unit0 && gl < unit0 + turning;
  const bool two = P == 2 && turn;
  const int at0 = INTER || gl < unit0 + turning ? gl * V : gl * V + half;  // first element of the lane's unit
  const uint64_t position = some ? static_cast<uint64_t>(static_cast<int64_t>(a.positions[tok])) : 0;
  int slot = a.kind != MOE_CACHE_NONE && some ? a.slots[tok] : -1;
  if (slot >= a.num_slots) slot = -1;
  // the piece's rounds, which run through q, k and v in turn: [begin, end) of the heads of each
  const int nq = (a.hq + step - 1) / step, nk = (a.hk + step - 1) / step;
  const int r0 = piece * a.heads_item, r1 = r0 + a.heads_item;
  const int q0 = r0 * step, q1 = min(r1 * step, a.hq);
  const int k0 = max(r0 - nq, 0) * step, k1 = min((r1 - nq) * step, a.hk);
  const int v0 = max(r0 - nq - nk, 0) * step, v1 = min((r1 - nq - nk) * step, a.hv);
  // All of the warp's heads on their way to L2 at once, while it forms sines and cosines: 16 KB a token of 64 heads, where the
  // loads into registers are a round of 1 KB (16,384 tokens of 64 + 4 heads of 128: 112 us without).
  auto warm = [&](const NormView& x, int begin, int end) {
    for (int h = begin + lane; h < end; h += 32) {
      const char* p = reinterpret_cast<const char*>(static_cast<const T*>(x.in) + tok * x.in_t + h * x.in_h);
      for (int c = 0; c < a.dim * static_cast<int>(sizeof(T)); c += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
    }
  };
  if (some && a.heads_item > 2) {  // (not for the few heads that are loaded at once below)
    warm(a.x[0], q0, q1);
    if (a.kind == MOE_CACHE_NONE || slot >= 0) {
      warm(a.x[1], k0, k1);
      warm(a.x[2], v0, v1);
    }
  }
  __syncthreads();
  if (!some) return;
  for (int i = lane; i < half; i += 32) {
    float cs, sn;
    turn_cos_sin(position * turns[i], cs, sn);
    table[i] = make_float2(cs * a.scale, sn * a.scale);
  }
  __syncwarp();
  // halves: pairs of angles of neighbouring elements; interleaved: (cos, cos), (-sin, sin) of every pair of elements
  uint64_t cs[H], sn[H];
  if (turn) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if constexpr (INTER) {
        const float2 c = table[(gl - unit0) * H + i];
        cs[i] = pair(c.x, c.x);
        sn[i] = pair(-c.y, c.y);
      } else {
        const float4 c = *reinterpret_cast<const float4*>(table + (gl - unit0) * V + 2 * i);
        cs[i] = pair(c.x, c.z);
        sn[i] = pair(c.y, c.w);
      }
    }
  }
  const bool cached = a.kind != MOE_CACHE_NONE;
  const float inv_dim = 1.f / static_cast<float>(a.dim);

  // Heads [begin, end) of q (WHICH = 0), k or v.
  auto section = [&](auto which, int begin, int end) {
    constexpr int WHICH = decltype(which)::value;
    if (begin >= end || (WHICH > 0 && cached && slot < 0)) return;
    const NormView& x = a.x[WHICH];
    const T* src = static_cast<const T*>(x.in) + tok * x.in_t + (begin + first) * x.in_h + at0;
    const long long src_step = step * x.in_h;
    const NormCache& c = a.cache[WHICH == 2 ? 1 : 0];
    const bool to_cache = WHICH > 0 && cached;
    const bool codes = to_cache && a.kind == MOE_CACHE_E4M3;
    long long dst_at, dst_step, scale_at = 0;  // of elements, of the lane's head and from one to the next
    if (to_cache) {
      const int page = div_by(slot, a.page), place = slot - page * a.page.d;
      dst_at = page * c.page + place * c.slot + (begin + first) * c.head + at0;
      dst_step = step * c.head;
      scale_at = page * c.s_page + place * c.s_slot + (begin + first) * c.s_head;
    } else {
      dst_at = tok * x.out_t + (begin + first) * x.out_h + at0;
      dst_step = step * x.out_h;
    }
    const bool normed = WHICH < 2 && x.weight != nullptr;
    uint64_t w[P][H] = {};  // (lanes without a unit have zeros throughout)
    if (normed && live) {
      widen_vec<T>(ld_v4(static_cast<const T*>(x.weight) + at0), w[0]);
      if (P == 2 && two) widen_vec<T>(ld_v4(static_cast<const T*>(x.weight) + at0 + half), w[P - 1]);
    }
    auto load = [&](const T* p, bool ok, uint4 (&r)[P]) {
      r[0] = ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
      if constexpr (P == 2) r[1] = ok && two ? *reinterpret_cast<const uint4*>(p + half) : make_uint4(0, 0, 0, 0);
    };
    uint4 raw[P];
    load(src, live && begin + first < end, raw);
    for (int h = begin + first; h - first < end; h += step) {
      const bool active = live && h < end;
      uint64_t y[P][H];
#pragma unroll
      for (int p = 0; p < P; ++p) widen_vec<T>(raw[p], y[p]);
      load(src + src_step, live && h + step < end, raw);
      if (normed) {
        uint64_t sum2[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          sum2[p] = mul2(y[p][0], y[p][0]);
#pragma unroll
          for (int i = 1; i < H; ++i) sum2[p] = fma2(y[p][i], y[p][i], sum2[p]);
        }
        const float2 s0 = unpair(sum2[0]), s1 = unpair(sum2[P - 1]);
        float sum = P == 2 ? (s0.x + s0.y) + (s1.x + s1.y) : s0.x + s0.y;
        for (int o = G >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float r = rsqrtf(fmaf(sum, inv_dim, a.eps));
        if (__any_sync(0xffffffffu, sum == INFINITY)) {  // squares past fp32's range: as in the kernel above
          float small = 0.f;
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const float2 f = unpair(y[p][i]);
              small = fmaf(f.x * 0x1p-80f, f.x * 0x1p-80f, fmaf(f.y * 0x1p-80f, f.y * 0x1p-80f, small));
            }
          for (int o = G >> 1; o > 0; o >>= 1) small += __shfl_xor_sync(0xffffffffu, small, o);
          if (sum == INFINITY) {
            r = rsqrtf(small * inv_dim) * 0x1p-40f;
            const uint64_t f = pair(0x1p-40f, 0x1p-40f);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
              for (int i = 0; i < H; ++i) y[p][i] = mul2(y[p][i], f);
          }
        }
        const uint64_t rr = pair(r, r);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          y[0][i] = mul2(mul2(y[0][i], rr), w[0][i]);
          if (P == 2 && two) y[P - 1][i] = mul2(mul2(y[P - 1][i], rr), w[P - 1][i]);
        }
      }
      if (WHICH < 2 && turn) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          if constexpr (INTER) {
            const float2 f = unpair(y[0][i]);
            y[0][i] = fma2(pair(f.y, f.x), sn[i], mul2(y[0][i], cs[i]));
          } else {
            const uint64_t p = y[0][i], q = y[P - 1][i];
            y[0][i] = fma2(p, cs[i], mul2(q, sn[i] ^ 0x8000000080000000ull));
            y[P - 1][i] = fma2(q, cs[i], mul2(p, sn[i]));
          }
        }
      }
      if (codes) {
        // the largest magnitude by its bits: those of infinities and NaN are above all others
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < H; ++i) {
            const float2 f = unpair(y[p][i]);
            top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
          }
        for (int o = G >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool fine = top < 0x7f800000u;
        const float s = top == 0 || !fine ? 1.f : fminf(fmaxf(__fdiv_rn(__uint_as_float(top), 448.f), 0x1p-64f), 0x1p64f);
        if (!fine) {
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < H; ++i) y[p][i] = 0;
        }
        if (active) {
          const float inv = __frcp_rn(s);
          uint8_t* dst = static_cast<uint8_t*>(c.data) + dst_at;
          store_codes2(dst, y[0], s, inv);
          if (two) store_codes2(dst + half, y[P - 1], s, inv);
          if (gl == 0) c.scale[scale_at] = fine ? s : __int_as_float(0x7fffffff);
        }
        scale_at += step * c.s_head;
      } else if (active) {
        T* dst = static_cast<T*>(to_cache ? c.data : x.out) + dst_at;
        *reinterpret_cast<uint4*>(dst) = narrow_vec<T>(y[0]);
        if (two) *reinterpret_cast<uint4*>(dst + half) = narrow_vec<T>(y[P - 1]);
      }
      src += src_step;
      dst_at += dst_step;
    }
  };
  section(std::integral_constant<int, 0>(), q0, q1);
  section(std::integral_constant<int, 1>(), k0, k1);
  section(std::integral_constant<int, 2>(), v0, v1);
}

// (up to 2^31 - 1 items: their number with what fills the last CTA up is no int)
unsigned norm_ctas(const NormArgs& a) { return (static_cast<unsigned>(a.items) + kNWarps - 1) / kNWarps; }

template <typename T, bool INTER>
cudaError_t launch_norm_vec(NormArgs& a, int sms, cudaStream_t s) {
  const int step = 32 / a.lanes, rounds = (a.hq + step - 1) / step + (a.hk + step - 1) / step + (a.hv + step - 1) / step;
  // rounds of a warp: as few as keep 48 warps an SM busy, so that a decode step spreads and a prompt's warp forms a
  // token's sines and cosines once
  long long per = static_cast<long long>(a.tokens) * rounds / (48LL * sms);
  per = per < 1 ? 1 : per > rounds ? rounds : per;
  const int pieces = static_cast<int>((rounds + per - 1) / per);
  a.heads_item = (rounds + pieces - 1) / pieces;
  const int real = (rounds + a.heads_item - 1) / a.heads_item;
  a.pieces = fast_div(real);
  a.items = a.tokens * real;
  const size_t smem = static_cast<size_t>(a.rot / 2) * 8 * (1 + kNWarps);
  return launch_kernel(norm_rope_vec_kernel<T, INTER>, dim3(norm_ctas(a)), dim3(kNWarps * 32), smem, s, true, a);
}

template <typename T, int V, bool INTER, int NU>
cudaError_t launch_norm_nu(NormArgs& a, int sms, cudaStream_t s) {
  const int heads = a.hq + a.hk + a.hv, step = 32 / a.lanes, turns = (heads + step - 1) / step;
  // rounds of a warp: as few as keep 48 warps an SM busy, so that a decode step spreads and a prompt's warp forms a
  // token's sines and cosines once
  long long per = static_cast<long long>(a.tokens) * turns / (48LL * sms);
  per = per < 1 ? 1 : per > turns ? turns : per;
  const int pieces = static_cast<int>((turns + per - 1) / per);
  a.heads_item = (turns + pieces - 1) / pieces * step;
  const int real = (heads + a.heads_item - 1) / a.heads_item;
  a.pieces = fast_div(real);
  a.items = a.tokens * real;
  const size_t smem = static_cast<size_t>(a.rot / 2) * 8 * (1 + kNWarps);
  return launch_kernel(norm_rope_kernel<T, V, INTER, NU>, dim3(norm_ctas(a)), dim3(kNWarps * 32), smem, s,
                       true, a);
}

template <typename T, int V, bool INTER>
cudaError_t launch_norm(NormArgs& a, int sms, cudaStream_t s) {
  constexpr int kMost = 1024 / V / 32;  // units a lane for the widest head
  a.units = INTER ? a.dim / V : (a.dim - a.rot / 2) / V;
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes < a.units) a.lanes *= 2;
  if constexpr (V * sizeof(T) == 16)
    if (a.units <= 32) return launch_norm_vec<T, INTER>(a, sms, s);
  return launch_norm_nu<T, V, INTER, kMost>(a, sms, s);
}

template <typename T>
cudaError_t launch_norm_typed(NormArgs& a, bool inter, bool wide, int sms, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  if (wide) return inter ? launch_norm<T, W, true>(a, sms, s) : launch_norm<T, W, false>(a, sms, s);
  return inter ? launch_norm<T, 2, true>(a, sms, s) : launch_norm<T, 1, false>(a, sms, s);
}

bool rows_on(const void* p, size_t es, size_t al, std::initializer_list<long long> strides) {
  bool ok = aligned(p, al);
  for (long long s : strides) ok = ok && (s * static_cast<long long>(es)) % static_cast<long long>(al) == 0;
  return ok;
}

}  // namespace
}  // namespace gbmoe

extern "C" moe_status_t moe_qk_norm_rope(const moe_qk_norm_rope_args_t* r, moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_qk_norm_rope", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_qk_norm_rope: ") + m); };
    auto not_built = [](const char* m) { return report_error(MOE_ERR_UNSUPPORTED, std::string("moe_qk_norm_rope: ") + m); };
    if (!r) return bad("NULL arguments");
    if (r->dtype != MOE_DTYPE_BF16 && r->dtype != MOE_DTYPE_FP16 && r->dtype != MOE_DTYPE_FP32) return bad("unknown dtype");
    const size_t es = r->dtype == MOE_DTYPE_FP32 ? 4 : 2;
    if (r->tokens < 0 || r->q_heads < 0 || r->k_heads < 0 || r->dim <= 0) return bad("sizes must be positive");
    if (r->rot_dim < 0 || r->rot_dim % 2 || r->rot_offset < 0 || r->rot_offset + static_cast<long long>(r->rot_dim) > r->dim)
      return bad("the turning part must be even and lie inside the head");
    if (r->interleaved && (r->rot_offset % 2 || r->dim % 2)) return bad("interleaved pairs need an even offset and an even head");
    if (!(r->eps >= 1e-20f && r->eps < INFINITY) || !(r->scale > -INFINITY && r->scale < INFINITY))
      return bad("eps must be at least 1e-20, eps and scale must be finite");
    if (r->cache != MOE_CACHE_NONE && r->cache != MOE_CACHE_SAME && r->cache != MOE_CACHE_E4M3) return bad("unknown kind of cache");
    if (r->dim > 1024 || r->q_heads > 4096 || r->k_heads > 4096) return not_built("heads above 1024 elements or more than 4096 heads");
    // (a piece of work, one warp's, is at least one head of one token)
    if (static_cast<long long>(r->tokens) * (r->q_heads + 2LL * r->k_heads) > 0x7fffffffLL) return not_built("more than 2^31 - 1 heads in all");
    const bool append = r->cache != MOE_CACHE_NONE, codes = r->cache == MOE_CACHE_E4M3;
    if (append && (r->page_size <= 0 || r->num_pages <= 0)) return bad("a cache needs pages");
    if (append && static_cast<long long>(r->page_size) * r->num_pages > 0x7fffffffLL) return not_built("more than 2^31 - 1 cache slots");
    if (r->tokens == 0 || r->q_heads + r->k_heads == 0) return MOE_OK;
    if (!r->positions || (r->rot_dim && !r->inv_freq)) return bad("NULL positions or frequencies");
    if (r->q_heads && (!r->q || !r->q_out)) return bad("NULL queries");
    if (r->k_heads && (!r->k || (!append && !r->k_out))) return bad("NULL keys");
    const bool kept = append && r->k_heads;
    if (kept && (!r->v || !r->slots || !r->k_cache.data || !r->v_cache.data)) return bad("NULL values, slots or cache");
    if (kept && codes && (!r->k_cache.scale || !r->v_cache.scale)) return bad("NULL scales");
    if (!aligned(r->positions, 4) || !aligned(r->inv_freq, 8) || !aligned(r->slots, 4) || !aligned(r->k_cache.scale, 4) ||
        !aligned(r->v_cache.scale, 4))
      return bad("unaligned positions, frequencies, slots or scales");
    // 16-byte vectors where every row, weight, half and edge of the turning part starts on one
    const int W = static_cast<int>(16 / es);
    auto views = [&](int n) {  // vectors of n elements
      const size_t al = es * n;
      auto cache = [&](const moe_cache_view_t& c) {
        const size_t one = codes ? 1 : es;
        // codes are stored n at once where n is 4 or more, else one by one
        return !kept || rows_on(c.data, one, codes ? (n >= 4 ? n : 1) : al, {c.page_stride, c.slot_stride, c.head_stride});
      };
      return (!r->q_heads || (rows_on(r->q, es, al, {r->q_stride_t, r->q_stride_h}) && rows_on(r->q_weight, es, al, {}) &&
                              rows_on(r->q_out, es, al, {r->q_out_stride_t, r->q_out_stride_h}))) &&
             (!r->k_heads || (rows_on(r->k, es, al, {r->k_stride_t, r->k_stride_h}) && rows_on(r->k_weight, es, al, {}) &&
                              (append || rows_on(r->k_out, es, al, {r->k_out_stride_t, r->k_out_stride_h})) &&
                              (!append || rows_on(r->v, es, al, {r->v_stride_t, r->v_stride_h})) && cache(r->k_cache) &&
                              cache(r->v_cache)));
    };
    const bool wide = r->dim % W == 0 && r->rot_offset % W == 0 && (r->interleaved ? r->rot_dim : r->rot_dim / 2) % W == 0 && views(W);
    if (!wide && !views(r->interleaved ? 2 : 1))
      return bad(r->interleaved ? "interleaved pairs must be aligned to a pair" : "unaligned tensors");
    NormArgs a{};
    a.x[0] = {r->q, r->q_out, r->q_stride_t, r->q_stride_h, r->q_out_stride_t, r->q_out_stride_h, r->q_weight};
    a.x[1] = {r->k, r->k_out, r->k_stride_t, r->k_stride_h, r->k_out_stride_t, r->k_out_stride_h, r->k_weight};
    a.x[2] = {r->v, nullptr, r->v_stride_t, r->v_stride_h, 0, 0, nullptr};
    const moe_cache_view_t* views_of[2] = {&r->k_cache, &r->v_cache};
    for (int i = 0; i < 2; ++i) {
      const moe_cache_view_t& c = *views_of[i];
      a.cache[i] = {c.data, c.scale, c.page_stride, c.slot_stride, c.head_stride, c.scale_page_stride, c.scale_slot_stride, c.scale_head_stride};
    }
    a.tokens = r->tokens; a.dim = r->dim; a.rot = r->rot_dim; a.offset = r->rot_offset;
    a.hq = r->q_heads; a.hk = r->k_heads; a.hv = kept ? r->k_heads : 0;
    a.scale = r->scale; a.eps = r->eps;
    a.positions = r->positions; a.inv_freq = r->inv_freq; a.slots = r->slots;
    a.kind = kept ? r->cache : MOE_CACHE_NONE;
    a.page = fast_div(1);
    if (kept) {
      a.num_slots = r->page_size * r->num_pages;
      a.page = fast_div(r->page_size);
    }
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_qk_norm_rope: no CUDA device");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched("moe_qk_norm_rope", r->dtype == MOE_DTYPE_FP32   ? launch_norm_typed<float>(a, r->interleaved, wide, sms, s)
                                        : r->dtype == MOE_DTYPE_FP16 ? launch_norm_typed<__half>(a, r->interleaved, wide, sms, s)
                                                                     : launch_norm_typed<__nv_bfloat16>(a, r->interleaved, wide, sms, s));
  });
}
