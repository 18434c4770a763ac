// Rotary positions: turns pairs of every query and key head by an angle that grows with the token's
// position, and optionally appends keys and values to a paged cache in the same pass.
//
// Mathematics.  Pair i of a head at position p turns by p * f_i radians:
//   y0 = (x0 cos - x1 sin) * scale,  y1 = (x1 cos + x0 sin) * scale.
// The angle needs more than fp32: at p = 10^6 an fp32 product is off by up to 0.06 radians.  Here f_i is
// turned once per CTA into a 64-bit fraction of a turn, F = round(f_i / (2 pi) * 2^64) mod 2^64; p * F in
// wrapping 64-bit integers is the angle modulo a turn, off by at most p * f_i * 2^-52 (f_i / (2 pi) in fp64) and
// p * 2^-62 radians, whatever the position.  The nearest quarter turn is taken off in integers, so that what is
// converted to fp32 for sincospif keeps 24 bits however small it is: sine and cosine are then right to a few units of
// their own last place.  No table of positions is kept.
//
// Bound: HBM for prompts (every element is read and written once), launch latency for decode steps.  Measured: 16,384
// tokens, 64 / 8 heads (302 MB) in 54.7 us = 5.5 TB/s; 32 tokens, 32 / 8 heads with the append in 2.8 us.
#include <cuda_runtime.h>

#include "step_ops.cuh"

namespace gbmoe {
namespace {

constexpr int kRopeThreads = 256;

struct RopeView {  // [token, head, dim], dim contiguous, strides in elements
  const void* in;
  void* out;
  long long in_t, in_h, out_t, out_h;
};

struct RopeKernelArgs {
  RopeView q, k, v;
  int tokens, dim, rot, offset;
  int hq, hk, hv;
  float scale;
  int inverse;
  const int32_t* positions;
  const double* inv_freq;
  const int32_t* slots;  // null: k goes to its own rows
  int num_slots;
  FastDiv page;          // slots a page
  long long kc_page, kc_slot, kc_head, vc_page, vc_slot, vc_head;
  int tile;              // tokens a CTA turns at once
  int units;             // vectors (or pairs of vectors) of a head that one thread handles in turn
  FastDiv unit_div, heads_div;
};

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T e[V]; };

template <typename T> __device__ __forceinline__ float as_float(T a) { return Elem<T>::to_float(a); }
template <> __device__ __forceinline__ float as_float<float>(float a) { return a; }
template <typename T> __device__ __forceinline__ T as_elem(float a) { return Elem<T>::from_float(a); }
template <> __device__ __forceinline__ float as_elem<float>(float a) { return a; }

// V elements a vector.  A head is cut into units: in the halves layout a unit inside the turning part is two
// vectors (one of each half), in the interleaved layout one vector of V / 2 pairs; outside that part a unit
// is one vector that is copied.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeKernelArgs a) {
  extern __shared__ float2 table[];  // [tile][rot / 2] (cos, sin) * scale, then [rot / 2] turn fractions
  const int half = a.rot >> 1;
  uint64_t* turns = reinterpret_cast<uint64_t*>(table + a.tile * half);
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const double r = a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    turns[i] = static_cast<uint64_t>(__double2ll_rn((r - rint(r)) * 18446744073709551616.0));
  }
  __syncthreads();
  const int heads = a.hq + a.hk + a.hv;
  const int unit0 = a.offset / V;  // units before the turning part
  const int turning = INTER ? a.rot / V : half / V;
  for (int t0 = blockIdx.x * a.tile; t0 < a.tokens; t0 += gridDim.x * a.tile) {
    const int nt = min(a.tile, a.tokens - t0);
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
      const int t = i / half, f = i - t * half;
      const uint64_t angle = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t0 + t])) * turns[f];
      const uint64_t quarter = (angle + (1ull << 61)) >> 62;  // the nearest one (4 stands for 0)
      // the rest (below 2^61 on either side) as high * 2^32 + low with both signed: two conversions of 32 bits at once are
      // 0.1 us of a decode step's 2.8 quicker than one of 64
      const uint64_t rest = angle - (quarter << 62);
      const int32_t low = static_cast<int32_t>(rest), high = static_cast<int32_t>((rest + (1ull << 31)) >> 32);
      float sn, cs;
      sincospif(fmaf(__int2float_rn(high), 0x1p-31f, __int2float_rn(low) * 0x1p-63f), &sn, &cs);
      if (quarter & 1) { const float c = cs; cs = -sn; sn = c; }
      if (quarter & 2) { cs = -cs; sn = -sn; }
      table[i] = make_float2(cs * a.scale, (a.inverse ? -sn : sn) * a.scale);
    }
    __syncthreads();
    const int work = nt * heads * a.units;
    for (int w = blockIdx.y * kRopeThreads + threadIdx.x; w < work; w += gridDim.y * kRopeThreads) {
      const int hw = div_by(w, a.unit_div), u = w - hw * a.units;
      const int t = div_by(hw, a.heads_div), head = hw - t * heads, tok = t0 + t;
      const T* src;
      T* dst;
      bool turn = u >= unit0 && u < unit0 + turning;
      if (head < a.hq) {
        src = static_cast<const T*>(a.q.in) + tok * a.q.in_t + head * a.q.in_h;
        dst = static_cast<T*>(a.q.out) + tok * a.q.out_t + head * a.q.out_h;
      } else {
        const bool is_v = head >= a.hq + a.hk;
        const RopeView& x = is_v ? a.v : a.k;
        const int h = head - a.hq - (is_v ? a.hk : 0);
        src = static_cast<const T*>(x.in) + tok * x.in_t + h * x.in_h;
        if (a.slots) {
          const int slot = a.slots[tok];
          if (slot < 0 || slot >= a.num_slots) continue;  // a row that is not kept
          const int page = div_by(slot, a.page), at = slot - page * a.page.d;
          dst = static_cast<T*>(x.out) + (is_v ? page * a.vc_page + at * a.vc_slot + h * a.vc_head
                                               : page * a.kc_page + at * a.kc_slot + h * a.kc_head);
        } else {
          dst = static_cast<T*>(x.out) + tok * x.out_t + h * x.out_h;
        }
        turn = turn && !is_v;
      }
      using W = Vec<T, V>;
      if constexpr (INTER) {
        W x = *reinterpret_cast<const W*>(src + u * V);
        if (turn) {
          const float2* cs = table + t * half + (u - unit0) * (V / 2);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float p = as_float<T>(x.e[2 * i]), r = as_float<T>(x.e[2 * i + 1]);
            x.e[2 * i] = as_elem<T>(p * cs[i].x - r * cs[i].y);
            x.e[2 * i + 1] = as_elem<T>(r * cs[i].x + p * cs[i].y);
          }
        }
        *reinterpret_cast<W*>(dst + u * V) = x;
      } else {
        // units: [0, unit0) copied, [unit0, unit0 + turning) pairs of vectors, the rest copied
        const int inside = u >= unit0 && u < unit0 + turning;
        const int c0 = u < unit0 + turning ? u * V : u * V + half;  // past the turning part: its second half is done
        W x = *reinterpret_cast<const W*>(src + c0);
        if (inside) {
          W y = *reinterpret_cast<const W*>(src + c0 + half);
          if (turn) {
            const float2* cs = table + t * half + (u - unit0) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float p = as_float<T>(x.e[i]), r = as_float<T>(y.e[i]);
              x.e[i] = as_elem<T>(p * cs[i].x - r * cs[i].y);
              y.e[i] = as_elem<T>(r * cs[i].x + p * cs[i].y);
            }
          }
          *reinterpret_cast<W*>(dst + c0 + half) = y;
        }
        *reinterpret_cast<W*>(dst + c0) = x;
      }
    }
    __syncthreads();
  }
}

template <typename T, int V>
cudaError_t launch_rope(RopeKernelArgs& a, bool inter, int sms, cudaStream_t s) {
  a.units = inter ? a.dim / V : (a.dim - a.rot / 2) / V;
  a.unit_div = fast_div(a.units);
  a.heads_div = fast_div(a.hq + a.hk + a.hv);
  // up to 4 tokens a CTA: several waves, so that tables are made while other CTAs stream (16384 tokens of 72 x 64
  // elements, GB300, one 32-bit division slower than now: tiles of 2, 4, 8, 16 59.7, 55.8, 61.7, 61.1 us)
  int tile = 1;
  while (tile < 4 && static_cast<long long>(a.tokens) > 2LL * sms * tile) tile *= 2;
  while (tile > 1 && (tile + 1) * (a.rot / 2) * 8 > 48 * 1024) tile /= 2;  // the table's shared memory
  a.tile = tile;
  const size_t smem = static_cast<size_t>(tile) * (a.rot / 2) * 8 + (a.rot / 2) * 8;
  const int ctas = (a.tokens + tile - 1) / tile;
  const int per = tile * (a.hq + a.hk + a.hv) * a.units;
  int gy = 1;
  while (gy < 8 && ctas * gy < 2 * sms && per > gy * kRopeThreads) gy *= 2;
  const int gx = ctas;
  auto kern = inter ? rope_kernel<T, V, true> : rope_kernel<T, V, false>;
  return launch_kernel(kern, dim3(gx, gy), dim3(kRopeThreads), smem, s, true, a);
}

template <typename T>
cudaError_t launch_rope_typed(RopeKernelArgs& a, bool inter, bool wide, int sms, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  if (wide) return launch_rope<T, W>(a, inter, sms, s);
  return inter ? launch_rope<T, 2>(a, inter, sms, s) : launch_rope<T, 1>(a, inter, sms, s);
}

bool view_ok(const void* p, long long st, long long sh, size_t es, size_t al) {
  return aligned(p, al) && (st * static_cast<long long>(es)) % static_cast<long long>(al) == 0 &&
         (sh * static_cast<long long>(es)) % static_cast<long long>(al) == 0;
}

}  // namespace
}  // namespace gbmoe

extern "C" moe_status_t moe_rope(const moe_rope_args_t* r, moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_rope", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_rope: ") + m); };
    if (!r) return bad("NULL arguments");
    const size_t es = r->dtype == MOE_DTYPE_FP32 ? 4 : 2;
    if (r->dtype != MOE_DTYPE_BF16 && r->dtype != MOE_DTYPE_FP16 && r->dtype != MOE_DTYPE_FP32)
      return bad("unknown dtype");
    if (r->tokens < 0 || r->q_heads < 0 || r->k_heads < 0 || r->dim <= 0) return bad("sizes must be positive");
    if (r->rot_dim <= 0 || r->rot_dim % 2 || r->rot_offset < 0 || r->rot_offset + static_cast<long long>(r->rot_dim) > r->dim)
      return bad("the turning part must be even and lie inside the head");
    if (r->interleaved && (r->rot_offset % 2 || r->dim % 2))
      return bad("interleaved pairs need an even offset and an even head");
    if (r->dim > 1024 || r->q_heads > 4096 || r->k_heads > 4096)
      return report_error(MOE_ERR_UNSUPPORTED, "moe_rope: heads above 1024 elements or more than 4096 heads");
    const bool append = r->slots != nullptr;
    if (append && (r->page_size <= 0 || r->num_pages <= 0)) return bad("a cache needs pages");
    if (append && static_cast<long long>(r->page_size) * r->num_pages > 0x7fffffffLL)
      return report_error(MOE_ERR_UNSUPPORTED, "moe_rope: more than 2^31 - 1 cache slots");
    if (r->tokens == 0 || r->q_heads + r->k_heads == 0) return MOE_OK;
    if (!r->positions || !r->inv_freq) return bad("NULL positions or frequencies");
    if (r->q_heads && (!r->q || !r->q_out)) return bad("NULL queries");
    if (r->k_heads && (!r->k || !r->k_out)) return bad("NULL keys");
    if (append && (!r->v || !r->v_cache)) return bad("NULL values");
    // 16-byte vectors where every row, every half and every edge of the turning part starts on one
    const int W = static_cast<int>(16 / es);
    bool wide = r->dim % W == 0 && r->rot_offset % W == 0 && (r->interleaved ? r->rot_dim : r->rot_dim / 2) % W == 0;
    auto views = [&](size_t al) {
      return (!r->q_heads || (view_ok(r->q, r->q_stride_t, r->q_stride_h, es, al) &&
                              view_ok(r->q_out, r->q_out_stride_t, r->q_out_stride_h, es, al))) &&
             (!r->k_heads ||
              (view_ok(r->k, r->k_stride_t, r->k_stride_h, es, al) &&
               view_ok(r->k_out, r->k_out_stride_t, r->k_out_stride_h, es, al) &&
               (!append || (r->k_page_stride * static_cast<long long>(es) % static_cast<long long>(al) == 0 &&
                            view_ok(r->v, r->v_stride_t, r->v_stride_h, es, al) &&
                            view_ok(r->v_cache, r->v_slot_stride, r->v_head_stride, es, al) &&
                            r->v_page_stride * static_cast<long long>(es) % static_cast<long long>(al) == 0))));
    };
    wide = wide && views(16);
    if (!wide && !views(r->interleaved ? 2 * es : es))
      return bad(r->interleaved ? "interleaved pairs must be aligned to a pair" : "unaligned tensors");
    RopeKernelArgs a{};
    a.q = {r->q, r->q_out, r->q_stride_t, r->q_stride_h, r->q_out_stride_t, r->q_out_stride_h};
    a.k = {r->k, r->k_out, r->k_stride_t, r->k_stride_h, r->k_out_stride_t, r->k_out_stride_h};
    a.v = {r->v, r->v_cache, r->v_stride_t, r->v_stride_h, 0, 0};
    a.tokens = r->tokens; a.dim = r->dim; a.rot = r->rot_dim; a.offset = r->rot_offset;
    a.hq = r->q_heads; a.hk = r->k_heads; a.hv = append ? r->k_heads : 0;
    a.scale = r->scale; a.inverse = r->inverse;
    a.positions = r->positions; a.inv_freq = r->inv_freq;
    a.slots = r->slots;
    if (append) {
      a.num_slots = r->page_size * r->num_pages;
      a.page = fast_div(r->page_size);
      a.kc_page = r->k_page_stride; a.kc_slot = r->k_out_stride_t; a.kc_head = r->k_out_stride_h;
      a.vc_page = r->v_page_stride; a.vc_slot = r->v_slot_stride; a.vc_head = r->v_head_stride;
    }
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_rope: no CUDA device");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = r->dtype == MOE_DTYPE_FP32 ? launch_rope_typed<float>(a, r->interleaved, wide, sms, s)
                      : r->dtype == MOE_DTYPE_FP16 ? launch_rope_typed<__half>(a, r->interleaved, wide, sms, s)
                                                   : launch_rope_typed<__nv_bfloat16>(a, r->interleaved, wide, sms, s);
    return launched("moe_rope", err);
  });
}
