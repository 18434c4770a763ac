// Matrix-vector products with 4-bit weights: y[m, n] = sum_k x[m, k] * q[n, k] * s[n, k / group], and the
// gated form y = SiLU(gate) * up of two such products, for the few rows of a decode step.
//
// Every weight is read once, so HBM bounds the product: N * K / 2 bytes of codes and 4 bytes a group of
// scales.  A warp owns 16 weight rows and walks over K in blocks of 128; each lane loads 16 bytes (32 codes)
// of two rows straight into registers, several blocks ahead, so nothing waits on a barrier.  The codes
// become exact 16-bit floats (bf16 or fp16, the type of x) and enter m16n8k16 tensor-core products as the
// 16-row operand with up to 8 tokens as columns; the K order inside a block is the same permutation for both
// operands.  Products are exact and summed in fp32; each group's sum is scaled by its row's scale in fp32,
// and the only rounding to 16 bits is the one of y.  The warps of a CTA split K and meet in shared memory in
// a fixed order, so results do not depend on scheduling.
#include <cuda_runtime.h>

#include "step_ops.cuh"

namespace gbmoe {
namespace {

constexpr int kWarps = 8;
constexpr int kKBlock = 128;

struct LinearArgs {
  const void* x;       // [M, K], row stride ldx
  const uint8_t* w;    // [N or 2N, K / 2]
  const float* scale;  // [N or 2N, K / group]
  void* y;             // [M, N], row stride ldy
  long long ldx, ldy;
  int M, N, K;
};

// Eight int4 codes of one word -> four pairs (k0,k4) (k1,k5) (k2,k6) (k3,k7) of exact floats.
__device__ __forceinline__ void expand8(__half, uint32_t w, uint32_t r[4]) { s4x8_to_f16x8(w, r); }
// bf16: a biased nibble (k + 8 in [0, 15]) in the low mantissa bits of 128 (0x4300) reads 128 + (k + 8), since
// bf16's spacing is 1 on [128, 256); subtracting 136 leaves k exactly.
__device__ __forceinline__ void expand8(__nv_bfloat16, uint32_t w, uint32_t r[4]) {
  const __nv_bfloat162 bias = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = lop3_sel_xor(w >> (4 * i), 0x000f000fu, 0x43084308u);
    const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), bias);
    r[i] = *reinterpret_cast<const uint32_t*>(&q);
  }
}

template <int G> struct Lanes;  // codes a lane loads of one group: 4 / P words in each of P phases
template <> struct Lanes<128> { using Load = uint4; static constexpr int P = 1; };
template <> struct Lanes<64> { using Load = uint2; static constexpr int P = 2; };
template <> struct Lanes<32> { using Load = uint32_t; static constexpr int P = 4; };

template <typename L> __device__ __forceinline__ L load_codes(const uint8_t* p) {
  return __ldg(reinterpret_cast<const L*>(p));
}
template <> __device__ __forceinline__ uint4 load_codes<uint4>(const uint8_t* p) { return ld_stream_v4(p); }

template <typename T, int G, int NT, int RT, bool GATED>
__global__ void __launch_bounds__(kWarps * 32) linear_int4_kernel(LinearArgs a) {
  using LN = Lanes<G>;
  using Load = typename LN::Load;
  constexpr int P = LN::P, WP = 4 / P;
  constexpr int U = RT * NT > 2 ? 2 : 4;  // K blocks in flight a warp
  __shared__ float red[kWarps][RT * 16][NT * 8 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * (GATED ? RT * 8 : RT * 16);
  const int m0 = blockIdx.y * NT * 8;
  const int kbytes = a.K >> 1, nblk = (a.K + kKBlock - 1) / kKBlock, groups = a.K / G;
  pdl_trigger();
  pdl_wait();

  const uint8_t* wrow[RT][2];
  const float* srow[RT][2];
  bool live[RT][2];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // GATED: the first half of the row tiles holds gate rows, the second the matching up rows
      const int local = GATED ? (r % (RT / 2)) * 16 + h * 8 + g : r * 16 + h * 8 + g;
      const int n = n0 + local;
      live[r][h] = n < a.N;
      const long long row = live[r][h] ? (GATED && r >= RT / 2 ? static_cast<long long>(a.N) + n : n) : 0;
      wrow[r][h] = a.w + row * kbytes;
      srow[r][h] = a.scale + row * groups;
    }

  Load buf[U][RT][2][P];
  float sc[U][RT][2][P];
  auto fetch = [&](int b, int u) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int byte = b * (kKBlock / 2) + p * (G / 2) + t * (G / 8);
      const int gi = b * P + p;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool ok = live[r][h] && b < nblk && byte < kbytes;
          buf[u][r][h][p] = ok ? load_codes<Load>(wrow[r][h] + byte) : Load{};
          sc[u][r][h][p] = live[r][h] && b < nblk && gi < groups ? __ldg(srow[r][h] + gi) : 0.f;
        }
    }
  };

  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.f;

  const T* x = static_cast<const T*>(a.x);
  auto consume = [&](int b, int u) {
    if (b >= nblk) return;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float part[RT][NT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[r][n][i] = 0.f;
#pragma unroll
      for (int j = 0; j < WP; ++j) {
        const int k = b * kKBlock + p * G + t * (G / 4) + 8 * j;
        uint32_t q[RT][2][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            expand8(T(), reinterpret_cast<const uint32_t*>(&buf[u][r][h][p])[j], q[r][h]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int m = m0 + n * 8 + g;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (m < a.M && k < a.K) v = ld_v4(x + m * a.ldx + k);
          const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);  // (k0,k4) (k1,k5)
          const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);  // (k2,k6) (k3,k7)
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const uint32_t f0[4] = {q[r][0][0], q[r][1][0], q[r][0][1], q[r][1][1]};
            mma_16816(T(), part[r][n], f0, b0, b1);
            const uint32_t f1[4] = {q[r][0][2], q[r][1][2], q[r][0][3], q[r][1][3]};
            mma_16816(T(), part[r][n], f1, b2, b3);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][n][i] = fmaf(sc[u][r][i >> 1][p], part[r][n][i], acc[r][n][i]);
    }
  };

#pragma unroll
  for (int u = 0; u < U; ++u) fetch(warp + u * kWarps, u);
  for (int b = warp; b < nblk; b += U * kWarps) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      consume(b + u * kWarps, u);
      fetch(b + (U + u) * kWarps, u);
    }
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][r * 16 + (i >> 1) * 8 + g][n * 8 + 2 * t + (i & 1)] = acc[r][n][i];
  __syncthreads();
  constexpr int ROWS = GATED ? RT * 8 : RT * 16;
  T* y = static_cast<T*>(a.y);
  for (int i = threadIdx.x; i < ROWS * NT * 8; i += kWarps * 32) {
    const int r = i % ROWS, m = i / ROWS;
    if (n0 + r >= a.N || m0 + m >= a.M) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][r][m];
    if constexpr (GATED) {
      float up = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) up += red[w][ROWS + r][m];
      v = silu_f32(v) * up;
    }
    y[(m0 + m) * a.ldy + n0 + r] = Elem<T>::from_float(v);
  }
}

template <typename T, int G, int NT, int RT, bool GATED>
cudaError_t launch_one(const LinearArgs& a, cudaStream_t s) {
  const int rows = GATED ? RT * 8 : RT * 16;
  const dim3 grid((a.N + rows - 1) / rows, (a.M + NT * 8 - 1) / (NT * 8));
  return launch_kernel(linear_int4_kernel<T, G, NT, RT, GATED>, grid, dim3(kWarps * 32), 0, s, true, a);
}

template <typename T, int G>
cudaError_t launch_linear(const LinearArgs& a, bool gated, cudaStream_t s) {
  if (a.M <= 8) return gated ? launch_one<T, G, 1, 2, true>(a, s) : launch_one<T, G, 1, 1, false>(a, s);
  if (a.M <= 16) return gated ? launch_one<T, G, 2, 2, true>(a, s) : launch_one<T, G, 2, 2, false>(a, s);
  return gated ? launch_one<T, G, 4, 2, true>(a, s) : launch_one<T, G, 4, 2, false>(a, s);
}

template <typename T>
cudaError_t launch_typed(const LinearArgs& a, int group, bool gated, cudaStream_t s) {
  if (group == 128) return launch_linear<T, 128>(a, gated, s);
  if (group == 64) return launch_linear<T, 64>(a, gated, s);
  return launch_linear<T, 32>(a, gated, s);
}

}  // namespace
}  // namespace gbmoe

extern "C" moe_status_t moe_linear_int4(int dtype, const void* x, int64_t x_stride, const uint8_t* w, const float* w_scale,
                                        int M, int N, int K, int group, int gated, void* y, int64_t y_stride,
                                        moe_stream_t stream) {
  using namespace gbmoe;
  return guarded("moe_linear_int4", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_linear_int4: ") + m); };
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return bad("x must be bf16 or fp16");
    if (M < 0 || N <= 0 || K <= 0) return bad("sizes must be positive (M >= 0)");
    if (group != 32 && group != 64 && group != 128)
      return report_error(MOE_ERR_UNSUPPORTED, "moe_linear_int4: the group size must be 32, 64 or 128");
    if (K % group) return bad("K must be a multiple of the group size");
    if (gated != 0 && gated != 1) return bad("gated must be 0 or 1");
    if (M > (1 << 20) || N > (1 << 29) || K > (1 << 30))
      return report_error(MOE_ERR_UNSUPPORTED, "moe_linear_int4: problem too large");
    if (M == 0) return MOE_OK;
    if (!x || !w || !w_scale || !y) return bad("NULL pointer");
    if (x_stride < K || y_stride < N) return bad("rows overlap: a row stride is shorter than its row");
    if (!aligned(x, 16) || x_stride % 8 || !aligned(w, 16)) return bad("x rows and w must start on 16 bytes");
    if (!aligned(w_scale, 4) || !aligned(y, 2)) return bad("unaligned scales or output");
    const LinearArgs a{x, w, w_scale, y, x_stride, y_stride, M, N, K};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched("moe_linear_int4", dtype == MOE_DTYPE_FP16 ? launch_typed<__half>(a, group, gated, s)
                                                               : launch_typed<__nv_bfloat16>(a, group, gated, s));
  });
}
