// Shared parts of the 4-bit linear kernels.
#pragma once

#include "step_ops.cuh"

namespace gbmoe {
namespace linear {

struct LinearArgs {
  const void* x;       // [M, K], row stride ldx
  const uint8_t* w;    // [N or 2N, K / 2]
  const float* scale;  // [N or 2N, K / group]
  void* y;             // [M, N], row stride ldy
  long long ldx, ldy;
  int M, N, K, gated, bf16;
  // one launch: warps that split the K of a tile (log2; the others take other rows), tiles
  int wk_log2, tiles;
  FastDiv tokens_div;
  // with a workspace: x as the products take it
  int tokens;          // M rounded up to whole products
  uint4* xf;           // fp16 [tokens][blocks * 128], each 8 columns in the codes' order
  int mt;              // tokens of a product
  float* sums;         // [blocks][tokens / mt][(P + 1) * mt + 4]: -8 * 2^-24 * the groups' sums, 2^(frame + 12), and
                       // for every 16 tokens a mark that is not 0 where they hold infinities or NaN
  float* part;         // fp32 parts of cut tiles
  DeviceStatus* status;
  long long chunk;     // blocks a CTA
};

// Pairs (k0,k4) (k1,k5) (k2,k6) (k3,k7) of a word's biased codes: u, 16 u, u, 16 u in units of 2^-24.
__device__ __forceinline__ void expand8(uint32_t w, uint32_t r[4]) {
  const uint32_t v = w >> 8;
  r[0] = lop3_sel_xor(w, 0x000f000fu, 0x00080008u);
  r[1] = lop3_sel_xor(w, 0x00f000f0u, 0x00800080u);
  r[2] = lop3_sel_xor(v, 0x000f000fu, 0x00080008u);
  r[3] = lop3_sel_xor(v, 0x00f000f0u, 0x00800080u);
}
// The codes themselves, q or 16 q in units of 2^-24 (exact).
__device__ __forceinline__ uint32_t unbias2(uint32_t v, uint32_t bias) {
  const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&q);
}

// How a call with a workspace is cut (linear_int4_wide.cu).
struct WidePlan {
  int mt = 0, parts = 0, ctas = 0;  // tokens of a product, parts of the tokens, CTAs a part
  bool cut = false;
  long long chunk = 0;
  size_t part_bytes = 0;
};
WidePlan wide_plan(int M, int N, int K, int group, int gated, int sms);
cudaError_t launch_wide_tc(const LinearArgs& a, int group, const WidePlan& p, cudaStream_t s);

}  // namespace linear
}  // namespace gbmoe
