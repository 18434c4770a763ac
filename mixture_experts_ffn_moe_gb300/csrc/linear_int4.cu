// Matrix-vector products with 4-bit weights: y[m, n] = sum_k x[m, k] * q[n, k] * s[n, k / group], and the
// gated form y = SiLU(gate) * up of two such products, for the few rows of a decode step.
//
// Every weight is read once, so HBM bounds the product: N * K / 2 bytes of codes and 4 bytes a group of
// scales.  A warp owns 32 weight rows (16 where that spreads better) and a share of K in blocks of 128; each
// lane loads 16 bytes (32 codes) of each of its rows straight into registers, blocks ahead of their use and
// across tiles, so the weight stream waits on no barrier.  The codes become fp16 and enter m16n8k16 tensor-core
// products as the 16-row operand with 8 tokens as columns.
//
// x is brought into the order in which the products take it: per block and 8 tokens four 16-byte pieces a lane,
// each 8 values paired (k0,k4) (k1,k5) (k2,k6) (k3,k7) as the codes come out of their words.  Like the layer's
// weight-only paths it is kept as fp16 in power-of-two frames, one per token and block: the block's largest |x|
// lies in [2^14, 2^15), so what fp16 rounds off (half a subnormal step of 2^-25, in the pieces that are stored divided by 16
// below) is at most 2^-35 of it, far below the fp32 sums.
//  * Up to 16 tokens whose x fits: every CTA (persistent, one an SM) does that itself into shared memory, where x
//    stays for all of its tiles: one launch.
//  * Otherwise a first kernel writes them to the workspace for the tcgen05 kernel (linear_int4_wide.cu).
//
// Expansion.  It is the integer pipe that limits this kernel beside HBM, so a pair of codes takes one LOP3 (and a
// word one shift): the biased code u = q + 8 stands alone in an fp16 as a subnormal, u * 2^-24, or 16 u * 2^-24
// where its nibble is the higher one; the tensor cores take subnormals exactly, and the pieces (k1,k5), (k3,k7)
// of x are stored divided by 16.  sum x u = sum x q + 8 sum x, so the accumulators of a group start at -8 times
// the group's sum of x (kept beside x).  All of that is exact but for the fp32 sums, which thus carry x (q + 8) and 8 x: a few
// units of 2^-24 of sum |x| (q + 16), where codes without a bias would have them of sum |x q|.  Where x holds an infinity
// or NaN the bias is subtracted from every code instead, so that they come out as they would.
//
// Each group's sum is scaled by its row's scale in fp32; the only rounding to 16 bits is the one of y.  The warps
// that share a tile's rows split K and meet in shared memory in a fixed order: results do not depend on scheduling.
//
// Measured: 8 rows, 129,280 x 7168 (495 MB): 102 us = 4.8 TB/s.  The loads alone take 83 us, bringing x into order 3, and the
// products' chain (expand, multiply, scale) the rest: four warps a scheduler, which 128 registers a thread allow, do not
// hide all of it, and the integer pipe is half busy.  More blocks in flight with fewer warps: the same.  4 rows, gated,
// 2 x 2048 x 7168: 7.6 us; 1 row, 7168 x 7168 (27 MB): 9.2 us, of which launch, x and the first weights' latency are about 5;
// 13 rows, 11,003 x 4000 in groups of 32 (codes in loads of 4 bytes): 19.5 us.  x is brought in by 16 values a thread: with 8,
// the indices and frames of 8 rows of 7168 took 14,000 cycles.
#include <cuda_runtime.h>

#include <type_traits>

#include "linear_int4.cuh"

namespace gbmoe {
namespace linear {
namespace {

constexpr int kKBlock = 128;
constexpr size_t kLinearSmem = 224 * 1024;

template <int N> constexpr int kLog2 = 1 + kLog2<N / 2>;
template <> constexpr int kLog2<1> = 0;
template <int RT> constexpr int kInFlight = RT == 1 ? 4 : 2;  // blocks in flight a warp: 128 bytes a lane

template <int G> struct Lanes;  // a lane's codes of a block: 4 / P words in each of P phases (one a group)
template <> struct Lanes<128> { using Load = uint4; static constexpr int P = 1; };
template <> struct Lanes<64> { using Load = uint2; static constexpr int P = 2; };
template <> struct Lanes<32> { using Load = uint32_t; static constexpr int P = 4; };

template <typename L> __device__ __forceinline__ L load_codes(const uint8_t* p) {
  return __ldg(reinterpret_cast<const L*>(p));
}
template <> __device__ __forceinline__ uint4 load_codes<uint4>(const uint8_t* p) { return ld_stream_v4(p); }

// One weight block's registers of a warp: codes and scales of RT tiles of 16 rows (rows g and g + 8 a lane).
template <int G, int RT> struct Block {
  typename Lanes<G>::Load c[RT][2][Lanes<G>::P];
  float s[RT][2];  // of group t of the block (t < P), shared in the quad
};

// Magnitudes of 16-bit floats are ordered like their bit patterns: the largest of 8, two at a time.
__device__ __forceinline__ uint32_t top_of(uint4 v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}
// Exponent of the frame of a block with these largest magnitudes.
template <typename T> __device__ __forceinline__ int frame_of(uint32_t top) {
  return x_frame_exp(Elem<T>::unpack(max(top & 0xffffu, top >> 16)).x);
}
// 8 neighbouring values in their frame and order: (k0,k4) (k1,k5)/16 (k2,k6) (k3,k7)/16.
template <typename T> __device__ __forceinline__ uint4 make_piece(uint4 v, float mul) {
  const float low = mul * 0.0625f;
  const float2 f01 = Elem<T>::unpack(v.x), f23 = Elem<T>::unpack(v.y), f45 = Elem<T>::unpack(v.z), f67 = Elem<T>::unpack(v.w);
  return make_uint4(pack_half2(f01.x * mul, f45.x * mul), pack_half2(f01.y * low, f45.y * low),
                    pack_half2(f23.x * mul, f67.x * mul), pack_half2(f23.y * low, f67.y * low));
}
// The sum of a group's values of one token (its G / 8 neighbouring threads' pieces), in the frame.
template <int G>
__device__ __forceinline__ float sum_of_group(uint4 h) {
  const float2 s0 = Elem<__half>::unpack(h.x), s1 = Elem<__half>::unpack(h.y), s2 = Elem<__half>::unpack(h.z), s3 = Elem<__half>::unpack(h.w);
  float sum = (s0.x + s0.y) + (s2.x + s2.y) + 16.f * ((s1.x + s1.y) + (s3.x + s3.y));
#pragma unroll
  for (int o = 1; o < G / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
constexpr float kMinusBias = -8.f * 0x1p-24f;  // of a code, in the units of the products

// The weight stream of a warp: its blocks of every tile of the CTA, in order.
template <int G, int RT, int NW> struct Stream {
  using LN = Lanes<G>;
  static constexpr int P = LN::P;
  const LinearArgs& a;
  int tile_rows, tiles, wk, wkid, nblk, full, groups, kbytes, rounds, rem, lane_row, wrow_base;
  int tile, it, blk, round;  // next block
  bool gated;
  const uint8_t* wbase;
  const float* sbase;
  long long up_w, up_s;
  uint32_t woff[RT][2], soff[RT][2];

  __device__ __forceinline__ Stream(const LinearArgs& args, int warp, int lane) : a(args) {
    gated = RT == 2 && a.gated;
    const int RW = gated ? 16 : RT * 16;
    wk = 1 << a.wk_log2;
    const int wrow = warp >> a.wk_log2;
    wkid = warp & (wk - 1);
    wrow_base = wrow * RW;
    lane_row = lane >> 2;
    kbytes = a.K >> 1;
    nblk = (a.K + kKBlock - 1) / kKBlock;
    full = a.K / kKBlock;
    groups = a.K / G;
    tile_rows = RW << (kLog2<NW> - a.wk_log2);
    tiles = a.tiles;
    rem = nblk & (wk - 1);
    rounds = (((nblk + wk - 1) >> a.wk_log2) + kInFlight<RT> - 1) / kInFlight<RT> * kInFlight<RT>;  // some may be empty
    up_w = gated ? static_cast<long long>(a.N) * kbytes : 0;
    up_s = gated ? static_cast<long long>(a.N) * groups : 0;
    tile = blockIdx.x;
    it = round = 0;
    enter(lane & 3);
  }
  // first block of the warp in the CTA's it-th tile: the longer shares go round
  __device__ __forceinline__ int start(int i) const { return (wkid + i * rem) & (wk - 1); }
  __device__ __forceinline__ void enter(int t) {
    const long long first = min(tile * tile_rows + wrow_base, a.N - 1);
    wbase = a.w + first * kbytes;
    sbase = a.scale + first * groups;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // rows past the last one read the last one again (and are not written); gated: tile 0 holds gate rows,
        // tile 1 the matching up rows
        const uint32_t d = min((gated ? 0 : r * 16) + h * 8 + lane_row, static_cast<int>(a.N - 1 - first));
        woff[r][h] = d * kbytes + t * (G / 8);
        soff[r][h] = d * groups + t % P;
      }
    blk = start(it);
  }
  __device__ __forceinline__ void fetch(Block<G, RT>& d, int t) {
    if (tile < tiles && blk < nblk) {
      const uint8_t* wp = wbase + static_cast<long long>(blk) * (kKBlock / 2);
      const float* sp = sbase + static_cast<long long>(blk) * P;
      if (blk < full) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p)
              d.c[r][h][p] = load_codes<typename LN::Load>(wp + (r == 1 ? up_w : 0) + woff[r][h] + p * (G / 2));
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) d.s[r][h] = __ldg(sp + (r == 1 ? up_s : 0) + soff[r][h]);
      } else {  // the last block of a K that is no multiple of 128: whole groups are missing
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p)
              d.c[r][h][p] = blk * P + p < groups ? load_codes<typename LN::Load>(wp + (r == 1 ? up_w : 0) + woff[r][h] + p * (G / 2))
                                                  : typename LN::Load{};
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            d.s[r][h] = blk * P + t % P < groups ? __ldg(sp + (r == 1 ? up_s : 0) + soff[r][h]) : 0.f;
      }
    }
    blk += wk;
    if (++round == rounds) {
      round = 0;
      tile += gridDim.x;
      ++it;
      if (tile < tiles) enter(t);
    }
  }
};

// acc += the block's products; xf: the block's pieces (offset of token tile n and step j by `piece`), sums as stored.
template <int G, int NT, int RT, bool PLAIN, typename Piece>
__device__ __forceinline__ void multiply(const Block<G, RT>& d, float (&acc)[RT][NT][4], const float* sums, int ld, int t, Piece piece) {
  constexpr int P = Lanes<G>::P, WP = 4 / P;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float part[RT][NT][4];
    if (p > 0 || !PLAIN) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[r][n][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < WP; ++j) {
      uint32_t q[RT][2][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          expand8(reinterpret_cast<const uint32_t*>(&d.c[r][h][p])[j], q[r][h]);
          if constexpr (!PLAIN) {
#pragma unroll
            for (int i = 0; i < 4; ++i) q[r][h][i] = unbias2(q[r][h][i], i & 1 ? 0x00800080u : 0x00080008u);
          }
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 v = piece(n, p * WP + j);
        if (PLAIN && j == 0) {
          const float2 c = *reinterpret_cast<const float2*>(sums + p * ld + n * 8 + 2 * t);
#pragma unroll
          for (int r = 0; r < RT; ++r) { part[r][n][0] = part[r][n][2] = c.x; part[r][n][1] = part[r][n][3] = c.y; }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const uint32_t f0[4] = {q[r][0][0], q[r][1][0], q[r][0][1], q[r][1][1]};
          mma_f16_16816(part[r][n], f0, v.x, v.y);
          const uint32_t f1[4] = {q[r][0][2], q[r][1][2], q[r][0][3], q[r][1][3]};
          mma_f16_16816(part[r][n], f1, v.z, v.w);
        }
      }
    }
    float sc[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) sc[r][h] = P == 1 ? d.s[r][h] : __shfl_sync(0xffffffffu, d.s[r][h], (threadIdx.x & 28) | p);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 fac = *reinterpret_cast<const float2*>(sums + P * ld + n * 8 + 2 * t);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[r][n][i] = fmaf(sc[r][i >> 1], part[r][n][i] * (i & 1 ? fac.y : fac.x), acc[r][n][i]);
    }
  }
}

// The warps of a row group meet ([warp][token][row] in shared memory) and y is written.
template <int NT, int RT, int NW>
__device__ __forceinline__ void join_and_write(const LinearArgs& a, const float (&acc)[RT][NT][4], float* red, int tile, int wk,
                                               bool gated, int m0, int live_m) {
  constexpr int PR = RT * 16 + 4;  // row pitch: no bank conflicts
  constexpr int NC = NT < 4 ? NT : 4;  // token tiles at once: room in shared memory
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int RW = gated ? 16 : RT * 16, wr = NW / wk;
  float* mine = red + warp * (NC * 8 * PR);
#pragma unroll
  for (int c = 0; c < NT; c += NC) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mine[(n * 8 + 2 * t + (i & 1)) * PR + r * 16 + (i >> 1) * 8 + g] = acc[r][c + n][i];
    __syncthreads();
    for (int i = tid; i < wr * NC * 8 * RW; i += NW * 32) {  // [row group][token][row], powers of two
      const int r = i & (RW - 1), gm = i / RW, m = gm % (NC * 8), grp = gm / (NC * 8);
      const int n = (tile * wr + grp) * RW + r;
      if (n >= a.N || c * 8 + m >= live_m) continue;
      const float* src = red + grp * wk * (NC * 8 * PR) + m * PR + r;
      float v = 0.f;
      for (int w = 0; w < wk; ++w) v += src[w * (NC * 8 * PR)];
      v *= 4096.f;
      if (gated) {
        float up = 0.f;
        for (int w = 0; w < wk; ++w) up += src[w * (NC * 8 * PR) + 16];
        v = silu_f32(v) * (up * 4096.f);
      }
      const long long at = (m0 + c * 8 + m) * a.ldy + n;
      if (a.bf16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
      else static_cast<__half*>(a.y)[at] = __float2half_rn(v);
    }
    __syncthreads();
  }
}

// Up to NT * 8 tokens, x in shared memory.
template <int G, int NT, int RT, int NW>
__global__ void __launch_bounds__(NW * 32, 1) linear_int4_kernel(LinearArgs a) {
  constexpr int P = Lanes<G>::P, U = kInFlight<RT>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int odd;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3;
  float* red = reinterpret_cast<float*>(smem);
  uint4* xf = reinterpret_cast<uint4*>(smem + NW * NT * 8 * (RT * 16 + 4) * 4);  // [block][token tile][4][32]
  const int nblk = (a.K + kKBlock - 1) / kKBlock;
  float* sums = reinterpret_cast<float*>(xf + nblk * NT * 128);                   // [block][P + 1][NT * 8]
  constexpr int LD = NT * 8;
  pdl_trigger();
  if (tid == 0) odd = 0;
  Stream<G, RT, NW> st(a, warp, lane);
  pdl_wait();

  // x: 8 neighbouring threads a block and token, two pieces of it each.  Tokens past the last one are left as they are:
  // columns of a product do not mix.  The first loads of x and of the weights are under way together.
  constexpr int B = 2;
  const int units = nblk * a.M * 8;
  uint4 v[B][2];
  auto load_x = [&](int w0) {
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int i = w0 + lane + k * NW * 32, b = div_by(i >> 3, a.tokens_div), m = (i >> 3) - b * a.M, col = b * kKBlock + (i & 7) * 8;
      const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ldx + col);
      v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      if (i < units && col < a.K) v[k][0] = at[0];
      if (i < units && col + 64 < a.K) v[k][1] = at[8];
    }
  };
  load_x(warp * 32);
  Block<G, RT> buf[U];
#pragma unroll
  for (int u = 0; u < U; ++u) st.fetch(buf[u], t);
  auto stage = [&](auto type) {
    using T = decltype(type);
    for (int w0 = warp * 32; w0 < units; w0 += B * NW * 32) {  // whole warps: the threads of a block talk to each other
      if (w0 != warp * 32) load_x(w0);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (w0 + k * NW * 32 >= units) break;
        uint32_t top = __vmaxu2(top_of(v[k][0]), top_of(v[k][1]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int i = w0 + lane + k * NW * 32, b = div_by(i >> 3, a.tokens_div), m = (i >> 3) - b * a.M;
        const int fe = frame_of<T>(top), c = i & 7;
        const float mul = exp2i(-fe);
        if (i < units) {
          uint4* to = xf + (b * NT + (m >> 3)) * 128 + (m & 7) * 4;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int p = (c + 8 * h) / (G / 8), cp = (c + 8 * h) % (G / 8);
            to[(p * (4 / P) + cp % (G / 32)) * 32 + cp / (G / 32)] = make_piece<T>(v[k][h], mul);
          }
          if (c == 0) sums[(b * (P + 1) + P) * LD + m] = exp2i(fe + 12);
        }
      }
    }
  };
  if (a.bf16) stage(__nv_bfloat16{}); else stage(__half{});
  __syncthreads();
  // the groups' sums: products with rows of ones (16 where the pieces stand divided by 16)
#pragma unroll 2
  for (int bn = warp; bn < nblk * NT; bn += NW) {
    const int b = bn / NT, m = bn % NT * 8 + 2 * t;
    const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x4c004c00u, 0x4c004c00u};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float d[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4 / P; ++j) {
        const uint4 x = xf[bn * 128 + (p * (4 / P) + j) * 32 + lane];
        mma_f16_16816(d, ones, x.x, x.y);
        mma_f16_16816(e, ones, x.z, x.w);
      }
      d[0] += e[0];
      d[1] += e[1];
      if (lane < 4) {  // row 0, tokens m and m + 1
        *reinterpret_cast<float2*>(sums + (b * (P + 1) + p) * LD + m) = make_float2(d[0] * kMinusBias, d[1] * kMinusBias);
        if ((m < a.M && !(fabsf(d[0]) < INFINITY)) || (m + 1 < a.M && !(fabsf(d[1]) < INFINITY))) odd = 1;
      }
    }
  }
  __syncthreads();
  const bool plain = !odd;
  for (int it = 0, tile = blockIdx.x; tile < st.tiles; ++it, tile += gridDim.x) {
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.f;
    int blk = st.start(it);
    auto run = [&](auto p) {
      for (int rd = 0; rd < st.rounds; rd += U)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (blk < nblk)
            multiply<G, NT, RT, decltype(p)::value>(buf[u], acc, sums + blk * (P + 1) * LD, LD, t,
                                                    [&](int n, int j) { return xf[(blk * NT + n) * 128 + j * 32 + lane]; });
          blk += st.wk;
          st.fetch(buf[u], t);
        }
    };
    if (plain) run(std::true_type{}); else run(std::false_type{});
    join_and_write<NT, RT, NW>(a, acc, red, tile, st.wk, st.gated, 0, a.M);
  }
}

// x into the workspace: a CTA a block of K and 16 tokens, 16 threads a token.
template <int G>
__global__ void __launch_bounds__(256) linear_pieces_kernel(LinearArgs a) {
  constexpr int P = Lanes<G>::P;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, c = threadIdx.x & 15, col = b * kKBlock + c * 8, m = blockIdx.y * 16 + (threadIdx.x >> 4);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (m < a.M && col < a.K) v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ldx + col);
  uint32_t top = top_of(v);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int fe = a.bf16 ? frame_of<__nv_bfloat16>(top) : frame_of<__half>(top);
  const float mul = exp2i(-fe);
  const uint4 x = a.bf16 ? make_piece<__nv_bfloat16>(v, mul) : make_piece<__half>(v, mul);
  const float sum = sum_of_group<G>(x);
  const int part = m / a.mt, mp = m - part * a.mt;
  float* sums = a.sums + (static_cast<long long>(b) * (a.tokens / a.mt) + part) * ((P + 1) * a.mt + 4);
  if (m < a.M) {
    a.xf[static_cast<long long>(m) * gridDim.x * 16 + b * 16 + c] = x;
    if (c % (G / 8) == 0) sums[c / (G / 8) * a.mt + mp] = sum * kMinusBias;
    if (c == 0) sums[P * a.mt + mp] = exp2i(fe + 12);
  }
  const bool odd = __syncthreads_or(!(fabsf(sum) < INFINITY) && m < a.M);
  if (threadIdx.x == 0) {
    sums[(P + 1) * a.mt + mp / 16] = odd ? 1.f : 0.f;
    if (b == 0 && blockIdx.y == 0) *a.status = DeviceStatus{};
  }
}

// Blocks of K that a CTA of the one-launch kernel can hold for nt tiles of 8 tokens.
int resident_blocks(int group, int nt) {
  return static_cast<int>((kLinearSmem - 16 * nt * 8 * 36 * 4) / (static_cast<size_t>(nt) * (2048 + (128 / group + 1) * 32)));
}

// Warps that share a tile's blocks: the split of least time, counted in blocks a warp (a tile's join costs one).
int choose_wr(const LinearArgs& a, int RW, int NW, int sms) {
  const int nblk = (a.K + kKBlock - 1) / kKBlock;
  long long best = -1;
  int wr = 1;
  for (int r = 1; r <= NW; r *= 2) {
    const long long tiles = (a.N + static_cast<long long>(RW) * r - 1) / (static_cast<long long>(RW) * r), wk = NW / r;
    const long long cost = (tiles + sms - 1) / sms * ((nblk + wk - 1) / wk + 1);
    if (best < 0 || cost < best) { best = cost; wr = r; }
  }
  return wr;
}

template <int G, int NT, int RT>
cudaError_t launch_resident(LinearArgs a, int sms, cudaStream_t s) {
  constexpr int NW = 16;
  const int RW = a.gated ? 16 : RT * 16, nblk = (a.K + kKBlock - 1) / kKBlock;
  const int wr = choose_wr(a, RW, NW, sms);
  a.wk_log2 = 0;
  while ((wr << a.wk_log2) < NW) ++a.wk_log2;
  a.tiles = (a.N + RW * wr - 1) / (RW * wr);
  a.tokens_div = fast_div(a.M);
  auto kern = linear_int4_kernel<G, NT, RT, NW>;
  cudaError_t err = set_smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(kLinearSmem));
  if (err != cudaSuccess) return err;
  const size_t smem = NW * NT * 8 * (RT * 16 + 4) * 4 + static_cast<size_t>(nblk) * NT * (2048 + (Lanes<G>::P + 1) * 32);
  return launch_kernel(kern, dim3(a.tiles < sms ? a.tiles : sms), dim3(NW * 32), smem, s, true, a);
}

template <int G>
cudaError_t launch_linear(const LinearArgs& a, const WidePlan* wide, int sms, cudaStream_t s) {
  if (!wide) {
    // 16 or 32 rows a warp: whichever leaves the busiest SM with fewer rows.  With two token tiles 16 rows take about a
    // quarter more instructions a row, so they have to save more: 16 tokens, 7168 x 5376: 14.7 us (32 rows: 16.8), 2048 x 4096:
    // 8.3 us (9.8); 13 tokens, 11003 x 4000 in groups of 32 (80 rows instead of 96): 19.8 us (19.3).
    const int t1 = (a.N + 15) / 16, t2 = (a.N + 31) / 32;
    const int r1 = (t1 + sms - 1) / sms * 16, r2 = (t2 + sms - 1) / sms * 32;
    if (a.M > 8) return !a.gated && 5 * r1 < 4 * r2 ? launch_resident<G, 2, 1>(a, sms, s) : launch_resident<G, 2, 2>(a, sms, s);
    return !a.gated && r1 < r2 ? launch_resident<G, 1, 1>(a, sms, s) : launch_resident<G, 1, 2>(a, sms, s);
  }
  cudaError_t err = launch_kernel(linear_pieces_kernel<G>, dim3((a.K + kKBlock - 1) / kKBlock, a.tokens / 16), dim3(256), 0, s, true, a);
  return err != cudaSuccess ? err : launch_wide_tc(a, G, *wide, s);
}

bool needs_workspace(int M, int K, int group) {
  return M > 16 || (K + kKBlock - 1) / kKBlock > resident_blocks(group, M <= 8 ? 1 : 2);
}

struct LinearLayout { size_t x = 0, sums = 0, part = 0, total = 0; };  // the status words stand first
LinearLayout linear_layout(int K, int group, const WidePlan& p) {
  LinearLayout l;
  const size_t nblk = (static_cast<size_t>(K) + kKBlock - 1) / kKBlock, tokens = static_cast<size_t>(p.parts) * p.mt;
  size_t at = kStatusBytes;
  auto take = [&](size_t n) { const size_t r = at; at = (at + n + 255) / 256 * 256; return r; };
  l.x = take(tokens * nblk * 256);
  l.sums = take(nblk * p.parts * 4 * ((128 / group + 1) * static_cast<size_t>(p.mt) + 4));
  l.part = take(p.part_bytes);
  l.total = at;
  return l;
}

bool valid_sizes(int M, int N, int K) {
  return M <= (1 << 19) && N <= (1 << 29) && K <= (1 << 25);  // (65,535 parts of 16 tokens at most)
}

}  // namespace
}  // namespace linear
}  // namespace gbmoe

extern "C" size_t moe_linear_int4_workspace_size(int M, int N, int K, int group, int gated) {
  using namespace gbmoe;
  using namespace gbmoe::linear;
  if (M <= 0 || N <= 0 || K <= 0 || !valid_sizes(M, N, K) || (group != 32 && group != 64 && group != 128) || K % group ||
      !needs_workspace(M, K, group))
    return 0;
  const int sms = num_sms_current();
  return linear_layout(K, group, wide_plan(M, N, K, group, gated != 0, sms > 0 ? sms : kMaxSms)).total;
}

extern "C" moe_status_t moe_linear_int4(int dtype, const void* x, int64_t x_stride, const uint8_t* w, const float* w_scale,
                                        int M, int N, int K, int group, int gated, void* y, int64_t y_stride,
                                        void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  using namespace gbmoe;
  using namespace gbmoe::linear;
  return guarded("moe_linear_int4", [&]() -> moe_status_t {
    auto bad = [](const char* m) { return report_error(MOE_ERR_INVALID_ARG, std::string("moe_linear_int4: ") + m); };
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return bad("x must be bf16 or fp16");
    if (M < 0 || N <= 0 || K <= 0) return bad("sizes must be positive (M >= 0)");
    if (group != 32 && group != 64 && group != 128)
      return report_error(MOE_ERR_UNSUPPORTED, "moe_linear_int4: the group size must be 32, 64 or 128");
    if (K % group) return bad("K must be a multiple of the group size");
    if (gated != 0 && gated != 1) return bad("gated must be 0 or 1");
    if (!valid_sizes(M, N, K))
      return report_error(MOE_ERR_UNSUPPORTED, "moe_linear_int4: problem too large");
    if (M == 0) return MOE_OK;
    if (!x || !w || !w_scale || !y) return bad("NULL pointer");
    if (x_stride < K || y_stride < N) return bad("rows overlap: a row stride is shorter than its row");
    if (!aligned(x, 16) || x_stride % 8 || !aligned(w, 16)) return bad("x rows and w must start on 16 bytes");
    if (!aligned(w_scale, 4) || !aligned(y, 2)) return bad("unaligned scales or output");
    const int sms = num_sms_current();
    if (sms <= 0) return report_error(MOE_ERR_CUDA, "moe_linear_int4: no CUDA device");
    LinearArgs a{};
    a.x = x; a.w = w; a.scale = w_scale; a.y = y;
    a.ldx = x_stride; a.ldy = y_stride;
    a.M = M; a.N = N; a.K = K; a.gated = gated; a.bf16 = dtype == MOE_DTYPE_BF16;
    WidePlan p;
    const bool wide = needs_workspace(M, K, group);
    if (wide) {
      p = wide_plan(M, N, K, group, gated, sms);
      const LinearLayout l = linear_layout(K, group, p);
      if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256))
        return report_error(MOE_ERR_WORKSPACE, "moe_linear_int4: workspace NULL, misaligned or too small");
      char* ws = static_cast<char*>(workspace);
      a.tokens = p.parts * p.mt;
      a.mt = p.mt;
      a.status = reinterpret_cast<DeviceStatus*>(ws);
      a.xf = reinterpret_cast<uint4*>(ws + l.x);
      a.sums = reinterpret_cast<float*>(ws + l.sums);
      a.part = reinterpret_cast<float*>(ws + l.part);
    }
    const WidePlan* wp = wide ? &p : nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched("moe_linear_int4", group == 128 ? launch_linear<128>(a, wp, sms, s)
                                       : group == 64 ? launch_linear<64>(a, wp, sms, s) : launch_linear<32>(a, wp, sms, s));
  });
}
