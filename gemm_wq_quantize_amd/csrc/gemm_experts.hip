// The experts' int4 products (gfx950): rows sorted by expert, each expert with
// a packed weight matrix of its own.
//
//   C[i][j] = sum_k A[src(i)][k] * (q[e][j][k] - z) * s[e][j][k / group],  e = bin of row i
//
// src(i) is i, or order[i] / topk when A holds the tokens' rows: the gather
// happens in the operand loads and no sorted copy of A is made.  The host knows
// the number of rows but not how they fall, so a launch covers the most row
// tiles that they can make; each workgroup finds its tile from the offsets and
// those past the last one return.
#include "route_tiles.h"
#include "w4_unpack.h"

namespace wq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------ up to 16 rows a tile
//
// Bound by the weights' bytes.  A workgroup computes 16 rows x 16 CB columns
// with v_mfma_f32_16x16x32_bf16; its four waves take every fourth chunk of k
// and join their sums in LDS.  Operands come from memory straight into
// registers: a lane holds 8 LW consecutive k of one column (LW packed words)
// and the same k of one row, so slot k of MFMA w is k = chunk + 8 LW (lane /
// 16) + 8 w + (0..7) on both sides.
//
// The codes enter the MFMA as 128 + q, exact in bf16, and a chunk lies in one
// group, so
//   sum_chunk A (q - z) s = s (sum A (128 + q) - (128 + z) sum A)
// with the row sums from one more MFMA per word against ones: they arrive in
// the accumulator's own layout.  No weight is rounded, and the unpacking is 7
// VALU instructions a word instead of the 17 that scaling each weight takes.
//
// Rows past the tile's last and columns past n repeat the last one: their
// results are not stored, and their loads hit the lines of the others.
struct EArgs {
  const uint16_t* a;
  const int* order;     // nullable: A's row of sorted row i is order[i] / topk
  const int* offsets;
  const uint8_t* b;
  const uint16_t* scales;
  const uint16_t* zeros;  // nullable
  uint16_t* c;
  int64_t n, k;
  float zero_const;
  int topk, a_rows, slots, experts;
  int tiles_n;
  int ngroups;      // k / group
  int group_chunks; // chunks per group
};

// the row of A that sorted row i reads; a position outside A reads its row 0
__device__ __forceinline__ int64_t a_row(const EArgs& p, int i) {
  if (!p.order) return i;
  const int r = p.order[i] / p.topk;
  return (unsigned)r < (unsigned)p.a_rows ? r : 0;
}

template <int LW> struct Words;
template <> struct Words<4> { typedef u32x4 type; };
template <> struct Words<2> { typedef u32x2 type; };

template <int CB, int LW, bool Z>
struct Chunk {
  typename Words<LW>::type w[CB];
  bf16x8 a[LW];
  uint16_t s[CB], z[CB];
};

template <int CB, int LW, bool Z>
__global__ __launch_bounds__(256) void k_experts_rows16(EArgs p) {
  typedef typename Words<LW>::type words_t;
  __shared__ __attribute__((aligned(16))) float part[4][CB][4][64];  // [wave][block][element][lane]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = (int)(blockIdx.x / (unsigned)p.tiles_n), tn = (int)(blockIdx.x % (unsigned)p.tiles_n);
  RowTile t;
  int count;
  if (!find_row_tile<false>(p.offsets, p.experts, p.slots, 4, m, t, count)) return;

  const int lr = lane & 15, lq = lane >> 4;
  const int64_t n0 = (int64_t)tn * (16 * CB);
  const uint16_t* arow = p.a + a_row(p, t.row0 + min(lr, t.rows - 1)) * p.k + lq * (8 * LW);
  const uint8_t* brow[CB];
  int64_t srow[CB];
#pragma unroll
  for (int j = 0; j < CB; ++j) {
    const int64_t col = min(n0 + j * 16 + lr, p.n - 1) + (int64_t)t.bin * p.n;
    brow[j] = p.b + col * (p.k / 2) + lq * (4 * LW);
    srow[j] = col * p.ngroups;
  }
  auto load = [&](int ch, Chunk<CB, LW, Z>& f) {
    const int64_t g = ch / p.group_chunks;
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      f.w[j] = *reinterpret_cast<const words_t*>(brow[j] + (int64_t)ch * (16 * LW));
      f.s[j] = p.scales[srow[j] + g];
      if (Z) f.z[j] = p.zeros[srow[j] + g];
    }
#pragma unroll
    for (int w = 0; w < LW; ++w)
      f.a[w] = *reinterpret_cast<const bf16x8*>(arow + (int64_t)ch * (32 * LW) + w * 8);
  };
  const uint32_t magic_v = vconst(0x43004300u);
  const u32x4 ones_u = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_u);
  floatx4 acc[CB];
#pragma unroll
  for (int j = 0; j < CB; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto fold = [&](const Chunk<CB, LW, Z>& f) {
    floatx4 sum[CB], rs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < CB; ++j) sum[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < LW; ++w) {
      rs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[w], ones, rs, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < CB; ++j)
        sum[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[w], unpack8(f.w[j][w], magic_v), sum[j], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const float s = bf16_to_f32(f.s[j]);
      const float zb = 128.f + (Z ? bf16_to_f32(f.z[j]) : p.zero_const);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(s, fmaf(-zb, rs[e], sum[j][e]), acc[j][e]);
    }
  };
  // this wave's chunks, two ahead of use
  const int nch = (int)(p.k / (32 * LW));
  Chunk<CB, LW, Z> f0, f1;
  if (wave < nch) load(wave, f0);
  if (wave + 4 < nch) load(wave + 4, f1);
  for (int ch = wave; ch < nch; ch += 8) {
    fold(f0);
    if (ch + 8 < nch) load(ch + 8, f0);
    if (ch + 4 < nch) {
      fold(f1);
      if (ch + 12 < nch) load(ch + 12, f1);
    }
  }

  // join the waves' sums: element e of lane l is row 4 (l / 16) + e, column l % 16
#pragma unroll
  for (int j = 0; j < CB; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][j][e][lane] = acc[j][e];
  __syncthreads();
  for (int i = threadIdx.x; i < CB * 256; i += 256) {
    const int j = i >> 8, e = (i >> 6) & 3, l = i & 63;
    const int row = 4 * (l >> 4) + e;
    const int64_t col = n0 + j * 16 + (l & 15);
    const float v = (part[0][j][e][l] + part[1][j][e][l]) + (part[2][j][e][l] + part[3][j][e][l]);
    if (row < t.rows && col < p.n)
      p.c[(int64_t)(t.row0 + row) * p.n + col] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

template <int CB, int LW>
hipError_t launch_rows16(EArgs p, hipStream_t s) {
  p.tiles_n = (int)((p.n + 16 * CB - 1) / (16 * CB));
  const unsigned grid = (unsigned)(row_tiles_bound(p.slots, p.experts, 4) * p.tiles_n);
  if (p.zeros) hipLaunchKernelGGL((k_experts_rows16<CB, LW, true>), dim3(grid), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((k_experts_rows16<CB, LW, false>), dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w4a16_experts(const uint16_t* a, int64_t a_rows, const int32_t* order, int64_t topk,
                                     const int32_t* offsets, int64_t slots, int64_t experts, const uint8_t* b,
                                     const uint16_t* scales, const uint16_t* zeros, int64_t group, float zero_const,
                                     int64_t n, int64_t k, uint16_t* c, hipStream_t s) {
  EArgs p{};
  p.a = a;
  p.order = order;
  p.offsets = offsets;
  p.b = b;
  p.scales = scales;
  p.zeros = zeros;
  p.c = c;
  p.n = n;
  p.k = k;
  p.zero_const = zero_const;
  p.topk = (int)topk;
  p.a_rows = (int)a_rows;
  p.slots = (int)slots;
  p.experts = (int)experts;
  p.ngroups = (int)(k / group);
  // 128-k chunks, or 64-k ones where a group or k is no multiple of 128
  if (group % 128 == 0) {
    p.group_chunks = (int)(group / 128);
    return launch_rows16<1, 4>(p, s);
  }
  p.group_chunks = (int)(group / 64);
  return launch_rows16<1, 2>(p, s);
}

}  // namespace wq
