// Low-rank adapters of many requests beside a shared projection (gfx950).
//
//   out[t] = base[t] + scale[l] * B[l] (A[l] x[t]),  l = the adapter of row t
//
// Rows are sorted by adapter (wq_sort_rows with one slot a row); the rows without
// one lie behind the last adapter and only copy base.  Two launches: the first
// makes v = A x in float32 (split over k when there are few row tiles, each
// part on its own in the workspace), the second joins the parts, multiplies by
// B and adds base.  Both are bound by bytes: A and B of the adapters in use, x,
// base and out.
#include "route_tiles.h"

namespace wq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct LArgs {
  const uint16_t* x;       // [t][k] bf16
  const int* order;        // [t]: row of each sorted row
  const int* offsets;      // [adapters + 1]
  const uint16_t* a;       // [adapters][rank][k] bf16
  const uint16_t* b;       // [adapters][n][rank] bf16
  const float* scales;     // [adapters]
  const void* base;        // nullable, [t][n]
  void* out;               // [t][n]
  float* v;                // [parts][t][rank_pad]
  int64_t n, k;
  int t, adapters, rank, rank_pad;  // rank_pad: rank rounded up to 16
  int parts;               // k parts of the first launch
  int rank_groups;         // first launch: workgroups along the rank
  int col_blocks;          // second launch: 32-column blocks per wave
  int tiles_n;             // second launch: workgroups along n
};

__device__ __forceinline__ int64_t x_row(const LArgs& p, int i) {
  const int r = p.order[i];
  return (unsigned)r < (unsigned)p.t ? r : -1;  // a row that does not exist is not touched
}

// ------------------------------------------------------------ v = A x
//
// A workgroup takes MB blocks of 16 rows, NR blocks of 16 ranks and one part of
// k; its four waves take every fourth 32-k chunk and join in LDS.  Operands
// go from memory to v_mfma_f32_16x16x32_bf16 as they lie: 16 bytes of a row
// are a lane's 8 slots.  Rows and ranks past the last repeat it.
template <int MB, int NR>
__global__ __launch_bounds__(256) void k_lora_shrink(LArgs p) {
  __shared__ __attribute__((aligned(16))) float part[4][MB * NR * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  unsigned id = blockIdx.x;
  const int rg = (int)(id % (unsigned)p.rank_groups);
  id /= (unsigned)p.rank_groups;
  const int part_k = (int)(id % (unsigned)p.parts), m = (int)(id / (unsigned)p.parts);
  RowTile t;
  int count;
  constexpr int SHIFT = MB == 1 ? 4 : 6;
  static_assert(MB == 1 || MB == 4, "tiles of 16 or 64 rows");
  if (!find_row_tile<false>(p.offsets, p.adapters, p.t, SHIFT, m, t, count)) return;

  const int lr = lane & 15, lq = lane >> 4;
  const uint16_t* xr[MB];
  const uint16_t* ar[NR];
#pragma unroll
  for (int i = 0; i < MB; ++i)
    xr[i] = p.x + max(x_row(p, t.row0 + min(i * 16 + lr, t.rows - 1)), (int64_t)0) * p.k + lq * 8;
#pragma unroll
  for (int j = 0; j < NR; ++j)
    ar[j] = p.a + ((int64_t)t.bin * p.rank + min(rg * (NR * 16) + j * 16 + lr, p.rank - 1)) * p.k + lq * 8;
  floatx4 acc[MB][NR];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NR; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int nch = (int)(p.k / 32);
  const int c0 = (int)((int64_t)nch * part_k / p.parts), c1 = (int)((int64_t)nch * (part_k + 1) / p.parts);
#pragma unroll 4
  for (int ch = c0 + wave; ch < c1; ch += 4) {
    bf16x8 xf[MB], af[NR];
#pragma unroll
    for (int i = 0; i < MB; ++i) xf[i] = *reinterpret_cast<const bf16x8*>(xr[i] + (int64_t)ch * 32);
#pragma unroll
    for (int j = 0; j < NR; ++j) af[j] = *reinterpret_cast<const bf16x8*>(ar[j] + (int64_t)ch * 32);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], af[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][(i * NR + j) * 4 + e][lane] = acc[i][j][e];
  __syncthreads();
  float* v = p.v + (int64_t)part_k * p.t * p.rank_pad;
  for (int q = threadIdx.x; q < MB * NR * 256; q += 256) {
    const int l = q & 63, e = (q >> 6) & 3, j = (q >> 8) % NR, i = (q >> 8) / NR;
    const int s = (i * NR + j) * 4 + e;
    const int row = i * 16 + 4 * (l >> 4) + e, r = rg * (NR * 16) + j * 16 + (l & 15);
    if (row < t.rows && r < p.rank_pad)
      v[(int64_t)(t.row0 + row) * p.rank_pad + r] =
          (part[0][s][l] + part[1][s][l]) + (part[2][s][l] + part[3][s][l]);
  }
}

// --------------------------------------------------- out = base + scale B v
//
// B's rows are the first MFMA operand, v's rows the second, so a lane's results
// are neighbouring columns of one row: blocks 0 and 1 of 32 columns take
// columns 8 (i / 4) + i % 4 and 4 more, and a lane then holds 8 in a row --
// one 16-byte access of base and out.  The MFMA takes bf16, so v enters as a
// sum of bf16 parts: two (17 bits) where out is bf16, three (all of float32's
// 24) where it is float32; they fill MFMA slots that a small rank leaves
// empty.  RS is the number of 32-slot steps a part takes; 0: rank <= 16, two
// parts share a step.
template <typename T> constexpr int v_parts() { return sizeof(T) == 2 ? 2 : 3; }

// eight elements in a row at the element's own alignment (16-byte accesses
// need no more on gfx950)
template <typename T> struct Eight;
template <> struct Eight<__bf16> { struct alignas(2) raw { uint16_t h[8]; }; };
template <> struct Eight<float> { struct alignas(4) raw { float f[8]; }; };

template <typename T, int MB, int RS>
__global__ __launch_bounds__(256) void k_lora_expand(LArgs p) {
  constexpr int NS = v_parts<T>();
  constexpr int RP = RS == 0 ? 16 : RS * 32;       // slots of a part
  constexpr int STEPS = (NS * RP + 31) / 32;
  constexpr int PITCH = STEPS * 32 + 8;            // bf16 per LDS row; 16 bytes off a power of two
  __shared__ __attribute__((aligned(16))) uint16_t vs[MB * 16 * PITCH];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = (int)(blockIdx.x / (unsigned)p.tiles_n), tn = (int)(blockIdx.x % (unsigned)p.tiles_n);
  RowTile t;
  int count;
  constexpr int SHIFT = MB == 1 ? 4 : 6;
  if (!find_row_tile<true>(p.offsets, p.adapters, p.t, SHIFT, m, t, count)) return;
  const bool live = t.bin < p.adapters;
  if (!live && p.out == p.base) return;  // nothing to copy

  if (live) {
    const float scale = p.scales[t.bin];
    for (int q = tid; q < t.rows * (STEPS * 32); q += 256) vs[(q / (STEPS * 32)) * PITCH + q % (STEPS * 32)] = 0;
    __syncthreads();
    for (int q = tid; q < t.rows * p.rank; q += 256) {
      const int row = q / p.rank, r = q % p.rank;
      const float* src = p.v + (int64_t)(t.row0 + row) * p.rank_pad + r;
      float sum = 0.f;
      for (int u = 0; u < p.parts; ++u) sum += src[(int64_t)u * p.t * p.rank_pad];
      float left = sum * scale;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const __bf16 h = (__bf16)left;
        vs[row * PITCH + s * RP + r] = __builtin_bit_cast(uint16_t, h);
        left -= (float)h;
      }
    }
    __syncthreads();
  }
  const int lr = lane & 15, lq = lane >> 4;
  int64_t orow[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) orow[i] = i * 16 + lr < t.rows ? x_row(p, t.row0 + i * 16 + lr) : -1;
  const uint16_t* bl = p.b + (int64_t)(live ? t.bin : 0) * p.n * p.rank;
  for (int cb = 0; cb < p.col_blocks; ++cb) {
    const int64_t n0 = ((int64_t)tn * p.col_blocks + cb) * 128 + wave * 32;
    if (n0 >= p.n) break;
    floatx4 acc[MB][2];
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[i][0] = acc[i][1] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (live) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int slot = s * 32 + lq * 8;
        const int r = min(slot % RP, p.rank - 8);  // slots past the rank meet a zero of v
        bf16x8 bf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t col = min(n0 + (lr >> 2) * 8 + h * 4 + (lr & 3), p.n - 1);
          bf[h] = *reinterpret_cast<const bf16x8*>(bl + col * p.rank + r);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const bf16x8 vf = *reinterpret_cast<const bf16x8*>(vs + (i * 16 + lr) * PITCH + slot);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[h], vf, acc[i][h], 0, 0, 0);
        }
      }
    }
    const int64_t c0 = n0 + lq * 8;
    if (c0 >= p.n) continue;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if (orow[i] < 0) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = acc[i][e >> 2][e & 3];
      const T* src = (const T*)p.base + orow[i] * p.n + c0;
      T* dst = (T*)p.out + orow[i] * p.n + c0;
      typedef typename Eight<T>::raw raw_t;
      if (c0 + 8 <= p.n) {
        T w[8];
        if (p.base) __builtin_memcpy(w, reinterpret_cast<const raw_t*>(src), sizeof(w));
        if (live || !p.base) {  // a row without an adapter keeps base's bits
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = (T)(p.base ? f[e] + (float)w[e] : f[e]);
        }
        __builtin_memcpy(reinterpret_cast<raw_t*>(dst), w, sizeof(w));
      } else {
        for (int e = 0; e < 8; ++e)
          if (c0 + e < p.n) dst[e] = !p.base ? (T)f[e] : live ? (T)(f[e] + (float)src[e]) : src[e];
      }
    }
  }
}

// Rows of a tile: 16 with up to 1024 rows, where most tiles hold a request's
// one or few rows; 64 above.
int lora_shift(int64_t t) { return t > 1024 ? 6 : 4; }

// k parts: enough workgroups to fill the card (512) where row tiles alone do
// not, each part at least 256 k, so that every wave has two chunks or more.
int lora_parts(int64_t t, int64_t adapters, int64_t rank, int64_t k) {
  const int64_t wgs = row_tiles_bound(t, adapters, lora_shift(t)) * ((rank + 63) / 64);
  int64_t parts = wgs > 0 ? (511 + wgs) / wgs : 1;
  if (parts > k / 256) parts = k / 256;
  if (parts > 16) parts = 16;
  return parts > 1 ? (int)parts : 1;
}

int pad16(int64_t rank) { return (int)((rank + 15) / 16 * 16); }

template <int MB>
hipError_t shrink(LArgs p, hipStream_t s) {
  const int nr = p.rank <= 16 ? 1 : p.rank <= 32 ? 2 : 4;
  p.rank_groups = (p.rank + nr * 16 - 1) / (nr * 16);
  const unsigned grid =
      (unsigned)(row_tiles_bound(p.t, p.adapters, MB == 1 ? 4 : 6) * p.parts * p.rank_groups);
  if (nr == 1) hipLaunchKernelGGL((k_lora_shrink<MB, 1>), dim3(grid), dim3(256), 0, s, p);
  else if (nr == 2) hipLaunchKernelGGL((k_lora_shrink<MB, 2>), dim3(grid), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((k_lora_shrink<MB, 4>), dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, int MB>
hipError_t expand(LArgs p, hipStream_t s) {
  const int64_t tiles = row_tiles_bound(p.t, p.adapters + 1, MB == 1 ? 4 : 6);
  const int64_t blocks = (p.n + 127) / 128;
  p.col_blocks = 1;
  while (p.col_blocks < 8 && tiles * (blocks / (2 * p.col_blocks)) >= 1024) p.col_blocks *= 2;
  p.tiles_n = (int)((blocks + p.col_blocks - 1) / p.col_blocks);
  const dim3 grid((unsigned)(tiles * p.tiles_n)), wg(256);
  if (p.rank <= 16) hipLaunchKernelGGL((k_lora_expand<T, MB, 0>), grid, wg, 0, s, p);
  else if (p.rank <= 32) hipLaunchKernelGGL((k_lora_expand<T, MB, 1>), grid, wg, 0, s, p);
  else if (p.rank <= 64) hipLaunchKernelGGL((k_lora_expand<T, MB, 2>), grid, wg, 0, s, p);
  else hipLaunchKernelGGL((k_lora_expand<T, MB, 4>), grid, wg, 0, s, p);
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace(int64_t t, int64_t adapters, int64_t rank, int64_t k) {
  return (size_t)lora_parts(t, adapters, rank, k) * (size_t)t * (size_t)pad16(rank) * sizeof(float);
}

hipError_t launch_lora(const uint16_t* x, int64_t t, int64_t k, const int32_t* order, const int32_t* offsets,
                       int64_t adapters, const uint16_t* a, const uint16_t* b, int64_t rank, const float* scales,
                       const void* base, void* out, bool out_bf16, int64_t n, void* ws, hipStream_t s) {
  LArgs p{};
  p.x = x;
  p.order = order;
  p.offsets = offsets;
  p.a = a;
  p.b = b;
  p.scales = scales;
  p.base = base;
  p.out = out;
  p.v = (float*)ws;
  p.n = n;
  p.k = k;
  p.t = (int)t;
  p.adapters = (int)adapters;
  p.rank = (int)rank;
  p.rank_pad = pad16(rank);
  p.parts = lora_parts(t, adapters, rank, k);
  const bool wide = lora_shift(t) == 6;
  const hipError_t e = wide ? shrink<4>(p, s) : shrink<1>(p, s);
  if (e != hipSuccess) return e;
  if (out_bf16) return wide ? expand<__bf16, 4>(p, s) : expand<__bf16, 1>(p, s);
  return wide ? expand<float, 4>(p, s) : expand<float, 1>(p, s);
}

}  // namespace wq
