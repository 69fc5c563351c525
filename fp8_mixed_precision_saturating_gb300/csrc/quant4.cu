// quant4.cu -- bf16 matrices into microscaled 4-bit operands and back (HBM-bound kernels).
//
// Formats, scale rule and layout: include/fp8gb.h, "Microscaled 4-bit operands".
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cast.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace fp8gb {
namespace {

using namespace castops;

// The tensor scale of a call: 1 without a state, else from the state's amax or history; the
// first thread of the grid records it.
__device__ __forceinline__ float tensor_scale(const QuantState& st, bool delayed, bool first) {
  if (st.scale == nullptr) return 1.0f;
  float s, d;
  scales_from_amax(effective_amax(st, delayed), fp4::kNvTensorMax, s, d);
  if (first) {
    *st.scale = s;
    *st.scale_inv = d;
  }
  return s;
}

// max |x| of a matrix onto *st.amax_cur (NaN ignored). With `bootstrap` only while the history is empty: later
// delayed casts take the scale from the history and record the amax themselves.
__global__ void __launch_bounds__(512) amax4_kernel(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, QuantState st, int bootstrap, int vec) {
  pdl_wait();
  pdl_trigger();
  if (bootstrap && *st.hist_count > 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5), w0 = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  uint32_t m = 0;
  if (vec) {  // whole 16-byte chunks, 8 of a lane's in flight; a contiguous matrix is one long row
    if (ld == cols) {
      cols *= rows;
      rows = 1;
    }
    const int64_t n = cols / 8;
    auto span = [&](const uint4* row, int64_t c) {  // 256 chunks of a row from c on
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + 32 * j < n ? __ldg(row + c + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = absmax_v(m, v[j]);
    };
    if (rows == 1)
      for (int64_t i = w0; i * 256 < n; i += warps) span(reinterpret_cast<const uint4*>(x), i * 256 + lane);
    else
      for (int64_t r = w0; r < rows; r += warps)
        for (int64_t c = 0; c < n; c += 256) span(reinterpret_cast<const uint4*>(x + r * ld), c + lane);
    m = fold2(m);
  } else {
    for (int64_t r = w0; r < rows; r += warps) {
      for (int64_t c0 = 0; c0 < cols; c0 += 256) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c0 + lane + 32 * j < cols ? x[r * ld + c0 + lane + 32 * j] & 0x7FFFu : 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = v[j] <= 0x7F80u ? max(m, v[j]) : m;
      }
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  __shared__ uint32_t part[16];
  if (lane == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = __reduce_max_sync(0xFFFFFFFFu, lane < (blockDim.x >> 5) ? part[lane] : 0u);
    if (lane == 0) atomic_max_amax(st.amax_cur, m);
  }
}

// 16 elements (8 words of two bf16) times mul -> 16 codes.
__device__ __forceinline__ uint2 cast16(const uint32_t (&w)[8], float mul) {
  unsigned long long mm;
  asm("mov.b64 %0, {%1, %1};" : "=l"(mm) : "f"(mul));
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = w[4 * h + i];
      asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%2, %3};\n\tmul.rn.f32x2 a, a, %4;\n\tmov.b64 {%0, %1}, a;\n\t}"
          : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
          : "f"(__uint_as_float(t << 16)), "f"(__uint_as_float(t & 0xFFFF0000u)), "l"(mm));
    }
    c[h] = fp4::cvt8_e2m1(v);
  }
  return make_uint2(c[0], c[1]);
}

// Both ways, or rows that are not aligned: one 128 x 128 tile of x per CTA, read once into shared memory (zero past the matrix, which gives the padding's
// codes and scales their values without a branch), then quantised along its rows (ROWS) and down its columns
// (COLS). Either way the tile is 64 bytes of each of 128 operand rows and whole scale atoms (2 for NVFP4, 1 for
// MXFP4), so codes leave in 64-byte pieces and scales in 512-byte ones. 4099 x 1536 both ways in 7.9 us, 2.6 TB/s: one wave of
// 396 tiles, bound by its latency; 512 threads per tile were no faster (76.3 -> 79.9 us for a 4096 x 14336 weight).
constexpr int kTile = 128, kPitch = 272;  // bytes per tile row: 16 more than 256, so rows start in other banks

template <int FMT, bool ROWS, bool COLS, bool VEC>
__global__ void __launch_bounds__(256) quant4_kernel(const uint16_t* x, int rows, int cols, int64_t ld, QuantState st, int delayed,
                                                     uint8_t* q, uint8_t* sf, uint8_t* qT, uint8_t* sfT, int tiles_x, int backwards) {
  constexpr int G = fp4::F4<FMT>::kGroup, ATOMS = FMT == 0 ? 2 : 1;
  __shared__ __align__(16) uint8_t tile[kTile * kPitch];
  __shared__ __align__(16) uint8_t s_sf[512 * ATOMS], s_sfT[512 * ATOMS];
  __shared__ __align__(16) uint8_t s_qT[COLS ? kTile * 64 : 16];
  __shared__ float table[8];  // (NVFP4) the tensor's scale over the eight E4M3 significands
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // behind a pass for the tensor's amax the tiles are taken from the end: what that pass read last is still in L2
  const int b = backwards ? gridDim.x - 1 - blockIdx.x : blockIdx.x, ty = b / tiles_x, tx = b - ty * tiles_x;
  const int r0 = ty * kTile, c0 = tx * kTile;
  if constexpr (VEC) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // 16 lanes take a row's 256 bytes
      const int r = r0 + 16 * i + (tid >> 4), c = c0 + 8 * (tid & 15);
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < rows && c + 8 <= cols) {
        v[i] = __ldcs(reinterpret_cast<const uint4*>(x + r * ld + c));
      } else if (r < rows && c < cols) {  // a row's last elements: what follows them is not read
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (c + j < cols) w[j >> 1] |= static_cast<uint32_t>(x[r * ld + c + j]) << (16 * (j & 1));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(tile + (16 * i + (tid >> 4)) * kPitch + 16 * (tid & 15)) = v[i];
  } else {
#pragma unroll 8
    for (int i = 0; i < 64; ++i) {  // a warp takes 32 elements of a row
      const int e = i * 256 + tid, r = e >> 7, c = e & 127;
      const uint16_t v = r0 + r < rows && c0 + c < cols ? x[(r0 + r) * ld + c0 + c] : static_cast<uint16_t>(0);
      *reinterpret_cast<uint16_t*>(tile + r * kPitch + 2 * c) = v;
    }
  }
  const float s = FMT == 0 ? tensor_scale(st, delayed != 0, blockIdx.x == 0 && tid == 0) : 1.0f;
  const uint32_t least = fp4::least_scale(s);
  if (FMT == 0 && tid < 8) table[tid] = fp4::quotient(s, tid);
  auto group = [&](uint32_t bf16_bits, float& mul) {
    return FMT == 0 ? fp4::group_scale_nv(bf16_bits << 16, s, least, table, mul) : fp4::group_scale<FMT>(bf16_bits << 16, s, least, mul);
  };
  __syncthreads();
  uint32_t am = 0;  // largest magnitude of the tile (NaN included; delayed scaling records it)
  if constexpr (ROWS) {
    // 8 lanes take a row (16 elements each), a warp 4 rows 32 apart, whose scale words are neighbours in an atom
    const int g = lane & 7, j = lane >> 3, half = (lane >> 2) & 1;
    const int64_t pitch = fp4::row_bytes(cols);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 32 * j + 8 * i + warp;
      const uint8_t* at = tile + r * kPitch + 32 * g;
      // lanes 4-7 of a row read their second half first: eight lanes' 16 bytes then fall in different banks
      uint4 a = *reinterpret_cast<const uint4*>(at + 16 * half), b = *reinterpret_cast<const uint4*>(at + 16 * (1 - half));
      const uint4 lo = half ? b : a, hi = half ? a : b;
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      if constexpr (FMT == 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      am = max(am, m);
      float mul;
      const uint32_t c = group(m, mul);
      uint2 o = cast16(w, mul);
      if (c == fp4::F4<FMT>::kScaleNaN) o = make_uint2(0u, 0u);
      const int byte = c0 / 2 + 8 * g;
      if (r0 + r < rows && byte < pitch) *reinterpret_cast<uint2*>(q + (r0 + r) * pitch + byte) = o;
      const int group = FMT == 0 ? g : g >> 1;
      if (FMT == 0 || (g & 1) == 0) s_sf[(group >> 2) * 512 + 16 * (r & 31) + 4 * (r >> 5) + (group & 3)] = static_cast<uint8_t>(c);
    }
  }
  if constexpr (COLS) {
    // NVFP4: a warp takes 16 rows, a lane 4 columns; MXFP4: 32 rows of half the columns, a lane 2
    constexpr int PER = FMT == 0 ? 4 : 2;
    const int k0 = FMT == 0 ? 16 * warp : 32 * (warp >> 1), col0 = FMT == 0 ? 4 * lane : 64 * (warp & 1) + 2 * lane;
    uint32_t v[G][PER / 2];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const uint8_t* at = tile + (k0 + i) * kPitch + 2 * col0;
      if constexpr (FMT == 0) {
        const uint2 t = *reinterpret_cast<const uint2*>(at);
        v[i][0] = t.x;
        v[i][PER / 2 - 1] = t.y;
      } else {
        v[i][0] = *reinterpret_cast<const uint32_t*>(at);
      }
    }
#pragma unroll
    for (int h = 0; h < PER / 2; ++h) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < G; ++i) m = __vmaxu2(m, v[i][h] & 0x7FFF7FFFu);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t a = e ? m >> 16 : m & 0xFFFFu;
        am = max(am, a);
        float mul;
        const uint32_t c = group(a, mul);
        const int col = col0 + 2 * h + e, group = FMT == 0 ? warp : warp >> 1;
        s_sfT[(group >> 2) * 512 + 16 * (col & 31) + 4 * (col >> 5) + (group & 3)] = static_cast<uint8_t>(c);
#pragma unroll
        for (int t = 0; t < G / 16; ++t) {
          uint32_t w[8];  // the column's elements two by two
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k] = e ? __byte_perm(v[16 * t + 2 * k][h], v[16 * t + 2 * k + 1][h], 0x7632) : __byte_perm(v[16 * t + 2 * k][h], v[16 * t + 2 * k + 1][h], 0x5410);
          uint2 o = cast16(w, mul);
          if (c == fp4::F4<FMT>::kScaleNaN) o = make_uint2(0u, 0u);
          // 8-byte piece k0 / 16 + t of the column's 64 bytes, moved by its column so that lanes use other banks
          *reinterpret_cast<uint2*>(s_qT + 64 * col + 8 * (((k0 >> 4) + t) ^ ((col >> 2) & 7))) = o;
        }
      }
    }
  }
  if (FMT == 0 && delayed && st.scale != nullptr && *st.hist_count > 0) {
    __shared__ uint32_t s_am;
    if (tid == 0) s_am = 0;
    if (__syncthreads_or(am > 0x7F80u)) {  // a tile with a NaN is looked at again, without it
      am = 0;
      for (int e = tid; e < kTile * kTile; e += 256) {
        const uint32_t b = *reinterpret_cast<const uint16_t*>(tile + (e >> 7) * kPitch + 2 * (e & 127)) & 0x7FFFu;
        am = b <= 0x7F80u ? max(am, b) : am;
      }
    }
    am = __reduce_max_sync(0xFFFFFFFFu, am);
    if (lane == 0) atomicMax(&s_am, am);
    __syncthreads();
    if (tid == 0) atomic_max_amax(st.amax_cur, s_am);
  }
  __syncthreads();
  // whole atoms: the one of 128 rows (columns) and 4 groups that this tile fills, 16 bytes per thread
  if constexpr (ROWS) {
    const int64_t atoms = fp4::atoms_along(FMT, cols);
    if (tid < 32 * ATOMS && tx * ATOMS + (tid >> 5) < atoms)
      reinterpret_cast<uint4*>(sf + (ty * atoms + tx * ATOMS) * 512)[tid] = reinterpret_cast<const uint4*>(s_sf)[tid];
  }
  if constexpr (COLS) {
    const int64_t atoms = fp4::atoms_along(FMT, rows), pitch = fp4::row_bytes(rows);
    const int t = tid - 64;
    if (t >= 0 && t < 32 * ATOMS && ty * ATOMS + (t >> 5) < atoms)
      reinterpret_cast<uint4*>(sfT + (tx * atoms + ty * ATOMS) * 512)[t] = reinterpret_cast<const uint4*>(s_sfT)[t];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 64 * i + (tid >> 2), piece = tid & 3, sw = (col >> 2) & 7, byte = r0 / 2 + 16 * piece;
      const uint2 a = *reinterpret_cast<const uint2*>(s_qT + 64 * col + 8 * ((2 * piece) ^ sw));
      const uint2 b = *reinterpret_cast<const uint2*>(s_qT + 64 * col + 8 * ((2 * piece + 1) ^ sw));
      if (c0 + col < cols && byte < pitch) *reinterpret_cast<uint4*>(qT + (c0 + col) * pitch + byte) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// Along the rows alone, from 16-byte aligned rows: no tile and no barrier. A lane takes 16 neighbouring elements of 4
// rows 32 apart (their scale words are neighbours in an atom), a warp 512 columns; all loads are in flight at once.
// 16384 x 4096: 30.1 us, 5.7 TB/s (through the tile 33.0); issue slots 64 % used, so the instructions per element (largest
// of the group, scale, multiply, conversion) count beside the memory.
template <int FMT>
__global__ void __launch_bounds__(256) quant4_rows_kernel(const uint16_t* x, int rows, int cols, int64_t ld, QuantState st, int delayed, uint8_t* q,
                                                          uint8_t* sf, int pieces, int backwards) {
  __shared__ float table[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const float s = FMT == 0 ? tensor_scale(st, delayed != 0, blockIdx.x == 0 && tid == 0) : 1.0f;
  const uint32_t least = fp4::least_scale(s);
  const int b = backwards ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  const int64_t item = b * 8ll + (tid >> 5), line = item / pieces;  // (128-row block, row in 32), piece of 512 columns
  const int c0 = static_cast<int>(item - line * pieces) * 512 + 16 * lane;
  const int64_t m0 = (line >> 5) * 128 + (line & 31);
  uint4 v[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[j][h] = make_uint4(0, 0, 0, 0);
      const int c = c0 + 8 * h;
      if (m0 + 32 * j < rows) {
        const uint16_t* row = x + (m0 + 32 * j) * ld;
        if (c + 8 <= cols) {
          v[j][h] = __ldcs(reinterpret_cast<const uint4*>(row + c));
        } else if (c < cols) {  // a row's last elements: what follows them is not read
          uint32_t* w = reinterpret_cast<uint32_t*>(&v[j][h]);
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (c + i < cols) w[i >> 1] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
        }
      }
    }
  if constexpr (FMT == 0) {
    if (tid < 8) table[tid] = fp4::quotient(s, tid);
    __syncthreads();
  }
  const int64_t pitch = fp4::row_bytes(cols), atoms = fp4::atoms_along(FMT, cols);
  uint32_t am = 0, scales = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w[8] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w, v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    if constexpr (FMT == 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    am = max(am, m);
    float mul;
    const uint32_t c = FMT == 0 ? fp4::group_scale_nv(m << 16, s, least, table, mul) : fp4::group_scale<FMT>(m << 16, s, least, mul);
    uint2 o = cast16(w, mul);
    if (c == fp4::F4<FMT>::kScaleNaN) o = make_uint2(0u, 0u);
    if (m0 + 32 * j < rows && c0 / 2 < pitch) *reinterpret_cast<uint2*>(q + (m0 + 32 * j) * pitch + c0 / 2) = o;
    scales |= c << (8 * j);
  }
  // four groups' lanes hold a byte of each of the four rows; afterwards each of them holds a row's word of four groups
  constexpr int STEP = FMT == 0 ? 1 : 2;  // lanes per group
  const int at = (lane / STEP) & 3;
  const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, scales, STEP);
  uint32_t t = at & 1 ? __byte_perm(o1, scales, 0x7351) : __byte_perm(scales, o1, 0x6240);  // rows {1, 3} or {0, 2} of two groups
  const uint32_t o2 = __shfl_xor_sync(0xFFFFFFFFu, t, 2 * STEP);
  t = at & 2 ? __byte_perm(o2, t, 0x7632) : __byte_perm(t, o2, 0x5410);
  const int64_t atom = (c0 / fp4::F4<FMT>::kGroup) >> 2;
  if (m0 < (rows + 127ll) / 128 * 128 && atom < atoms && lane % STEP == 0)
    *reinterpret_cast<uint32_t*>(sf + ((m0 >> 7) * atoms + atom) * 512 + 16 * (m0 & 31) + 4 * at) = t;
  if (FMT == 0 && delayed && st.scale != nullptr && *st.hist_count > 0) {
    __shared__ uint32_t s_am;
    if (tid == 0) s_am = 0;
    if (__syncthreads_or(am > 0x7F80u)) {  // a CTA with a NaN looks at its elements again, without it
      am = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w[4] = {v[j][h].x, v[j][h].y, v[j][h].z, v[j][h].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
            if (lo <= 0x7F80u) am = max(am, lo);
            if (hi <= 0x7F80u) am = max(am, hi);
          }
        }
    }
    am = __reduce_max_sync(0xFFFFFFFFu, am);
    if (lane == 0) atomicMax(&s_am, am);
    __syncthreads();
    if (tid == 0) atomic_max_amax(st.amax_cur, s_am);
  }
}

// Down the columns alone, from 16-byte aligned rows: 128 rows by 128 columns per CTA, read straight into registers (a
// warp takes 16 rows, a lane 4 columns; MXFP4: 32 rows of half the columns, a lane 2); only codes and scales pass
// through shared memory, to leave in 64- and 512-byte pieces. 4096 x 14336: 28.1 us, 5.4 TB/s (when it was 30.2: through
// the tile 31.9, 256 rows per CTA 32.9).
template <int FMT>
__global__ void __launch_bounds__(256) quant4_cols_kernel(const uint16_t* x, int rows, int cols, int64_t ld, QuantState st, int delayed, uint8_t* qT,
                                                          uint8_t* sfT, int tiles_x, int backwards) {
  constexpr int G = fp4::F4<FMT>::kGroup, ATOMS = FMT == 0 ? 2 : 1, PAIRS = FMT == 0 ? 2 : 1;  // pairs of columns per lane
  __shared__ __align__(16) uint8_t s_sfT[512 * ATOMS];
  __shared__ __align__(16) uint8_t s_qT[kTile * 64];
  __shared__ float table[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = backwards ? gridDim.x - 1 - blockIdx.x : blockIdx.x, ty = b / tiles_x, tx = b - ty * tiles_x;
  const int r0 = ty * kTile, c0 = tx * kTile;
  const int k0 = FMT == 0 ? 16 * warp : 32 * (warp >> 1), col0 = FMT == 0 ? 4 * lane : 64 * (warp & 1) + 2 * lane;
  uint32_t v[G][PAIRS];
  {
    const uint16_t* at = x + (r0 + k0) * ld + c0 + col0;
    const bool whole = c0 + col0 + 2 * PAIRS <= cols;
#pragma unroll
    for (int i = 0; i < G; ++i, at += ld) {
      const bool in = r0 + k0 + i < rows;
#pragma unroll
      for (int h = 0; h < PAIRS; ++h) v[i][h] = 0;
      if (in && whole) {
        if constexpr (FMT == 0) {
          const uint2 t = __ldcs(reinterpret_cast<const uint2*>(at));
          v[i][0] = t.x;
          v[i][PAIRS - 1] = t.y;
        } else {
          v[i][0] = __ldcs(reinterpret_cast<const uint32_t*>(at));
        }
      } else if (in) {  // the last columns
#pragma unroll
        for (int e = 0; e < 2 * PAIRS; ++e)
          if (c0 + col0 + e < cols) v[i][e >> 1] |= static_cast<uint32_t>(at[e]) << (16 * (e & 1));
      }
    }
  }
  const float s = FMT == 0 ? tensor_scale(st, delayed != 0, blockIdx.x == 0 && tid == 0) : 1.0f;
  const uint32_t least = fp4::least_scale(s);
  if constexpr (FMT == 0) {
    if (tid < 8) table[tid] = fp4::quotient(s, tid);
    __syncthreads();
  }
  uint32_t am = 0;
#pragma unroll
  for (int h = 0; h < PAIRS; ++h) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) m = __vmaxu2(m, v[i][h] & 0x7FFF7FFFu);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t a = e ? m >> 16 : m & 0xFFFFu;
      am = max(am, a);
      float mul;
      const uint32_t c = FMT == 0 ? fp4::group_scale_nv(a << 16, s, least, table, mul) : fp4::group_scale<FMT>(a << 16, s, least, mul);
      const int col = col0 + 2 * h + e, grp = k0 / G;
      s_sfT[(grp >> 2) * 512 + 16 * (col & 31) + 4 * (col >> 5) + (grp & 3)] = static_cast<uint8_t>(c);
#pragma unroll
      for (int t = 0; t < G / 16; ++t) {
        uint32_t w[8];  // the column's elements two by two
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __byte_perm(v[16 * t + 2 * k][h], v[16 * t + 2 * k + 1][h], e ? 0x7632 : 0x5410);
        uint2 o = cast16(w, mul);
        if (c == fp4::F4<FMT>::kScaleNaN) o = make_uint2(0u, 0u);
        // 8-byte piece k0 / 16 + t of the column's 64 bytes, moved by its column so that lanes use other banks
        *reinterpret_cast<uint2*>(s_qT + 64 * col + 8 * (((k0 >> 4) + t) ^ ((col >> 2) & 7))) = o;
      }
    }
  }
  if (FMT == 0 && delayed && st.scale != nullptr && *st.hist_count > 0) {
    __shared__ uint32_t s_am;
    if (tid == 0) s_am = 0;
    if (__syncthreads_or(am > 0x7F80u)) {  // a CTA with a NaN looks at its elements again, without it
      am = 0;
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int h = 0; h < PAIRS; ++h) {
          const uint32_t lo = v[i][h] & 0x7FFFu, hi = (v[i][h] >> 16) & 0x7FFFu;
          if (lo <= 0x7F80u) am = max(am, lo);
          if (hi <= 0x7F80u) am = max(am, hi);
        }
    }
    am = __reduce_max_sync(0xFFFFFFFFu, am);
    if (lane == 0) atomicMax(&s_am, am);
    __syncthreads();
    if (tid == 0) atomic_max_amax(st.amax_cur, s_am);
  }
  __syncthreads();
  const int64_t atoms = fp4::atoms_along(FMT, rows), pitch = fp4::row_bytes(rows);
  if (tid < 32 * ATOMS && ty * ATOMS + (tid >> 5) < atoms)
    reinterpret_cast<uint4*>(sfT + (tx * atoms + ty * ATOMS) * 512)[tid] = reinterpret_cast<const uint4*>(s_sfT)[tid];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = 64 * i + (tid >> 2), piece = tid & 3, sw = (col >> 2) & 7, byte = r0 / 2 + 16 * piece;
    const uint2 lo = *reinterpret_cast<const uint2*>(s_qT + 64 * col + 8 * ((2 * piece) ^ sw));
    const uint2 hi = *reinterpret_cast<const uint2*>(s_qT + 64 * col + 8 * ((2 * piece + 1) ^ sw));
    if (c0 + col < cols && byte < pitch) *reinterpret_cast<uint4*>(qT + (c0 + col) * pitch + byte) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

// A warp takes 256 elements of 4 rows 32 apart (their scale words are 16 bytes of an atom), a lane 8 of each. 16384 x 4096
// to bf16: 26.2 us, 6.6 TB/s, the memory's rate; 1536 x 4099 (rows that are not aligned) 5.7 us.
template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(256) dequant4_kernel(const uint8_t* q, const uint8_t* sf, int64_t mn, int64_t k, const float* scale_inv, T* y,
                                                       int64_t ldy, int pieces) {
  constexpr int G = fp4::F4<FMT>::kGroup;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t atoms = fp4::atoms_along(FMT, k), pitch = fp4::row_bytes(k);
  const int64_t item = blockIdx.x * 8ll + (threadIdx.x >> 5);  // (128-row block, row in 32, piece of 256 elements)
  const int64_t line = item / pieces, k0 = (item - line * pieces) * 256 + 8 * lane;
  const int64_t m0 = (line >> 5) * 128 + (line & 31);
  if (m0 >= mn) return;
  const float d = scale_inv != nullptr ? *scale_inv : 1.0f;
  const bool live = k0 < k;
  uint32_t code[4] = {0, 0, 0, 0};
  uint4 sw = make_uint4(0, 0, 0, 0);
  const int64_t g = k0 / G;
  if (live) {
    sw = __ldg(reinterpret_cast<const uint4*>(sf + ((m0 >> 7) * atoms + (g >> 2)) * 512 + 16 * (m0 & 31)));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (m0 + 32 * j < mn) code[j] = __ldcs(reinterpret_cast<const uint32_t*>(q + (m0 + 32 * j) * pitch + k0 / 2));
  }
  const uint32_t words[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t m = m0 + 32 * j;
    if (m >= mn) break;
    const uint32_t b = (words[j] >> (8 * (g & 3))) & 0xFFu;
    const float c = FMT == 0 ? fp4::e4m3_value(b) : fp4::ue8m0_value(b);
    float v[8];
    fp4::e2m1_values(code[j], v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // code * c is exact in fp32 (5 significant bits), so the tensor's scale brings the only rounding but the output's
      asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
          : "+f"(v[i]), "+f"(v[i + 1])
          : "f"(c));
      if (scale_inv != nullptr)
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "+f"(v[i]), "+f"(v[i + 1])
            : "f"(d));
    }
    if constexpr (VEC) {
      T* at = y + m * ldy + k0;
      if (k0 + 8 <= k) {
        if constexpr (sizeof(T) == 2) {
          uint4 o;
          uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
          for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
          __stcs(reinterpret_cast<uint4*>(at), o);
        } else {
          __stcs(reinterpret_cast<float4*>(at), make_float4(v[0], v[1], v[2], v[3]));
          __stcs(reinterpret_cast<float4*>(at) + 1, make_float4(v[4], v[5], v[6], v[7]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (k0 + i >= k) break;
          if constexpr (sizeof(T) == 2)
            at[i] = __float2bfloat16_rn(v[i]);
          else
            at[i] = v[i];
        }
      }
    } else {
      // rows that start anywhere: neighbouring lanes store neighbouring elements, through shared memory
      __shared__ float line_buf[8][256 + 8];
      float* buf = line_buf[threadIdx.x >> 5];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) buf[8 * lane + i + (lane >> 2)] = v[i];
      __syncwarp();
      const int64_t first = k0 - 8 * lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = 32 * i + lane;
        if (first + e >= k) break;
        const float f = buf[e + (e >> 5)];
        if constexpr (sizeof(T) == 2)
          y[m * ldy + first + e] = __float2bfloat16_rn(f);
        else
          y[m * ldy + first + e] = f;
      }
      __syncwarp();
    }
  }
}

template <int FMT, bool ROWS, bool COLS>
cudaError_t launch_tiles(const void* x, int64_t rows, int64_t cols, int64_t ld, const QuantState& st, bool delayed, bool vec, void* q, void* sf,
                         void* qT, void* sfT, cudaStream_t stream) {
  const int64_t tx = (cols + kTile - 1) / kTile, ty = (rows + kTile - 1) / kTile;
  if (tx * ty > INT32_MAX) return cudaErrorInvalidConfiguration;  // (more than the memory holds)
  auto* xb = static_cast<const uint16_t*>(x);
  auto b = [](void* p) { return static_cast<uint8_t*>(p); };
  const dim3 grid(static_cast<unsigned>(tx * ty));
  if constexpr (ROWS && COLS) {
    if (vec)
      return launch_pdl(quant4_kernel<FMT, ROWS, COLS, true>, grid, dim3(256), 0, stream, xb, static_cast<int>(rows), static_cast<int>(cols), ld, st,
                        delayed ? 1 : 0, b(q), b(sf), b(qT), b(sfT), static_cast<int>(tx), st.scale != nullptr && !delayed ? 1 : 0);
  }
  return launch_pdl(quant4_kernel<FMT, ROWS, COLS, false>, grid, dim3(256), 0, stream, xb, static_cast<int>(rows), static_cast<int>(cols), ld, st,
                    delayed ? 1 : 0, b(q), b(sf), b(qT), b(sfT), static_cast<int>(tx), st.scale != nullptr && !delayed ? 1 : 0);
}

template <int FMT>
cudaError_t launch_ways(const void* x, int64_t rows, int64_t cols, int64_t ld, const QuantState& st, bool delayed, bool vec, void* q, void* sf,
                        void* qT, void* sfT, cudaStream_t stream) {
  if (q != nullptr && qT != nullptr) return launch_tiles<FMT, true, true>(x, rows, cols, ld, st, delayed, vec, q, sf, qT, sfT, stream);
  if (q != nullptr && vec) {
    const int64_t pieces = (cols + 511) / 512, grid = ((rows + 127) / 128 * 32 * pieces + 7) / 8;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;  // (more than the memory holds)
    return launch_pdl(quant4_rows_kernel<FMT>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, static_cast<const uint16_t*>(x),
                      static_cast<int>(rows), static_cast<int>(cols), ld, st, delayed ? 1 : 0, static_cast<uint8_t*>(q), static_cast<uint8_t*>(sf),
                      static_cast<int>(pieces), st.scale != nullptr && !delayed ? 1 : 0);
  }
  if (q != nullptr) return launch_tiles<FMT, true, false>(x, rows, cols, ld, st, delayed, false, q, sf, qT, sfT, stream);
  if (vec) {
    const int64_t tx = (cols + kTile - 1) / kTile, grid = tx * ((rows + kTile - 1) / kTile);
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;  // (more than the memory holds)
    return launch_pdl(quant4_cols_kernel<FMT>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, static_cast<const uint16_t*>(x),
                      static_cast<int>(rows), static_cast<int>(cols), ld, st, delayed ? 1 : 0, static_cast<uint8_t*>(qT), static_cast<uint8_t*>(sfT),
                      static_cast<int>(tx), st.scale != nullptr && !delayed ? 1 : 0);
  }
  return launch_tiles<FMT, false, true>(x, rows, cols, ld, st, delayed, false, q, sf, qT, sfT, stream);
}

template <int FMT, typename T>
cudaError_t launch_values(const void* q, const void* sf, int64_t mn, int64_t k, const float* scale_inv, void* y, int64_t ldy, cudaStream_t stream) {
  const int64_t pieces = (k + 255) / 256, items = (mn + 127) / 128 * 32 * pieces, grid = (items + 7) / 8;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;  // (more than the memory holds)
  const bool vec = (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && (ldy * static_cast<int64_t>(sizeof(T))) % 16 == 0;
  auto* qb = static_cast<const uint8_t*>(q);
  auto* sb = static_cast<const uint8_t*>(sf);
  if (vec)
    return launch_pdl(dequant4_kernel<FMT, T, true>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, qb, sb, mn, k, scale_inv,
                      static_cast<T*>(y), ldy, static_cast<int>(pieces));
  return launch_pdl(dequant4_kernel<FMT, T, false>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, qb, sb, mn, k, scale_inv,
                    static_cast<T*>(y), ldy, static_cast<int>(pieces));
}

}  // namespace

cudaError_t launch_quant4(int fmt, bool delayed, const void* x, int64_t rows, int64_t cols, int64_t ld,
                          const QuantState& st, void* q, void* sf, void* qT, void* sfT, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ld % 8 == 0;
  if (st.scale != nullptr) {
    cudaError_t e = cudaSuccess;
    if (!delayed && (e = cudaMemsetAsync(st.amax_cur, 0, sizeof(float), stream)) != cudaSuccess) return e;
    const int64_t want = (rows * cols + 16383) / 16384, most = 4ll * num_sms();
    const bool whole = vec && cols % 8 == 0;
    e = launch_pdl(amax4_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(512), 0, stream,
                   static_cast<const uint16_t*>(x), rows, cols, ld, st, delayed ? 1 : 0, whole ? 1 : 0);
    if (e != cudaSuccess) return e;
  }
  return fmt == 0 ? launch_ways<0>(x, rows, cols, ld, st, delayed, vec, q, sf, qT, sfT, stream)
                  : launch_ways<1>(x, rows, cols, ld, st, delayed, vec, q, sf, qT, sfT, stream);
}

cudaError_t launch_dequant4(int fmt, bool f32, const void* q, const void* sf, int64_t mn, int64_t k,
                            const float* scale_inv, void* y, int64_t ldy, cudaStream_t stream) {
  if (f32)
    return fmt == 0 ? launch_values<0, float>(q, sf, mn, k, scale_inv, y, ldy, stream) : launch_values<1, float>(q, sf, mn, k, scale_inv, y, ldy, stream);
  return fmt == 0 ? launch_values<0, __nv_bfloat16>(q, sf, mn, k, scale_inv, y, ldy, stream)
                  : launch_values<1, __nv_bfloat16>(q, sf, mn, k, scale_inv, y, ldy, stream);
}

}  // namespace fp8gb
