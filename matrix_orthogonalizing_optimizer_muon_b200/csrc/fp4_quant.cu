// Quantisation to 4-bit matrices and back (format: fp4.cuh), of one matrix or
// of a list in one launch: the 4-bit copies of the weights that a model's
// products read after an optimizer step, and the activations and output
// gradients of those products.
//
// A source [R, C] is cut into 128 x 128 tiles, one CTA each.  A thread loads
// 16 consecutive values of a row at a time (one block of MUON_FP4_NV, half a
// block of MUON_FP4_MX), so the form along the columns comes straight from
// registers; for the form along the rows (the transpose, blocks down a
// column) the tile is kept in shared memory and read back by column pairs.
// Both forms are so written from one read of the source.  A tile holds whole
// blocks and whole scale atoms in both directions, so no two CTAs share an
// output byte.  MUON_FP4_NV needs the matrix's largest magnitude first: one
// more pass over the source, whose maximum (over bits, order does not matter)
// is kept beside the scale.
#include "fp4.cuh"

#include <new>

namespace {

using namespace muon;
using namespace muon::fp4;

constexpr int kTile = 128;
constexpr int kThreads = 256;

struct Form {
  uint8_t* data;   // codes, NULL: this form is not wanted
  uint8_t* scales;
  float* ts;       // tensor scale (NV)
  int64_t pitch;
  int64_t atoms;   // scale atoms of a row block
};

struct Item {
  const void* src;
  int64_t ld;      // elements
  int32_t rows, cols;
  int32_t tiles_x; // tiles of 128 columns
  int32_t vec;     // rows start on 16-byte boundaries
  unsigned* amax;  // NV: bits of the largest finite magnitude
  Form c, r;       // along the columns [rows, cols], along the rows [cols, rows]
};

struct TileRef {
  int32_t item, tile;
};

template <typename T>
struct Src;
template <>
struct Src<__nv_bfloat16> {
  static constexpr int kWords = 8;                 // words of 16 values
  static constexpr int kPitch = kTile * 2 + 16;    // shared-memory row
};
template <>
struct Src<float> {
  static constexpr int kWords = 16;
  static constexpr int kPitch = kTile * 4 + 16;
};

// 16 values of row `row` from column `col` on, as words; zeros past the edges.
template <typename T>
__device__ __forceinline__ void load16(const Item& it, int row, int col, uint32_t (&w)[Src<T>::kWords]) {
  constexpr int kW = Src<T>::kWords;
  if (row >= it.rows || col >= it.cols) {
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = 0u;
    return;
  }
  const T* p = static_cast<const T*>(it.src) + static_cast<int64_t>(row) * it.ld + col;
  if (it.vec && col + 16 <= it.cols) {
#pragma unroll
    for (int i = 0; i < kW / 4; ++i) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
    return;
  }
  const int left = it.cols - col;
  if (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = i < left ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p) + 2 * i;
      const uint32_t lo = 2 * i < left ? __ldg(h) : 0u, hi = 2 * i + 1 < left ? __ldg(h + 1) : 0u;
      w[i] = lo | (hi << 16);
    }
  }
}

// Bits (as fp32) of the largest magnitude of 16 values.
template <typename T>
__device__ __forceinline__ uint32_t amax16(const uint32_t (&w)[Src<T>::kWords]) {
  if (sizeof(T) == 4) {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < Src<T>::kWords; ++i) a = max(a, w[i] & 0x7FFFFFFFu);
    return a;
  }
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < Src<T>::kWords; ++i) a = __vmaxu2(a, w[i] & 0x7FFF7FFFu);
  return max(a & 0xFFFF0000u, a << 16);
}

template <typename T>
__device__ __forceinline__ float value_at(const uint32_t (&w)[Src<T>::kWords], int i) {
  if (sizeof(T) == 4) return __uint_as_float(w[i]);
  const uint32_t v = w[i >> 1];
  return __uint_as_float((i & 1) ? (v & 0xFFFF0000u) : (v << 16));
}

__device__ __forceinline__ float scale_of_amax(uint32_t bits) {
  return __uint_as_float(static_cast<uint32_t>(tensor_exponent(bits) + 127) << 23);
}

// ---------------------------------------------------------------- largest magnitude
template <typename T>
__global__ void __launch_bounds__(kThreads) amax_kernel(const Item one, const Item* __restrict__ items,
                                                        const TileRef* __restrict__ tiles) {
  __shared__ uint32_t part[kThreads / 32];
  TileRef ref{0, static_cast<int32_t>(blockIdx.x)};
  if (tiles != nullptr) ref = tiles[blockIdx.x];
  const Item it = items != nullptr ? items[ref.item] : one;
  const int row0 = ref.tile / it.tiles_x * kTile, col0 = ref.tile % it.tiles_x * kTile;
  uint32_t a = 0u;
#pragma unroll 2
  for (int u = threadIdx.x; u < kTile * 8; u += kThreads) {
    uint32_t w[Src<T>::kWords];
    load16<T>(it, row0 + (u >> 3), col0 + (u & 7) * 16, w);
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < Src<T>::kWords; ++i) {
        const uint32_t m = w[i] & 0x7FFFFFFFu;
        a = max(a, m < 0x7F800000u ? m : 0u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < Src<T>::kWords; ++i) {
        const uint32_t hi = w[i] & 0x7FFF0000u, lo = (w[i] << 16) & 0x7FFF0000u;
        a = max(a, max(hi < 0x7F800000u ? hi : 0u, lo < 0x7F800000u ? lo : 0u));
      }
    }
  }
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    a = threadIdx.x < kThreads / 32 ? part[threadIdx.x] : 0u;
    a = __reduce_max_sync(0xffffffffu, a);
    if (threadIdx.x == 0 && a != 0u) atomicMax(it.amax, a);
  }
}

// ---------------------------------------------------------------- quantisation
template <typename T, bool kNv, bool kCols, bool kRows>
__global__ void __launch_bounds__(kThreads) quant_kernel(const Item one, const Item* __restrict__ items,
                                                         const TileRef* __restrict__ tiles) {
  constexpr int kW = Src<T>::kWords;
  constexpr int kPitch = Src<T>::kPitch;
  constexpr int kAtoms = kNv ? 2 : 1;      // scale atoms of a tile in one direction
  constexpr int kStage = kTile / 2 + 8;    // staged row of codes along the rows
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* stage = smem + kTile * kPitch;  // [128][kStage], rows form only
  __shared__ __align__(16) uint8_t sc_c[1024];
  __shared__ __align__(16) uint8_t sc_r[1024];
  TileRef ref{0, static_cast<int32_t>(blockIdx.x)};
  if (tiles != nullptr) ref = tiles[blockIdx.x];
  const Item it = items != nullptr ? items[ref.item] : one;
  const int ty = ref.tile / it.tiles_x, tx = ref.tile % it.tiles_x;
  const int row0 = ty * kTile, col0 = tx * kTile;
  const int t = threadIdx.x;
  float g = 1.0f;
  if (kNv) {
    const uint32_t bits = *it.amax;
    g = scale_of_amax(bits);
    if (ref.tile == 0 && t == 0) {
      if (kCols) {
        it.c.ts[0] = g;
        it.c.ts[1] = __uint_as_float(bits);
      }
      if (kRows) {
        it.r.ts[0] = g;
        it.r.ts[1] = __uint_as_float(bits);
      }
    }
  }

  // ---- by rows: units of 16 values, unit u = (row u / 8, columns 16 (u % 8))
#pragma unroll 2
  for (int k = 0; k < kTile * 8 / kThreads; ++k) {
    const int u = t + k * kThreads;
    const int r = u >> 3, c16 = u & 7;
    uint32_t w[kW];
    load16<T>(it, row0 + r, col0 + c16 * 16, w);
    if (kRows) {
      uint4* s = reinterpret_cast<uint4*>(smem + r * kPitch + c16 * 16 * sizeof(T));
#pragma unroll
      for (int i = 0; i < kW / 4; ++i) s[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    if (kCols) {
      uint32_t a = amax16<T>(w);
      if (!kNv) a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      const BlockScale bs = block_scale<kNv>(a, g);
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = scaled<kNv>(value_at<T>(w, i), bs);
      const int64_t byte = static_cast<int64_t>(col0) / 2 + c16 * 8;
      if (row0 + r < it.rows && byte < it.c.pitch)
        *reinterpret_cast<uint2*>(it.c.data + static_cast<int64_t>(row0 + r) * it.c.pitch + byte) =
            make_uint2(e2m1_pack8(v), e2m1_pack8(v + 8));
      if (kNv) sc_c[(c16 >> 2) * kAtomBytes + atom_byte(r, c16)] = static_cast<uint8_t>(bs.byte);
      else if ((c16 & 1) == 0) sc_c[atom_byte(r, c16 >> 1)] = static_cast<uint8_t>(bs.byte);
    }
  }
  __syncthreads();
  if (kCols && t < kAtoms * 32) {
    // the tile's atoms follow each other in memory; the second may be past the last
    const int64_t atom = static_cast<int64_t>(tx) * kAtoms + (t >> 5);
    if (atom < it.c.atoms)
      reinterpret_cast<uint4*>(it.c.scales + (static_cast<int64_t>(ty) * it.c.atoms + atom) * kAtomBytes)[t & 31] =
          reinterpret_cast<const uint4*>(sc_c)[t];
  }
  if (!kRows) return;

  // ---- by columns: unit = (column pair, block of rows)
  constexpr int kBlk = kNv ? 16 : 32;
  for (int u = t; u < (kTile / 2) * (kTile / kBlk); u += kThreads) {
    const int cp = u & 63, rb = u >> 6;
    const uint8_t* s = smem + rb * kBlk * kPitch + cp * 2 * sizeof(T);
    uint32_t x0[kBlk], x1[kBlk];  // as fp32 bits
    uint32_t a0 = 0u, a1 = 0u;
#pragma unroll
    for (int i = 0; i < kBlk; ++i) {
      if (sizeof(T) == 4) {
        const uint2 p = *reinterpret_cast<const uint2*>(s + i * kPitch);
        x0[i] = p.x;
        x1[i] = p.y;
      } else {
        const uint32_t p = *reinterpret_cast<const uint32_t*>(s + i * kPitch);
        x0[i] = p << 16;
        x1[i] = p & 0xFFFF0000u;
      }
      a0 = max(a0, x0[i] & 0x7FFFFFFFu);
      a1 = max(a1, x1[i] & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t* x = h ? x1 : x0;
      const BlockScale bs = block_scale<kNv>(h ? a1 : a0, g);
      const int c = 2 * cp + h;
      uint8_t* out = stage + c * kStage + rb * (kBlk / 2);
#pragma unroll
      for (int q = 0; q < kBlk / 16; ++q) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = scaled<kNv>(__uint_as_float(x[16 * q + i]), bs);
        *reinterpret_cast<uint2*>(out + 8 * q) = make_uint2(e2m1_pack8(v), e2m1_pack8(v + 8));
      }
      sc_r[(rb >> 2) * kAtomBytes + atom_byte(c, rb)] = static_cast<uint8_t>(bs.byte);
    }
  }
  __syncthreads();
  for (int u = t; u < kTile * 8; u += kThreads) {
    const int c = u >> 3, q = u & 7;
    const int64_t byte = static_cast<int64_t>(row0) / 2 + q * 8;
    if (col0 + c < it.cols && byte < it.r.pitch)
      *reinterpret_cast<uint2*>(it.r.data + static_cast<int64_t>(col0 + c) * it.r.pitch + byte) =
          *reinterpret_cast<const uint2*>(stage + c * kStage + q * 8);
  }
  if (t < kAtoms * 32) {
    const int64_t atom = static_cast<int64_t>(ty) * kAtoms + (t >> 5);
    if (atom < it.r.atoms)
      reinterpret_cast<uint4*>(it.r.scales + (static_cast<int64_t>(tx) * it.r.atoms + atom) * kAtomBytes)[t & 31] =
          reinterpret_cast<const uint4*>(sc_r)[t];
  }
}

template <typename T, bool kRows>
constexpr int quant_smem() {
  return kRows ? kTile * Src<T>::kPitch + kTile * (kTile / 2 + 8) : 0;
}

template <typename T, bool kNv, bool kCols, bool kRows>
cudaError_t launch_quant_t(const Item& one, const Item* items, const TileRef* tiles, int ntiles, cudaStream_t st) {
  constexpr int smem = quant_smem<T, kRows>();
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(quant_kernel<T, kNv, kCols, kRows>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  quant_kernel<T, kNv, kCols, kRows><<<ntiles, kThreads, smem, st>>>(one, items, tiles);
  return cudaGetLastError();
}

template <typename T, bool kNv>
cudaError_t launch_quant_n(const Item& one, const Item* items, const TileRef* tiles, int ntiles, bool cols, bool rows,
                           cudaStream_t st) {
  if (kNv) {
    amax_kernel<T><<<ntiles, kThreads, 0, st>>>(one, items, tiles);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (cols && rows) return launch_quant_t<T, kNv, true, true>(one, items, tiles, ntiles, st);
  if (cols) return launch_quant_t<T, kNv, true, false>(one, items, tiles, ntiles, st);
  return launch_quant_t<T, kNv, false, true>(one, items, tiles, ntiles, st);
}

cudaError_t launch_quant(const Item& one, const Item* items, const TileRef* tiles, int ntiles, int dtype, int format,
                         bool cols, bool rows, cudaStream_t st) {
  const bool nv = format == MUON_FP4_NV;
  if (dtype == MUON_DT_BF16)
    return nv ? launch_quant_n<__nv_bfloat16, true>(one, items, tiles, ntiles, cols, rows, st)
              : launch_quant_n<__nv_bfloat16, false>(one, items, tiles, ntiles, cols, rows, st);
  return nv ? launch_quant_n<float, true>(one, items, tiles, ntiles, cols, rows, st)
            : launch_quant_n<float, false>(one, items, tiles, ntiles, cols, rows, st);
}

// ---------------------------------------------------------------- back to values
struct Deq {
  const uint8_t* data;
  const uint8_t* scales;
  const float* ts;
  void* dst;
  int64_t ld;      // elements
  int64_t pitch, atoms;
  int32_t rows, k;
  int32_t vec;     // destination rows start on 16-byte boundaries
  int32_t units;   // ceil(k / 8): units of a row
};

constexpr int kDeqChunk = 8192;  // units (of 8 values) per CTA

struct DeqRef {
  int32_t item;
  int32_t pad;
  int64_t first;  // first unit of the CTA
};

template <typename T, bool kNv>
__global__ void __launch_bounds__(kThreads) dequant_kernel(const Deq one, const Deq* __restrict__ items,
                                                           const DeqRef* __restrict__ refs) {
  DeqRef ref{0, 0, static_cast<int64_t>(blockIdx.x) * kDeqChunk};
  if (refs != nullptr) ref = refs[blockIdx.x];
  const Deq it = items != nullptr ? items[ref.item] : one;
  const int64_t total = static_cast<int64_t>(it.rows) * it.units;
  const int64_t left = total - ref.first;
  const int n = static_cast<int>(left < kDeqChunk ? left : kDeqChunk);
  const float g = kNv ? it.ts[0] : 1.0f;
  // the CTA's first unit by one wide division, the rest relative to it
  const int64_t first_row = ref.first / it.units;
  const uint32_t first_unit = static_cast<uint32_t>(ref.first - first_row * it.units);
#pragma unroll 4
  for (int e = threadIdx.x; e < n; e += kThreads) {
    const uint32_t lin = first_unit + static_cast<uint32_t>(e);
    const uint32_t dr = lin / static_cast<uint32_t>(it.units);
    const int unit = static_cast<int>(lin - dr * static_cast<uint32_t>(it.units));
    const int64_t row = first_row + dr;
    const int b = unit / (kNv ? 2 : 4);
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(it.data + row * it.pitch) + unit);
    const uint32_t sb = __ldg(it.scales + ((row >> 7) * it.atoms + (b >> 2)) * kAtomBytes +
                              atom_byte(static_cast<int>(row & 127), b));
    const float s = kNv ? e4m3_value(sb) * g : e8m0_value(sb);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = e2m1_pair((w >> (8 * i)) & 0xFFu);
      v[2 * i] = p.x * s;
      v[2 * i + 1] = p.y * s;
    }
    const int k0 = unit * 8;
    T* out = static_cast<T*>(it.dst) + row * it.ld + k0;
    if (it.vec && k0 + 8 <= it.k) {
      if (sizeof(T) == 4) {
        reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        __align__(16) __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k0 + i < it.k) {
          if (sizeof(T) == 4) reinterpret_cast<float*>(out)[i] = v[i];
          else reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v[i]);
        }
    }
  }
}

cudaError_t launch_dequant(const Deq& one, const Deq* items, const DeqRef* refs, int64_t nblocks, int dtype, int format,
                           cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(nblocks));
  const bool nv = format == MUON_FP4_NV;
  if (dtype == MUON_DT_BF16) {
    if (nv) dequant_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(one, items, refs);
    else dequant_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(one, items, refs);
  } else {
    if (nv) dequant_kernel<float, true><<<grid, kThreads, 0, st>>>(one, items, refs);
    else dequant_kernel<float, false><<<grid, kThreads, 0, st>>>(one, items, refs);
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------- host checks
bool valid_dtype(int32_t d) { return d == MUON_DT_BF16 || d == MUON_DT_FP32; }
int size_of(int32_t d) { return d == MUON_DT_BF16 ? 2 : 4; }

ByteRange matrix_range(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + (static_cast<size_t>(rows - 1) * ld + cols) * size_of(dtype)};
}

// A source and its two forms; fills `it` and says whether there is work.
muon_status_t make_item(const muon_fp4_source_t& s, Item& it, bool& empty) {
  empty = true;
  if (!valid_dtype(s.src_dtype) || s.reserved != 0 || s.rows < 0 || s.cols < 0 || s.rows > kMaxDim || s.cols > kMaxDim)
    return MUON_ERR_INVALID_ARG;
  const bool c = s.along_cols.format >= 0, r = s.along_rows.format >= 0;
  if (!c && !r) return MUON_ERR_INVALID_ARG;
  if (c && !valid(s.along_cols)) return MUON_ERR_INVALID_ARG;
  if (r && !valid(s.along_rows)) return MUON_ERR_INVALID_ARG;
  if (c && r && s.along_cols.format != s.along_rows.format) return MUON_ERR_INVALID_ARG;
  if (c && (s.along_cols.rows != s.rows || s.along_cols.k != s.cols)) return MUON_ERR_SHAPE_MISMATCH;
  if (r && (s.along_rows.rows != s.cols || s.along_rows.k != s.rows)) return MUON_ERR_SHAPE_MISMATCH;
  if (s.rows == 0 || s.cols == 0) return MUON_OK;
  if (s.src == nullptr || s.ld < s.cols || s.ld > (int64_t(1) << 40)) return MUON_ERR_INVALID_ARG;
  const int es = size_of(s.src_dtype);
  const uintptr_t a = reinterpret_cast<uintptr_t>(s.src);
  if (a % es != 0) return MUON_ERR_INVALID_ARG;
  const int64_t tx = (s.cols + kTile - 1) / kTile, ty = (s.rows + kTile - 1) / kTile;
  if (tx * ty > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
  it = Item{};
  it.src = s.src;
  it.ld = s.ld;
  it.rows = static_cast<int32_t>(s.rows);
  it.cols = static_cast<int32_t>(s.cols);
  it.tiles_x = static_cast<int32_t>(tx);
  it.vec = (a % 16 == 0 && s.ld * es % 16 == 0) ? 1 : 0;
  auto form = [](const muon_fp4_matrix_t& m) {
    return Form{static_cast<uint8_t*>(m.data), static_cast<uint8_t*>(m.scales), m.tensor_scale, pitch_of(m.k),
                atoms_of(m.format, m.k)};
  };
  if (c) it.c = form(s.along_cols);
  if (r) it.r = form(s.along_rows);
  empty = false;
  return MUON_OK;
}

int tiles_of(const Item& it) { return it.tiles_x * ((it.rows + kTile - 1) / kTile); }

template <class List>
void item_ranges(const muon_fp4_source_t& s, List& reads, List& writes) {
  reads.push_back(matrix_range(s.src, s.rows, s.cols, s.ld, s.src_dtype));
  if (s.along_cols.format >= 0) add_ranges(s.along_cols, writes);
  if (s.along_rows.format >= 0) add_ranges(s.along_rows, writes);
}

muon_status_t make_deq(const muon_fp4_matrix_t& m, void* dst, int64_t ld, int32_t dtype, Deq& d) {
  if (dst == nullptr || ld < m.k || ld > (int64_t(1) << 40)) return MUON_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(dst);
  if (a % size_of(dtype) != 0) return MUON_ERR_INVALID_ARG;
  d = Deq{static_cast<const uint8_t*>(m.data), static_cast<const uint8_t*>(m.scales), m.tensor_scale, dst, ld,
          pitch_of(m.k), atoms_of(m.format, m.k), static_cast<int32_t>(m.rows), static_cast<int32_t>(m.k),
          (a % 16 == 0 && ld * size_of(dtype) % 16 == 0) ? 1 : 0, static_cast<int32_t>((m.k + 7) / 8)};
  return MUON_OK;
}

int64_t deq_blocks(const Deq& d) {
  return (static_cast<int64_t>(d.rows) * d.units + kDeqChunk - 1) / kDeqChunk;
}

}  // namespace

struct muon_fp4_plan_s {
  int device = 0;
  int dtype = 0, format = 0, values_dtype = -1;
  bool cols = false, rows = false;
  int ntiles = 0, nitems = 0;
  int64_t ndeq = 0;
  uint8_t* dmem = nullptr;
  Item* items_d = nullptr;
  TileRef* tiles_d = nullptr;
  unsigned* amax_d = nullptr;
  Deq* deqs_d = nullptr;
  DeqRef* refs_d = nullptr;
  cudaStream_t last_stream = nullptr;
};

extern "C" {

muon_status_t muon_fp4_sizes(int32_t format, int64_t rows, int64_t k, int64_t* pitch, size_t* data_bytes,
                             size_t* scale_bytes) {
  if ((format != MUON_FP4_MX && format != MUON_FP4_NV) || rows < 0 || k < 0 || rows > kMaxDim || k > kMaxDim)
    return MUON_ERR_INVALID_ARG;
  if (pitch != nullptr) *pitch = pitch_of(k);
  if (data_bytes != nullptr) *data_bytes = data_bytes_of(rows, k);
  if (scale_bytes != nullptr) *scale_bytes = scale_bytes_of(format, rows, k);
  return MUON_OK;
}

muon_status_t muon_fp4_quantize(const muon_fp4_source_t* src, void* stream) {
  if (src == nullptr) return MUON_ERR_INVALID_ARG;
  Item it;
  bool empty = true;
  const muon_status_t s = make_item(*src, it, empty);
  if (s != MUON_OK || empty) return s;
  RangeList reads, writes;
  item_ranges(*src, reads, writes);
  if (conflict(reads, writes)) return MUON_ERR_ALIAS;
  const bool c = it.c.data != nullptr, r = it.r.data != nullptr;
  const int format = c ? src->along_cols.format : src->along_rows.format;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (format == MUON_FP4_NV) {
    it.amax = reinterpret_cast<unsigned*>((c ? it.c.ts : it.r.ts) + 1);
    if (cudaMemsetAsync(it.amax, 0, sizeof(unsigned), st) != cudaSuccess) {
      cudaGetLastError();
      return MUON_ERR_CUDA;
    }
  }
  return launch_quant(it, nullptr, nullptr, tiles_of(it), src->src_dtype, format, c, r, st) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

muon_status_t muon_fp4_dequantize(const muon_fp4_matrix_t* m, void* dst, int64_t ld, int32_t dst_dtype, void* stream) {
  if (m == nullptr || !valid(*m) || !valid_dtype(dst_dtype)) return MUON_ERR_INVALID_ARG;
  if (m->rows == 0 || m->k == 0) return MUON_OK;
  Deq d;
  const muon_status_t s = make_deq(*m, dst, ld, dst_dtype, d);
  if (s != MUON_OK) return s;
  RangeList reads, writes;
  writes.push_back(matrix_range(dst, m->rows, m->k, ld, dst_dtype));
  add_ranges(*m, reads);
  if (conflict(reads, writes)) return MUON_ERR_ALIAS;
  const int64_t nb = deq_blocks(d);
  if (nb > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
  return launch_dequant(d, nullptr, nullptr, nb, dst_dtype, m->format, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

muon_status_t muon_fp4_init(muon_fp4_plan_t* out, const muon_fp4_source_t* srcs, int32_t n, int32_t values_dtype,
                            void* stream) {
  if (out == nullptr) return MUON_ERR_INVALID_ARG;
  *out = nullptr;
  if (srcs == nullptr || n < 1 || n > (1 << 24)) return MUON_ERR_INVALID_ARG;
  if (values_dtype >= 0 && !valid_dtype(values_dtype)) return MUON_ERR_INVALID_ARG;
  muon_fp4_plan_s* pl = nullptr;
  try {
    std::vector<Item> items;
    std::vector<TileRef> tiles;
    std::vector<Deq> deqs;
    std::vector<DeqRef> refs;
    std::vector<ByteRange> reads, writes;
    const bool c = srcs[0].along_cols.format >= 0, r = srcs[0].along_rows.format >= 0;
    const int32_t format = c ? srcs[0].along_cols.format : srcs[0].along_rows.format;
    for (int32_t i = 0; i < n; ++i) {
      const muon_fp4_source_t& s = srcs[i];
      Item it;
      bool empty = true;
      const muon_status_t e = make_item(s, it, empty);
      if (e != MUON_OK) return e;
      // one launch covers the list: one source type, one format, the same forms
      if (s.src_dtype != srcs[0].src_dtype || (s.along_cols.format >= 0) != c || (s.along_rows.format >= 0) != r ||
          (c ? s.along_cols.format : s.along_rows.format) != format)
        return MUON_ERR_INVALID_ARG;
      if (empty) continue;
      item_ranges(s, reads, writes);
      const int32_t id = static_cast<int32_t>(items.size());
      items.push_back(it);
      const int nt = tiles_of(it);
      if (static_cast<int64_t>(tiles.size()) + nt > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
      for (int k = 0; k < nt; ++k) tiles.push_back(TileRef{id, k});
      if (values_dtype >= 0)
        for (int f = 0; f < 2; ++f) {
          if (f == 0 ? !c : !r) continue;
          const muon_fp4_matrix_t& m = f == 0 ? s.along_cols : s.along_rows;
          void* dst = f == 0 ? s.values_cols : s.values_rows;
          if (dst == nullptr) return MUON_ERR_INVALID_ARG;
          Deq d;
          const muon_status_t e2 = make_deq(m, dst, m.k, values_dtype, d);
          if (e2 != MUON_OK) return e2;
          writes.push_back(matrix_range(dst, m.rows, m.k, m.k, values_dtype));
          const int32_t did = static_cast<int32_t>(deqs.size());
          deqs.push_back(d);
          for (int64_t b = 0; b < deq_blocks(d); ++b) refs.push_back(DeqRef{did, 0, b * kDeqChunk});
        }
    }
    if (conflict(reads, writes)) return MUON_ERR_ALIAS;
    if (refs.size() > static_cast<size_t>(0x7fffffff)) return MUON_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MUON_ERR_CUDA;
    pl = new (std::nothrow) muon_fp4_plan_s();
    if (pl == nullptr) return MUON_ERR_NO_MEMORY;
    pl->device = dev;
    pl->dtype = srcs[0].src_dtype;
    pl->format = format;
    pl->values_dtype = values_dtype;
    pl->cols = c;
    pl->rows = r;
    pl->nitems = static_cast<int>(items.size());
    pl->ntiles = static_cast<int>(tiles.size());
    pl->ndeq = static_cast<int64_t>(refs.size());
    pl->last_stream = static_cast<cudaStream_t>(stream);
    if (!items.empty()) {
      auto up = [](size_t b) { return (b + 255) / 256 * 256; };
      const size_t bi = up(items.size() * sizeof(Item)), bt = up(tiles.size() * sizeof(TileRef)),
                   ba = up(items.size() * sizeof(unsigned)), bd = up(deqs.size() * sizeof(Deq)),
                   br = up(refs.size() * sizeof(DeqRef));
      if (cudaMalloc(&pl->dmem, bi + bt + ba + bd + br) != cudaSuccess) {
        cudaGetLastError();
        delete pl;
        return MUON_ERR_NO_MEMORY;
      }
      pl->items_d = reinterpret_cast<Item*>(pl->dmem);
      pl->tiles_d = reinterpret_cast<TileRef*>(pl->dmem + bi);
      pl->amax_d = reinterpret_cast<unsigned*>(pl->dmem + bi + bt);
      pl->deqs_d = reinterpret_cast<Deq*>(pl->dmem + bi + bt + ba);
      pl->refs_d = reinterpret_cast<DeqRef*>(pl->dmem + bi + bt + ba + bd);
      for (size_t i = 0; i < items.size(); ++i) items[i].amax = pl->amax_d + i;
      auto put = [](void* d, const void* h, size_t b) {
        return b == 0 || cudaMemcpy(d, h, b, cudaMemcpyHostToDevice) == cudaSuccess;
      };
      if (!put(pl->items_d, items.data(), items.size() * sizeof(Item)) ||
          !put(pl->tiles_d, tiles.data(), tiles.size() * sizeof(TileRef)) ||
          !put(pl->deqs_d, deqs.data(), deqs.size() * sizeof(Deq)) ||
          !put(pl->refs_d, refs.data(), refs.size() * sizeof(DeqRef))) {
        cudaGetLastError();
        cudaFree(pl->dmem);
        delete pl;
        return MUON_ERR_CUDA;
      }
    }
  } catch (const std::bad_alloc&) {
    return MUON_ERR_NO_MEMORY;
  }
  *out = pl;
  return MUON_OK;
}

muon_status_t muon_fp4_run(muon_fp4_plan_t pl, void* stream) {
  if (pl == nullptr) return MUON_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pl->device) return MUON_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  pl->last_stream = st;
  if (pl->nitems == 0) return MUON_OK;
  if (pl->format == MUON_FP4_NV && cudaMemsetAsync(pl->amax_d, 0, pl->nitems * sizeof(unsigned), st) != cudaSuccess) {
    cudaGetLastError();
    return MUON_ERR_CUDA;
  }
  return launch_quant(Item{}, pl->items_d, pl->tiles_d, pl->ntiles, pl->dtype, pl->format, pl->cols, pl->rows, st) ==
                 cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

muon_status_t muon_fp4_values(muon_fp4_plan_t pl, void* stream) {
  if (pl == nullptr || pl->values_dtype < 0) return MUON_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pl->device) return MUON_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  pl->last_stream = st;
  if (pl->ndeq == 0) return MUON_OK;
  return launch_dequant(Deq{}, pl->deqs_d, pl->refs_d, pl->ndeq, pl->values_dtype, pl->format, st) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

void muon_fp4_destroy(muon_fp4_plan_t pl) {
  if (pl == nullptr) return;
  cudaStreamSynchronize(pl->last_stream);
  cudaGetLastError();
  cudaFree(pl->dmem);
  delete pl;
}

}  // extern "C"
