// Quantisation to 4-bit matrices and back (format: fp4.cuh), of one matrix or
// of a list in one launch: the 4-bit copies of the weights that a model's
// products read after an optimizer step, and the activations and output
// gradients of those products.
//
// A source [R, C] is cut into tiles of 64 rows x 128 columns, one CTA each
// (128 x 128 left two CTAs of fp32 tiles a SM, whose loads and column passes
// hardly overlapped).  A thread takes 16 consecutive values of a row at a time
// (one block of MUON_FP4_NV, half a block of MUON_FP4_MX), so the form along
// the columns comes straight from registers; for the form along the rows (the
// transpose, blocks down a column) the tile is kept in shared memory and read
// back by columns.  Both forms are so written from one read of the source.  A
// tile holds whole blocks in both directions, so no two CTAs write a byte;
// there is an even number of tile rows, so that whole scale atoms are written.
// MUON_FP4_NV needs the matrix's largest magnitude first: one more pass over
// the source (the maximum of its bits, whose order does not matter).  (Running
// a list in groups that stay in L2 between the passes was slower for every
// group size: 24 fp32 matrices of 2048 x 1408, both forms, 155 us in one piece,
// 173 to 221 us in groups of 100 to 24 MB, whose launches do not fill the GPU.)
// Both kernels are bound by the instructions they issue, so the set-up of a
// thread counts as much as its 32 values: a single matrix is described by
// kernel parameters, a list by tables, in kernels of their own, and tiles
// inside the matrix load and store without looking at its edges.
#include "fp4.cuh"

#include <new>

namespace {

using namespace muon;
using namespace muon::fp4;

constexpr int kTileR = 64, kTile = 128;  // rows and columns of a tile
constexpr int kThreads = 256;
// NV matrices of up to so many values (a few tokens) are looked through by
// every CTA instead of in a pass before: one launch instead of a memset and
// two.  A CTA reads 64 values a thread at most.
constexpr int64_t kSmall = 16384;

constexpr int kStagePitch = kTileR / 2 + 8;  // a staged row of codes along the rows
static_assert(kTileR * kTile * 4 + kTile * kStagePitch <= 48 * 1024, "dynamic shared memory without opt-in");

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
  int32_t tiles_x, tiles_y;  // tiles of 128 columns and 64 rows, the latter an even number
  int32_t vec;     // rows start on 16-byte boundaries
  unsigned* amax;  // NV: bits of the largest finite magnitude; NULL (a single small matrix): found by every CTA
  Form c, r;       // along the columns [rows, cols], along the rows [cols, rows]
};

struct TileRef {
  int32_t item, tx, ty;
};

constexpr int kGridY = 32768;  // tile rows of a single matrix along the grid's y, the rest along z

template <bool kList>
__device__ __forceinline__ TileRef my_tile(const TileRef* __restrict__ tiles) {
  if constexpr (kList) return tiles[blockIdx.x];
  else return TileRef{0, static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(blockIdx.z * kGridY + blockIdx.y)};
}

template <typename T>
struct Src;
template <>
struct Src<__nv_bfloat16> {
  using Raw = unsigned short;
  static constexpr int kWords = 8;                 // words of 16 values
  static constexpr int kPitch = kTile * 2;         // shared-memory row
};
template <>
struct Src<float> {
  using Raw = unsigned int;
  static constexpr int kWords = 16;
  static constexpr int kPitch = kTile * 4;
};

// Where 16-byte piece j of a row lies in the shared-memory tile.  The pieces of
// each 128 bytes are permuted: a thread stores the pieces of its 16 values one
// by one, and without this the eight threads of a row would meet the same
// banks (64 or 32 bytes apart); a warp that reads 128 bytes of a row meets
// every bank once either way.
template <typename T>
__device__ __forceinline__ int swizzled(int j) {
  return j ^ ((j >> 3) & (sizeof(T) == 4 ? 3 : 1));
}

// 16 values on a 16-byte boundary, as words.
template <typename T>
__device__ __forceinline__ void load16(const T* p, uint32_t (&w)[Src<T>::kWords]) {
#pragma unroll
  for (int i = 0; i < Src<T>::kWords / 4; ++i) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
    w[4 * i] = q.x;
    w[4 * i + 1] = q.y;
    w[4 * i + 2] = q.z;
    w[4 * i + 3] = q.w;
  }
}

// 16 values of row `row` from column `col` on; zeros past the edges.
template <typename T>
__device__ __forceinline__ void load16_edge(const Item& it, int row, int col, uint32_t (&w)[Src<T>::kWords]) {
  constexpr int kW = Src<T>::kWords;
  if (row >= it.rows || col >= it.cols) {
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = 0u;
    return;
  }
  const T* p = static_cast<const T*>(it.src) + static_cast<int64_t>(row) * it.ld + col;
  if (col + 16 <= it.cols) {
    load16<T>(p, w);
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

// This thread's units of a tile: unit k is row t / 8 + 32 k, columns 16 (t % 8) on.
constexpr int kUnits = kTileR * 8 / kThreads;
template <typename T>
__device__ __forceinline__ void load_units(const Item& it, int row0, int col0, bool inside,
                                           uint32_t (&w)[kUnits][Src<T>::kWords]) {
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 16;
  if (inside) {
    const T* p = static_cast<const T*>(it.src) + static_cast<int64_t>(row0 + r) * it.ld + (col0 + c);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) load16<T>(p + static_cast<int64_t>(k * (kThreads / 8)) * it.ld, w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) load16_edge<T>(it, row0 + r + k * (kThreads / 8), col0 + c, w[k]);
  }
}

// The tile of a source whose rows start anywhere: a warp's lanes take
// consecutive values of a row, into the shared-memory tile.
template <typename T>
__device__ __forceinline__ void fill_tile(const Item& it, int row0, int col0, uint8_t* smem) {
  using Raw = typename Src<T>::Raw;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 4
  for (int r = warp; r < kTileR; r += kThreads / 32) {
    const Raw* p = static_cast<const Raw*>(it.src) + static_cast<int64_t>(row0 + r) * it.ld + col0;
    constexpr int kPiece = 16 / sizeof(T);
#pragma unroll
    for (int c = 0; c < kTile; c += 32) {
      Raw* d = reinterpret_cast<Raw*>(smem + r * Src<T>::kPitch + swizzled<T>((c + lane) / kPiece) * 16);
      d[lane % kPiece] = row0 + r < it.rows && col0 + c + lane < it.cols ? __ldg(p + c + lane) : Raw(0);
    }
  }
}

// The larger magnitude; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Bits (as fp32) of the largest magnitude of 16 values; at or above infinity's
// bits where one is not finite.
template <typename T>
__device__ __forceinline__ uint32_t amax16(const uint32_t (&w)[Src<T>::kWords]) {
  if (sizeof(T) == 4) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < Src<T>::kWords; ++i) a = max_nan(a, fabsf(__uint_as_float(w[i])));
    return __float_as_uint(a);
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

// ---------------------------------------------------------------- largest magnitude
// bits, or 0 for a NaN or an infinity
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  const uint32_t m = w & 0x7FFFFFFFu;
  return m < 0x7F800000u ? m : 0u;
}

template <typename T, bool kList>
__global__ void __launch_bounds__(kThreads) amax_kernel(const __grid_constant__ Item one, const Item* __restrict__ items,
                                                        const TileRef* __restrict__ tiles) {
  __shared__ uint32_t part[kThreads / 32];
  const TileRef ref = my_tile<kList>(tiles);
  Item listed;
  if constexpr (kList) listed = items[ref.item];  // all of it at once
  const Item& it = kList ? listed : one;
  const int row0 = ref.ty * kTileR, col0 = ref.tx * kTile;
  pdl_trigger();
  if (row0 >= it.rows) return;  // the tiles that only fill up scale atoms
  uint32_t a = 0u;
  if (it.vec) {
    uint32_t w[kUnits][Src<T>::kWords];
    load_units<T>(it, row0, col0, row0 + kTileR <= it.rows && col0 + kTile <= it.cols, w);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) a = max(a, amax16<T>(w[k]));
    if (a >= 0x7F800000u) {  // not finite: the finite values alone
      a = 0u;
#pragma unroll
      for (int k = 0; k < kUnits; ++k)
#pragma unroll
        for (int i = 0; i < Src<T>::kWords; ++i) {
          if (sizeof(T) == 4) a = max(a, finite_bits(w[k][i]));
          else a = max(a, max(finite_bits(w[k][i] & 0xFFFF0000u), finite_bits(w[k][i] << 16)));
        }
    }
  } else {
    using Raw = typename Src<T>::Raw;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 4
    for (int r = warp; r < kTileR; r += kThreads / 32) {
      const Raw* p = static_cast<const Raw*>(it.src) + static_cast<int64_t>(row0 + r) * it.ld + col0;
#pragma unroll
      for (int c = 0; c < kTile; c += 32)
        if (row0 + r < it.rows && col0 + c + lane < it.cols)
          a = max(a, finite_bits(static_cast<uint32_t>(__ldg(p + c + lane)) << (sizeof(T) == 4 ? 0 : 16)));
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

// The same of a whole small matrix by every CTA for itself.
template <typename T>
__device__ uint32_t small_amax(const Item& it) {
  using Raw = typename Src<T>::Raw;
  __shared__ uint32_t part[kThreads / 32];
  const uint32_t n = static_cast<uint32_t>(it.rows) * static_cast<uint32_t>(it.cols);
  uint32_t a = 0u;
#pragma unroll 8
  for (uint32_t e = threadIdx.x; e < n; e += kThreads) {
    const uint32_t r = e / static_cast<uint32_t>(it.cols);
    const Raw* p = static_cast<const Raw*>(it.src) + static_cast<int64_t>(r) * it.ld + (e - r * it.cols);
    a = max(a, finite_bits(static_cast<uint32_t>(__ldg(p)) << (sizeof(T) == 4 ? 0 : 16)));
  }
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = max(a, part[i]);
  return a;
}

// ---------------------------------------------------------------- quantisation
template <typename T, bool kNv, bool kCols, bool kRows, bool kList>
__global__ void __launch_bounds__(kThreads) quant_kernel(const __grid_constant__ Item one,
                                                         const Item* __restrict__ items,
                                                         const TileRef* __restrict__ tiles) {
  constexpr int kW = Src<T>::kWords;
  constexpr int kPitch = Src<T>::kPitch;
  constexpr int kBlk = kNv ? 16 : 32;
  constexpr int kAtomsC = kTile / (4 * kBlk);  // atoms of a tile along the columns (of each, the half with its 64 rows)
  extern __shared__ __align__(16) uint8_t smem[];  // the tile: rows form, or rows that start anywhere
  uint8_t* stage = smem + kTileR * kPitch;         // [128][kStagePitch] codes along the rows
  __shared__ __align__(16) uint8_t sc_c[kAtomsC * 256];
  __shared__ __align__(16) uint8_t sc_r[kAtomBytes];
  // NV: the tiles that the pass before read last come first, being in L2
  const TileRef ref = kList && kNv ? tiles[gridDim.x - 1 - blockIdx.x] : my_tile<kList>(tiles);
  Item listed;
  if constexpr (kList) listed = items[ref.item];  // all of it at once
  const Item& it = kList ? listed : one;
  if (!kList && ref.ty >= it.tiles_y) return;
  const int tx = ref.tx, ty = !kList && kNv ? it.tiles_y - 1 - ref.ty : ref.ty;
  const int row0 = ty * kTileR, col0 = tx * kTile;
  const bool inside = row0 + kTileR <= it.rows && col0 + kTile <= it.cols;
  const int half = ty & 1;  // of the 128 rows of an atom
  const int t = threadIdx.x;

  // ---- by rows: units of 16 values, unit u = (row u / 8, columns 16 (u % 8))
  constexpr int kN = kUnits;
  uint32_t w[kN][kW];
  if (it.vec) {
    load_units<T>(it, row0, col0, inside, w);
    if (kRows) {
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        uint4* s = reinterpret_cast<uint4*>(smem + ((t >> 3) + k * (kThreads / 8)) * kPitch);
#pragma unroll
        for (int i = 0; i < kW / 4; ++i)
          s[swizzled<T>((t & 7) * (kW / 4) + i)] = make_uint4(w[k][4 * i], w[k][4 * i + 1], w[k][4 * i + 2], w[k][4 * i + 3]);
      }
    }
  } else {
    fill_tile<T>(it, row0, col0, smem);
    __syncthreads();
    if (kCols) {
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const uint4* s = reinterpret_cast<const uint4*>(smem + ((t >> 3) + k * (kThreads / 8)) * kPitch);
#pragma unroll
        for (int i = 0; i < kW / 4; ++i) {
          const uint4 q = s[swizzled<T>((t & 7) * (kW / 4) + i)];
          w[k][4 * i] = q.x;
          w[k][4 * i + 1] = q.y;
          w[k][4 * i + 2] = q.z;
          w[k][4 * i + 3] = q.w;
        }
      }
    }
  }
  MatrixScale g = {};
  if (kNv) {
    // the pass before (which started after everything before it had ended) may
    // still run while this tile is loaded; its maximum, and all writes, wait
    pdl_wait();
    const uint32_t bits = !kList && it.amax == nullptr ? small_amax<T>(it) : *it.amax;
    g = matrix_scale(bits);
    if ((tx | ty | t) == 0) {
      if (kCols) {
        it.c.ts[0] = g.g;
        it.c.ts[1] = __uint_as_float(bits);
      }
      if (kRows) {
        it.r.ts[0] = g.g;
        it.r.ts[1] = __uint_as_float(bits);
      }
    }
  }
  if (kCols) {
    const int c16 = t & 7;
    const int64_t byte = static_cast<int64_t>(col0) / 2 + c16 * 8;
    uint8_t* out = it.c.data + static_cast<int64_t>(row0 + (t >> 3)) * it.c.pitch + byte;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int r = (t >> 3) + k * (kThreads / 8);
      uint32_t a = amax16<T>(w[k]);
      if (!kNv) a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      const BlockScale bs = block_scale<kNv>(a, g);
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = value_at<T>(w[k], i);
      if (inside || (row0 + r < it.rows && byte < it.c.pitch))
        *reinterpret_cast<uint2*>(out + static_cast<int64_t>(k * (kThreads / 8)) * it.c.pitch) =
            make_uint2(codes8<kNv>(v, bs), codes8<kNv>(v + 8, bs));
      // [atom][r % 32][r / 32][block]: the tile's half of each 16 bytes
      const int b = kNv ? c16 : c16 >> 1;
      if (kNv || (c16 & 1) == 0) sc_c[(b >> 2) * 256 + (r & 31) * 8 + (r >> 5) * 4 + (b & 3)] = static_cast<uint8_t>(bs.byte);
    }
  }
  if (kCols || it.vec) __syncthreads();
  if (kCols && t < kAtomsC * 32) {
    // the tile's atoms follow each other in memory; the second may be past the last
    const int64_t atom = static_cast<int64_t>(tx) * kAtomsC + (t >> 5);
    if (atom < it.c.atoms)
      *reinterpret_cast<uint2*>(it.c.scales + (static_cast<int64_t>(ty >> 1) * it.c.atoms + atom) * kAtomBytes +
                                (t & 31) * 16 + half * 8) = reinterpret_cast<const uint2*>(sc_c)[t];
  }
  if (!kRows) return;

  // ---- by columns: NV a thread takes two columns of one block of rows, MX one column
  static_assert(kTile / (kNv ? 2 : 1) * (kTileR / kBlk) == kThreads, "one unit a thread");
  {
    constexpr int kCw = kNv ? 2 : 1;
    const int c0 = (t % (kTile / kCw)) * kCw, rb = t / (kTile / kCw);
    constexpr int kPiece = 16 / sizeof(T);
    const uint8_t* s = smem + rb * kBlk * kPitch + swizzled<T>(c0 / kPiece) * 16 + c0 % kPiece * sizeof(T);
    uint32_t x[kCw][kBlk];  // as fp32 bits
    uint32_t a[kCw] = {}, both = 0u;
    float m[kCw] = {};
#pragma unroll
    for (int i = 0; i < kBlk; ++i) {
      if constexpr (kNv) {
        if (sizeof(T) == 4) {
          const uint2 p = *reinterpret_cast<const uint2*>(s + i * kPitch);
          x[0][i] = p.x;
          x[1][i] = p.y;
        } else {
          const uint32_t p = *reinterpret_cast<const uint32_t*>(s + i * kPitch);
          x[0][i] = p << 16;
          x[1][i] = p & 0xFFFF0000u;
          both = __vmaxu2(both, p & 0x7FFF7FFFu);
        }
      } else {
        x[0][i] = sizeof(T) == 4 ? *reinterpret_cast<const uint32_t*>(s + i * kPitch)
                                 : static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(s + i * kPitch)) << 16;
      }
      if (sizeof(T) == 4 || !kNv) {
#pragma unroll
        for (int h = 0; h < kCw; ++h) m[h] = max_nan(m[h], fabsf(__uint_as_float(x[h][i])));
      }
    }
    if (sizeof(T) == 2 && kNv) {
      a[0] = both << 16;
      a[kCw - 1] = both & 0xFFFF0000u;
    } else {
#pragma unroll
      for (int h = 0; h < kCw; ++h) a[h] = __float_as_uint(m[h]);
    }
#pragma unroll
    for (int h = 0; h < kCw; ++h) {
      const BlockScale bs = block_scale<kNv>(a[h], g);
      const int c = c0 + h;
      uint8_t* out = stage + c * kStagePitch + rb * (kBlk / 2);
#pragma unroll
      for (int q = 0; q < kBlk / 16; ++q) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[h][16 * q + i]);
        *reinterpret_cast<uint2*>(out + 8 * q) = make_uint2(codes8<kNv>(v, bs), codes8<kNv>(v + 8, bs));
      }
      // NV: the atom's four blocks; MX: two of them, [c % 32][c / 32][block]
      sc_r[(c & 31) * (kNv ? 16 : 8) + (c >> 5) * (kNv ? 4 : 2) + rb] = static_cast<uint8_t>(bs.byte);
    }
  }
  __syncthreads();
  {
    const int c = t >> 2, q = t & 3;
    const int64_t byte = static_cast<int64_t>(row0) / 2 + q * 8;
    uint8_t* out = it.r.data + static_cast<int64_t>(col0 + c) * it.r.pitch + byte;
#pragma unroll
    for (int k = 0; k < kTile * 4 / kThreads; ++k)
      if (inside || (col0 + c + k * (kThreads / 4) < it.cols && byte < it.r.pitch))
        *reinterpret_cast<uint2*>(out + static_cast<int64_t>(k * (kThreads / 4)) * it.r.pitch) =
            *reinterpret_cast<const uint2*>(stage + (c + k * (kThreads / 4)) * kStagePitch + q * 8);
  }
  if (kNv) {
    if (t < 32 && ty < it.r.atoms)
      reinterpret_cast<uint4*>(it.r.scales + (static_cast<int64_t>(tx) * it.r.atoms + ty) * kAtomBytes)[t] =
          reinterpret_cast<const uint4*>(sc_r)[t];
  } else if (t < 128) {
    *reinterpret_cast<unsigned short*>(it.r.scales + (static_cast<int64_t>(tx) * it.r.atoms + (ty >> 1)) * kAtomBytes +
                                       t * 4 + half * 2) = reinterpret_cast<const unsigned short*>(sc_r)[t];
  }
}


struct Launch {
  const Item* one;         // a single matrix, or
  const Item* items;       // a list
  const TileRef* tiles;
  dim3 grid;
  int dtype, format;
  bool cols, rows, vec;    // vec: every source's rows start on 16-byte boundaries
  bool after_amax() const { return format == MUON_FP4_NV && !(one && one->amax == nullptr); }
};

template <typename T, bool kNv, bool kCols, bool kRows>
cudaError_t launch_quant_t(const Launch& l, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = l.grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (kRows || !l.vec ? kTileR * Src<T>::kPitch : 0) + (kRows ? kTile * kStagePitch : 0);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = l.after_amax() ? 1 : 0;
  const Item* none = nullptr;
  const TileRef* no_tiles = nullptr;
  if (l.one) return cudaLaunchKernelEx(&cfg, quant_kernel<T, kNv, kCols, kRows, false>, *l.one, none, no_tiles);
  return cudaLaunchKernelEx(&cfg, quant_kernel<T, kNv, kCols, kRows, true>, Item{}, l.items, l.tiles);
}

template <typename T, bool kNv>
cudaError_t launch_quant_n(const Launch& l, cudaStream_t st) {
  if (l.after_amax()) {
    if (l.one) amax_kernel<T, false><<<l.grid, kThreads, 0, st>>>(*l.one, nullptr, nullptr);
    else amax_kernel<T, true><<<l.grid, kThreads, 0, st>>>(Item{}, l.items, l.tiles);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (l.cols && l.rows) return launch_quant_t<T, kNv, true, true>(l, st);
  if (l.cols) return launch_quant_t<T, kNv, true, false>(l, st);
  return launch_quant_t<T, kNv, false, true>(l, st);
}

cudaError_t launch_quant(const Launch& l, cudaStream_t st) {
  const bool nv = l.format == MUON_FP4_NV;
  if (l.dtype == MUON_DT_BF16) return nv ? launch_quant_n<__nv_bfloat16, true>(l, st) : launch_quant_n<__nv_bfloat16, false>(l, st);
  return nv ? launch_quant_n<float, true>(l, st) : launch_quant_n<float, false>(l, st);
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
  uint32_t units;  // of a row: ceil(k / 16), or a head and ceil(k / 8)
  uint32_t magic;  // ceil(2^32 / units): the quotient of a small number by `units` is the high word of a product
};

constexpr int kDeqChunk = 1024;  // units per CTA

struct DeqRef {
  int32_t item;
  int32_t pad;
  int64_t first;  // first unit of the CTA
};

// The CTA's unit e of a matrix, as (row, unit of the row): first_unit + e =
// dr units + unit with e < 2^11, so the rounded-up reciprocal is off by at most one.
__device__ __forceinline__ void place(const Deq& it, int64_t first_row, uint32_t first_unit, int e, int64_t& row, int& unit) {
  const uint32_t lin = first_unit + static_cast<uint32_t>(e);
  uint32_t dr = it.units == 1u ? lin : __umulhi(lin, it.magic);
  if (dr * it.units > lin) --dr;
  unit = static_cast<int>(lin - dr * it.units);
  row = first_row + dr;
}

// Eight values from `out` on, the first `len` of them.
template <typename T>
__device__ __forceinline__ void store_values(T* out, const float* v, int len) {
  if (len >= 8) {
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
      if (i < len) {
        if (sizeof(T) == 4) reinterpret_cast<float*>(out)[i] = v[i];
        else reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v[i]);
      }
  }
}

// Rows of the destination on 16-byte boundaries: a unit is 16 values, within one block.
template <typename T, bool kNv, bool kList>
__global__ void __launch_bounds__(kThreads) dequant_kernel(const __grid_constant__ Deq one, const Deq* __restrict__ items,
                                                           const DeqRef* __restrict__ refs) {
  DeqRef ref{0, 0, static_cast<int64_t>(blockIdx.x) * kDeqChunk};
  Deq listed;
  if constexpr (kList) {
    ref = refs[blockIdx.x];
    listed = items[ref.item];
  }
  const Deq& it = kList ? listed : one;
  const int64_t left = static_cast<int64_t>(it.rows) * it.units - ref.first;
  const int n = static_cast<int>(left < kDeqChunk ? left : kDeqChunk);
  const float g = kNv ? it.ts[0] : 1.0f;
  const int64_t first_row = ref.first / it.units;
  const uint32_t first_unit = static_cast<uint32_t>(ref.first - first_row * it.units);
#pragma unroll 4
  for (int e = threadIdx.x; e < n; e += kThreads) {
    int64_t row;
    int unit;
    place(it, first_row, first_unit, e, row, unit);
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(it.data + row * it.pitch) + unit);
    const int b = kNv ? unit : unit >> 1;
    const uint32_t sb = __ldg(it.scales + ((row >> 7) * it.atoms + (b >> 2)) * kAtomBytes +
                              atom_byte(static_cast<int>(row & 127), b));
    const float s = kNv ? e4m3_value(sb) * g : e8m0_value(sb);
    float v[16];
    e2m1_values8(w.x, s, v);
    e2m1_values8(w.y, s, v + 8);
    T* out = static_cast<T*>(it.dst) + row * it.ld + unit * 16;
    const int len = it.k - unit * 16;
    store_values<T>(out, v, len);
    if (len > 8) store_values<T>(out + 8, v + 8, len - 8);
  }
}

// Rows of the destination that start anywhere: a row's first unit is its head
// up to a 16-byte boundary, the units after it are eight values each, stored
// as whole 16-byte pieces (codes are four bits, so any eight of them are a
// funnel shift of two words).
template <typename T, bool kNv, bool kList>
__global__ void __launch_bounds__(kThreads) dequant_any_kernel(const __grid_constant__ Deq one, const Deq* __restrict__ items,
                                                           const DeqRef* __restrict__ refs) {
  DeqRef ref{0, 0, static_cast<int64_t>(blockIdx.x) * kDeqChunk};
  Deq listed;
  if constexpr (kList) {
    ref = refs[blockIdx.x];
    listed = items[ref.item];
  }
  const Deq& it = kList ? listed : one;
  const int64_t left = static_cast<int64_t>(it.rows) * it.units - ref.first;
  const int n = static_cast<int>(left < kDeqChunk ? left : kDeqChunk);
  const float g = kNv ? it.ts[0] : 1.0f;
  // the CTA's first unit by one wide division, the rest relative to it
  const int64_t first_row = ref.first / it.units;
  const uint32_t first_unit = static_cast<uint32_t>(ref.first - first_row * it.units);
#pragma unroll 4
  for (int e = threadIdx.x; e < n; e += kThreads) {
    int64_t row;
    int unit;
    place(it, first_row, first_unit, e, row, unit);
    T* dst = static_cast<T*>(it.dst) + row * it.ld;
    int k0, len;
    const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / static_cast<int>(sizeof(T));
    k0 = unit == 0 ? 0 : head + (unit - 1) * 8;
    len = unit == 0 ? head : 8;
    len = min(len, it.k - k0);
    if (len <= 0) continue;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(it.data + row * it.pitch);
    const int wi = k0 >> 3, sh = (k0 & 7) * 4;
    uint32_t w = __ldg(codes + wi);
    if (sh != 0) w = __funnelshift_r(w, (wi + 1) * 4 < it.pitch ? __ldg(codes + wi + 1) : 0u, sh);
    const uint8_t* srow = it.scales + (row >> 7) * it.atoms * kAtomBytes + atom_byte(static_cast<int>(row & 127), 0);
    const int b0 = k0 / (kNv ? 16 : 32), b1 = (k0 + len - 1) / (kNv ? 16 : 32);
    auto scale = [&](int b) {
      const uint32_t sb = __ldg(srow + static_cast<int64_t>(b >> 2) * kAtomBytes + (b & 3));
      return kNv ? e4m3_value(sb) * g : e8m0_value(sb);
    };
    const float s0 = scale(b0);
    const float s1 = b1 != b0 ? scale(b1) : s0;
    const int turn = b1 * (kNv ? 16 : 32) - k0;  // values from here on are the next block's
    float v[8];
    e2m1_values8(w, 1.0f, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= i < turn ? s0 : s1;
    store_values<T>(dst + k0, v, len);
  }
}

template <typename T, bool kNv>
cudaError_t launch_dequant_t(const Deq& one, const Deq* items, const DeqRef* refs, int64_t nblocks, bool vec,
                             cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(nblocks));
  if (items != nullptr) {
    if (vec) dequant_kernel<T, kNv, true><<<grid, kThreads, 0, st>>>(one, items, refs);
    else dequant_any_kernel<T, kNv, true><<<grid, kThreads, 0, st>>>(one, items, refs);
  } else {
    if (vec) dequant_kernel<T, kNv, false><<<grid, kThreads, 0, st>>>(one, items, refs);
    else dequant_any_kernel<T, kNv, false><<<grid, kThreads, 0, st>>>(one, items, refs);
  }
  return cudaGetLastError();
}

cudaError_t launch_dequant(const Deq& one, const Deq* items, const DeqRef* refs, int64_t nblocks, int dtype, int format,
                           bool vec, cudaStream_t st) {
  const bool nv = format == MUON_FP4_NV;
  if (dtype == MUON_DT_BF16)
    return nv ? launch_dequant_t<__nv_bfloat16, true>(one, items, refs, nblocks, vec, st)
              : launch_dequant_t<__nv_bfloat16, false>(one, items, refs, nblocks, vec, st);
  return nv ? launch_dequant_t<float, true>(one, items, refs, nblocks, vec, st)
            : launch_dequant_t<float, false>(one, items, refs, nblocks, vec, st);
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
  const int64_t tx = (s.cols + kTile - 1) / kTile, ty = (s.rows + kAtomRows - 1) / kAtomRows * (kAtomRows / kTileR);
  if (tx * ty > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
  it = Item{};
  it.src = s.src;
  it.ld = s.ld;
  it.rows = static_cast<int32_t>(s.rows);
  it.cols = static_cast<int32_t>(s.cols);
  it.tiles_x = static_cast<int32_t>(tx);
  it.tiles_y = static_cast<int32_t>(ty);
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

int tiles_of(const Item& it) { return it.tiles_x * it.tiles_y; }

template <class List>
void item_ranges(const muon_fp4_source_t& s, List& reads, List& writes) {
  reads.push_back(matrix_range(s.src, s.rows, s.cols, s.ld, s.src_dtype));
  if (s.along_cols.format >= 0) add_ranges(s.along_cols, writes);
  if (s.along_rows.format >= 0) add_ranges(s.along_rows, writes);
}

// destination rows start on 16-byte boundaries
bool deq_vec(const void* dst, int64_t ld, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(dst) % 16 == 0 && ld * size_of(dtype) % 16 == 0;
}

muon_status_t make_deq(const muon_fp4_matrix_t& m, void* dst, int64_t ld, int32_t dtype, bool vec, Deq& d) {
  if (dst == nullptr || ld < m.k || ld > (int64_t(1) << 40)) return MUON_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(dst);
  if (a % size_of(dtype) != 0) return MUON_ERR_INVALID_ARG;
  const uint32_t units = vec ? static_cast<uint32_t>((m.k + 15) / 16) : static_cast<uint32_t>((m.k + 7) / 8) + 1u;
  d = Deq{static_cast<const uint8_t*>(m.data), static_cast<const uint8_t*>(m.scales), m.tensor_scale, dst, ld,
          pitch_of(m.k), atoms_of(m.format, m.k), static_cast<int32_t>(m.rows), static_cast<int32_t>(m.k), units,
          static_cast<uint32_t>(((uint64_t(1) << 32) + units - 1) / units)};
  return MUON_OK;
}

int64_t deq_blocks(const Deq& d) {
  return (static_cast<int64_t>(d.rows) * d.units + kDeqChunk - 1) / kDeqChunk;
}

}  // namespace

struct muon_fp4_plan_s {
  int device = 0;
  int dtype = 0, format = 0, values_dtype = -1;
  bool cols = false, rows = false, vec = true;
  int nitems = 0, ntiles = 0;
  int64_t ndeq = 0, ndeq_vec = 0;
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
  if (format == MUON_FP4_NV && src->rows * src->cols > kSmall) {
    it.amax = reinterpret_cast<unsigned*>((c ? it.c.ts : it.r.ts) + 1);
    if (cudaMemsetAsync(it.amax, 0, sizeof(unsigned), st) != cudaSuccess) {
      cudaGetLastError();
      return MUON_ERR_CUDA;
    }
  }
  const unsigned gy = it.tiles_y < kGridY ? it.tiles_y : kGridY;
  const Launch l{&it, nullptr, nullptr, dim3(it.tiles_x, gy, (it.tiles_y + kGridY - 1) / kGridY), src->src_dtype, format,
                 c, r, it.vec != 0};
  return launch_quant(l, st) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

muon_status_t muon_fp4_dequantize(const muon_fp4_matrix_t* m, void* dst, int64_t ld, int32_t dst_dtype, void* stream) {
  if (m == nullptr || !valid(*m) || !valid_dtype(dst_dtype)) return MUON_ERR_INVALID_ARG;
  if (m->rows == 0 || m->k == 0) return MUON_OK;
  Deq d;
  const bool vec = deq_vec(dst, ld, dst_dtype);
  const muon_status_t s = make_deq(*m, dst, ld, dst_dtype, vec, d);
  if (s != MUON_OK) return s;
  RangeList reads, writes;
  writes.push_back(matrix_range(dst, m->rows, m->k, ld, dst_dtype));
  add_ranges(*m, reads);
  if (conflict(reads, writes)) return MUON_ERR_ALIAS;
  const int64_t nb = deq_blocks(d);
  if (nb > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
  return launch_dequant(d, nullptr, nullptr, nb, dst_dtype, m->format, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
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
    std::vector<DeqRef> refs;      // vector kernel first, then the others
    std::vector<DeqRef> refs_any;
    std::vector<ByteRange> reads, writes;
    bool vec = true;
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
      vec = vec && it.vec;
      for (int k = 0; k < nt; ++k) tiles.push_back(TileRef{id, k % it.tiles_x, k / it.tiles_x});
      if (values_dtype >= 0)
        for (int f = 0; f < 2; ++f) {
          if (f == 0 ? !c : !r) continue;
          const muon_fp4_matrix_t& m = f == 0 ? s.along_cols : s.along_rows;
          void* dst = f == 0 ? s.values_cols : s.values_rows;
          if (dst == nullptr) return MUON_ERR_INVALID_ARG;
          Deq d;
          const bool dv = deq_vec(dst, m.k, values_dtype);
          const muon_status_t e2 = make_deq(m, dst, m.k, values_dtype, dv, d);
          if (e2 != MUON_OK) return e2;
          writes.push_back(matrix_range(dst, m.rows, m.k, m.k, values_dtype));
          const int32_t did = static_cast<int32_t>(deqs.size());
          deqs.push_back(d);
          for (int64_t b = 0; b < deq_blocks(d); ++b) (dv ? refs : refs_any).push_back(DeqRef{did, 0, b * kDeqChunk});
        }
    }
    if (conflict(reads, writes)) return MUON_ERR_ALIAS;
    const int64_t ndeq_vec = static_cast<int64_t>(refs.size());
    refs.insert(refs.end(), refs_any.begin(), refs_any.end());
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
    pl->vec = vec;
    pl->ntiles = static_cast<int>(tiles.size());
    pl->ndeq = static_cast<int64_t>(refs.size());
    pl->ndeq_vec = ndeq_vec;
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
          !put(pl->refs_d, refs.data(), refs.size() * sizeof(DeqRef)) || !uploads_done()) {
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
  const Launch l{nullptr, pl->items_d, pl->tiles_d, dim3(pl->ntiles), pl->dtype, pl->format, pl->cols, pl->rows, pl->vec};
  return launch_quant(l, st) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

muon_status_t muon_fp4_values(muon_fp4_plan_t pl, void* stream) {
  if (pl == nullptr || pl->values_dtype < 0) return MUON_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pl->device) return MUON_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  pl->last_stream = st;
  cudaError_t e = cudaSuccess;
  if (pl->ndeq_vec > 0)
    e = launch_dequant(Deq{}, pl->deqs_d, pl->refs_d, pl->ndeq_vec, pl->values_dtype, pl->format, true, st);
  if (e == cudaSuccess && pl->ndeq > pl->ndeq_vec)
    e = launch_dequant(Deq{}, pl->deqs_d, pl->refs_d + pl->ndeq_vec, pl->ndeq - pl->ndeq_vec, pl->values_dtype,
                       pl->format, false, st);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

void muon_fp4_destroy(muon_fp4_plan_t pl) {
  if (pl == nullptr) return;
  cudaStreamSynchronize(pl->last_stream);
  cudaGetLastError();
  cudaFree(pl->dmem);
  delete pl;
}

}  // extern "C"
