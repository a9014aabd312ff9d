// The 4-bit matrix format shared by the quantisation, product and few-row
// kernels (declared in muon.h, muon_fp4_matrix_t).
//
// A row holds k values in blocks along k: e2m1 codes (bit 3 the sign, bits
// 2..1 the exponent, bit 0 the mantissa) times their block's scale.
//   MUON_FP4_MX  blocks of 32, scale 2^(byte - 127) (e8m0, 255 = NaN)
//   MUON_FP4_NV  blocks of 16, scale e4m3(byte) * g, g one power of two per matrix
// Codes are packed two a byte, lower k in the low four bits, rows at a pitch of
// 16 ceil(k / 32) bytes (a TMA stride).  Scale bytes lie in atoms of 512
// bytes, one for 128 rows x 4 blocks, so that an atom is one row-block's
// share of a K step in the order in which the tensor core's scale memory takes
// it: lane r % 32, 32-bit column r % 128 / 32, byte b % 4.
#pragma once

#include "muon.h"
#include "muon_internal.cuh"

#include <atomic>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace muon {
namespace fp4 {

constexpr int kAtomBytes = 512;
constexpr int kAtomRows = 128;
constexpr int64_t kMaxDim = int64_t(1) << 30;  // rows and k of one matrix

__host__ __device__ constexpr int block_of(int format) { return format == MUON_FP4_NV ? 16 : 32; }
__host__ __device__ constexpr int atom_k_of(int format) { return 4 * block_of(format); }
__host__ __device__ inline int64_t pitch_of(int64_t k) { return (k + 31) / 32 * 16; }
__host__ __device__ inline int64_t atoms_of(int format, int64_t k) {
  return (k + atom_k_of(format) - 1) / atom_k_of(format);
}
inline int64_t row_blocks_of(int64_t rows) { return (rows + kAtomRows - 1) / kAtomRows; }
inline size_t data_bytes_of(int64_t rows, int64_t k) { return static_cast<size_t>(rows) * pitch_of(k); }
inline size_t scale_bytes_of(int format, int64_t rows, int64_t k) {
  return static_cast<size_t>(row_blocks_of(rows)) * atoms_of(format, k) * kAtomBytes;
}

// Host: the fields of a descriptor are usable (sizes, format, pointers and
// their alignment; a matrix without elements needs no pointers).
inline bool valid(const muon_fp4_matrix_t& m) {
  if (m.format != MUON_FP4_MX && m.format != MUON_FP4_NV) return false;
  if (m.rows < 0 || m.k < 0 || m.rows > kMaxDim || m.k > kMaxDim || m.reserved != 0) return false;
  if (m.rows == 0 || m.k == 0) return true;
  if (m.data == nullptr || m.scales == nullptr) return false;
  if (m.format == MUON_FP4_NV && m.tensor_scale == nullptr) return false;
  return reinterpret_cast<uintptr_t>(m.data) % 16 == 0 && reinterpret_cast<uintptr_t>(m.scales) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(m.tensor_scale) % 4 == 0;
}

// A few byte ranges without an allocation (single-matrix calls); the list
// calls use std::vector.
struct RangeList {
  ByteRange v[12];
  int n = 0;
  void push_back(const ByteRange& r) { v[n++] = r; }
};

template <class List>
inline void add_ranges(const muon_fp4_matrix_t& m, List& v) {
  if (m.rows == 0 || m.k == 0) return;
  const uintptr_t d = reinterpret_cast<uintptr_t>(m.data), s = reinterpret_cast<uintptr_t>(m.scales);
  v.push_back(ByteRange{d, d + data_bytes_of(m.rows, m.k)});
  v.push_back(ByteRange{s, s + scale_bytes_of(m.format, m.rows, m.k)});
  if (m.format == MUON_FP4_NV) {
    const uintptr_t t = reinterpret_cast<uintptr_t>(m.tensor_scale);
    v.push_back(ByteRange{t, t + 2 * sizeof(float)});
  }
}

// true if two of `writes` meet, or one of `reads` meets one of them
inline bool conflict(const RangeList& reads, const RangeList& writes) {
  auto meet = [](const ByteRange& x, const ByteRange& y) { return x.lo < y.hi && y.lo < x.hi; };
  for (int i = 0; i < writes.n; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(writes.v[i], writes.v[j])) return true;
    for (int j = 0; j < reads.n; ++j)
      if (meet(writes.v[i], reads.v[j])) return true;
  }
  return false;
}

// the same over lists (sorts writes)
inline bool conflict(const std::vector<ByteRange>& reads, std::vector<ByteRange>& writes) {
  if (any_overlap(writes)) return true;
  for (const ByteRange& r : reads) {
    auto it = std::upper_bound(writes.begin(), writes.end(), r.lo,
                               [](uintptr_t v, const ByteRange& x) { return v < x.lo; });
    if (it != writes.end() && it->lo < r.hi) return true;
    if (it != writes.begin() && (it - 1)->hi > r.lo) return true;
  }
  return false;
}

// Host: SMs of an sm_100 device, 0 for another; read once for all devices, so
// the calls that follow touch no device state.
inline int device_sms(int dev) {
  static const struct All {
    int sms[64];
    All() {
      int n = 0;
      if (cudaGetDeviceCount(&n) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      for (int i = 0; i < 64; ++i) {
        sms[i] = 0;
        int major = 0, count = 0;
        if (i < n && cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, i) == cudaSuccess && major == 10 &&
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, i) == cudaSuccess)
          sms[i] = count;
      }
    }
  } all;
  return dev >= 0 && dev < 64 ? all.sms[dev] : 0;
}

// Host: let `kernel` use up to `bytes` of dynamic shared memory on device
// `dev`; set once per kernel and device.
template <auto kKernel>
inline cudaError_t allow_smem(int dev, int bytes) {
  static std::atomic<uint64_t> done{0};  // one bit per device
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Byte of row r, block b within its atom.
__host__ __device__ __forceinline__ int atom_byte(int r, int b) {
  return (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3);
}

__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  // 2^(byte - 127): byte 0 is the subnormal 2^-127, byte 255 NaN
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : byte == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// v as m 2^e with 1 <= |m| < 2, subnormals too (v itself and e = 0 for zeros and what is not finite).
__device__ __forceinline__ float significand(float v, int& e) {
  const bool below = fabsf(v) < pow2(-126), plain = v == 0.0f || !(fabsf(v) < __uint_as_float(0x7F800000u));
  const uint32_t b = __float_as_uint(below ? v * pow2(64) : v);
  e = plain ? 0 : static_cast<int>((b >> 23) & 255u) - (below ? 127 + 64 : 127);
  return plain ? v : __uint_as_float((b & 0x807FFFFFu) | 0x3F800000u);
}

// Eight codes (lowest four bits first) as four fp16 pairs.
__device__ __forceinline__ void e2m1_expand8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight codes as their values times s.
__device__ __forceinline__ void e2m1_values8(uint32_t w, float s, float* v) {
  uint32_t h[4];
  e2m1_expand8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = p.x * s;
    v[2 * i + 1] = p.y * s;
  }
}

// The matrix's power of two: the least g = 2^e, e >= -100, with amax <= 2688 g,
// so that the largest block scale amax / (6 g) is at most 448, e4m3's largest.
// 2688 = 1.3125 * 2^11, so e follows from the bits of amax (a finite fp32).
// The floor keeps the least scales, their quotients and remainders below normal.
__host__ __device__ __forceinline__ int tensor_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127 - 11 + ((amax_bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return e < -100 ? -100 : e;
}

// Scale of one block from the bits of its largest magnitude (anything at or
// above the bits of infinity says that the block holds a NaN or an infinity;
// the codes of such a block do not matter, but for those past k).
struct BlockScale {
  uint32_t byte;       // the scale byte
  uint64_t r, r_rest;  // the scale's reciprocal as a pair of equal floats: MX r alone, exact; NV rounded down,
                       // and what is left of it (both 0 for a zero scale and a NaN, so that the zeros past k are code 0)
};

// A matrix's scale and what its blocks' scales are found with.
struct MatrixScale {
  float g, six, sixth;  // g, 6 g and its reciprocal
};

__device__ __forceinline__ MatrixScale matrix_scale(uint32_t amax_bits) {
  MatrixScale m;
  m.g = __uint_as_float(static_cast<uint32_t>(tensor_exponent(amax_bits) + 127) << 23);
  m.six = 6.0f * m.g;
  m.sixth = __frcp_rn(m.six);
  return m;
}

__device__ __forceinline__ float rcp_approx(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

__device__ __forceinline__ uint64_t twice(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}

template <bool kNv>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, const MatrixScale& m) {
  BlockScale b;
  if (kNv) {
    // amax / (6 g), the product with the reciprocal corrected once by its
    // remainder (Markstein's division), is rounded twice, to fp32 and then to e4m3, with the result
    // of one rounding: a quotient by 6 g (significand 1.5) that is not itself
    // a midpoint of e4m3 (5 significant bits) lies more than half an fp32
    // step from every midpoint.
    const float x = __uint_as_float(amax_bits), q = x * m.sixth;
    b.byte = __nv_cvt_float_to_fp8(fmaf(-fmaf(q, m.six, -x), m.sixth, q), __NV_SATFINITE, __NV_E4M3);
    if (amax_bits >= 0x7F800000u) b.byte = 0x7Fu;
    // 1 / d as r + rest, r rounded down so that neither is negative: one
    // Newton-Raphson step on the approximate reciprocal, and its remainder
    const float d = e4m3_value(b.byte) * m.g;  // exact: four significant bits; below 2^126
    const float a = rcp_approx(d);
    const float r = __fmaf_rd(fmaf(-d, a, 1.0f), a, a);
    const float rest = fmaf(-d, r, 1.0f) * r;
    const bool some = b.byte != 0u && b.byte != 0x7Fu;
    b.r = some ? twice(r) : 0u;
    b.r_rest = some ? twice(rest) : 0u;
  } else {
    const int e = static_cast<int>(amax_bits >> 23) - 2;
    b.byte = e < 0 ? 0u : static_cast<uint32_t>(e);
    b.r = twice(__uint_as_float((254u - b.byte) << 23));
    b.r_rest = 0u;
    if (amax_bits >= 0x7F800000u) b.byte = 255u;
  }
  return b;
}

// Two values divided by their block's scale.  MX: the product with a power of
// two is exact.  NV: x r + x rest, one rounding of the quotient to within
// 2^-46 of it, which is exact where the quotient has few bits and else on the
// right side of every border: a quotient by a four-bit scale that is no
// midpoint of e2m1 (three significant bits) is more than half an fp32 step
// from every midpoint.  From scales of about 2^102 on `rest` is subnormal and
// the pair is good to fewer bits, 2^-25 at 2^125; the codes are still right at
// every midpoint and both its neighbours, by exact arithmetic over all scale
// bytes and the highest g, but for the scale 448 under g = 2^117, and there
// the largest finite amax is 342 times 6 g, a scale of 352 at most.  A zero
// keeps its sign, since r and rest are not negative.  Both lanes in one
// instruction each (f32x2).
template <bool kNv>
__device__ __forceinline__ uint64_t quotients(float x0, float x1, const BlockScale& b) {
  uint64_t x, q;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  if (kNv) {
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(b.r_rest));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(x), "l"(b.r), "l"(q));
  } else {
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(b.r));
  }
  return q;
}

// Eight values to eight codes, v[0] in the lowest four bits: quotients rounded
// to nearest, ties to the even code, saturating at 6.
template <bool kNv>
__device__ __forceinline__ uint32_t codes8(const float* v, const BlockScale& b) {
  uint64_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = quotients<kNv>(v[2 * i], v[2 * i + 1], b);
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .f32 x, y;\n\t"
      "mov.b64 {x, y}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, y, x;\n\t"
      "mov.b64 {x, y}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, y, x;\n\t"
      "mov.b64 {x, y}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, y, x;\n\t"
      "mov.b64 {x, y}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, y, x;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "l"(q[0]), "l"(q[1]), "l"(q[2]), "l"(q[3]));
  return w;
}

}  // namespace fp4
}  // namespace muon
