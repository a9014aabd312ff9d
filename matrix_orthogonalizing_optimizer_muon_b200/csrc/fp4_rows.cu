// Product of a few bf16 rows with a 4-bit matrix, out[t, n] = X W^T (format:
// fp4.cuh): the form for single tokens, bound by reading W once.
#include "fp4.cuh"

namespace {

using namespace muon;
using namespace muon::fp4;

constexpr int kThreadsR = 256;
constexpr int kGroup = 8;  // rows of X per pass over W

struct RowsArgs {
  const __nv_bfloat16* x;
  const uint8_t* data;
  const uint8_t* scales;
  const float* ts;
  void* out;
  int64_t ldx, ldo, pitch, atoms;
  int32_t t, n, k, out_dtype;
};

template <bool kNv>
__global__ void __launch_bounds__(kThreadsR) fp4_rows_kernel(const RowsArgs g) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreadsR / 32) + (threadIdx.x >> 5);
  if (row >= g.n) return;
  const float ts = kNv ? *g.ts : 1.0f;
  const uint8_t* codes = g.data + row * g.pitch;
  const uint8_t* scales = g.scales + (row >> 7) * g.atoms * kAtomBytes;
  for (int t0 = 0; t0 < g.t; t0 += kGroup) {
    float acc[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) acc[i] = 0.0f;
    for (int k0 = lane * 8; k0 < g.k; k0 += 256) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + k0 / 2));
      const int b = k0 / (kNv ? 16 : 32);
      const uint32_t sb = __ldg(scales + static_cast<int64_t>(b >> 2) * kAtomBytes + atom_byte(static_cast<int>(row & 127), b));
      const float s = kNv ? e4m3_value(sb) : e8m0_value(sb);
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = e2m1_pair((w >> (8 * i)) & 0xFFu);
        v[2 * i] = p.x * s;
        v[2 * i + 1] = p.y * s;
      }
#pragma unroll
      for (int t = 0; t < kGroup; ++t) {
        if (t0 + t >= g.t) continue;
        const __nv_bfloat16* x = g.x + (t0 + t) * g.ldx + k0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k0 + i < g.k) acc[t] = fmaf(__bfloat162float(x[i]), v[i], acc[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < kGroup; ++t) {
      float a = acc[t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      if (lane == 0 && t0 + t < g.t) {
        a *= ts;
        const int64_t at = (t0 + t) * g.ldo + row;
        if (g.out_dtype == MUON_DT_BF16) static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(a);
        else static_cast<float*>(g.out)[at] = a;
      }
    }
  }
}

}  // namespace

extern "C" muon_status_t muon_fp4_rows_product(const void* x, int64_t t, int64_t ldx, const muon_fp4_matrix_t* w,
                                               void* out, int64_t ldo, int32_t out_dtype, void* stream) {
  if (w == nullptr || !valid(*w) || t < 0 || t > MUON_FP4_MAX_ROWS) return MUON_ERR_INVALID_ARG;
  if (out_dtype != MUON_DT_BF16 && out_dtype != MUON_DT_FP32) return MUON_ERR_INVALID_ARG;
  if (t == 0 || w->rows == 0) return MUON_OK;
  const int es = out_dtype == MUON_DT_BF16 ? 2 : 4;
  const uintptr_t o = reinterpret_cast<uintptr_t>(out);
  if (out == nullptr || o % es != 0 || ldo < w->rows || ldo > (int64_t(1) << 40)) return MUON_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (w->k == 0)
    return cudaMemset2DAsync(out, static_cast<size_t>(ldo) * es, 0, static_cast<size_t>(w->rows) * es,
                             static_cast<size_t>(t), st) == cudaSuccess
               ? MUON_OK
               : MUON_ERR_CUDA;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x);
  if (x == nullptr || xa % 2 != 0 || ldx < w->k || ldx > (int64_t(1) << 40)) return MUON_ERR_INVALID_ARG;
  RangeList reads, writes;
  add_ranges(*w, reads);
  reads.push_back(ByteRange{xa, xa + (static_cast<size_t>(t - 1) * ldx + w->k) * 2});
  writes.push_back(ByteRange{o, o + (static_cast<size_t>(t - 1) * ldo + w->rows) * es});
  if (conflict(reads, writes)) return MUON_ERR_ALIAS;
  RowsArgs g{static_cast<const __nv_bfloat16*>(x), static_cast<const uint8_t*>(w->data),
             static_cast<const uint8_t*>(w->scales), w->tensor_scale, out, ldx, ldo, pitch_of(w->k),
             atoms_of(w->format, w->k), static_cast<int32_t>(t), static_cast<int32_t>(w->rows),
             static_cast<int32_t>(w->k), out_dtype};
  const unsigned blocks = static_cast<unsigned>((w->rows + kThreadsR / 32 - 1) / (kThreadsR / 32));
  if (w->format == MUON_FP4_NV) fp4_rows_kernel<true><<<blocks, kThreadsR, 0, st>>>(g);
  else fp4_rows_kernel<false><<<blocks, kThreadsR, 0, st>>>(g);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
