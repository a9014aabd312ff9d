// Product of a few bf16 rows with a 4-bit matrix, out[t, n] = X W^T (format:
// fp4.cuh): the form for single tokens.
//
// The bound is reading W once: 0.56 (NV) or 0.53 (MX) bytes a value, so per
// SM about 44 values must be expanded and multiplied a cycle.  Multiplying on
// the CUDA cores costs an instruction per value and row of X; here 16 rows of
// W meet 8 rows of X in one mma.sync m16n8k16, whose cost does not grow with
// the rows up to 8.  (tcgen05 has no kind that takes 4-bit and 16-bit
// operands, and needs both in shared memory.)
//
//   W  goes to shared memory by cp.async, in steps of 128 k of a warp's 16
//      rows, kDepth - 1 steps ahead (with plain loads into registers, which
//      the compiler moved down to their use, 65536 x 2048 had taken 36 us where
//      the first such ring took 25).  A code becomes an fp16 by one conversion for two.
//      NV: times the block's scale, exactly (e2m1 x e4m3 has at most six
//      significant bits within fp16's range).  MX: the exponent of a scale may
//      be outside fp16's range, so the products of a block are summed from
//      zero (its 32 values are exactly two MMAs) and scaled in fp32, times
//      2^30: a sum of 10240 products then neither overflows for scales below
//      2^65 nor loses a bit for the least, whatever power of two X's row is to
//      be given back.  Blocks with larger scales are summed apart, times 2^-31.
//   X  is held in shared memory as fp16, each row times its own power of two
//      that puts its largest magnitude into [2^14, 2^15); the power is undone
//      at the end, so a row's result does not depend on the other rows.  A bf16
//      has 8 significant bits and an fp16 goes down to 2^-24, so the values
//      within 32 exponents of the largest are exact.  A CTA that finds one
//      below (an output whose codes are zero under the larger values is made
//      of such alone) takes X in parts instead, 32 exponents each with a power
//      of two of its own, and multiplies W by one part after the other: eight
//      cover all of bf16.  (bf16 operands would need no powers of two, but a
//      code becomes a bf16 in about five instructions a pair instead of two,
//      in a kernel that its instructions bound.)
// Sums are fp32 in a fixed order.  KS warps split the k of a row tile where
// there are too few row tiles to fill the GPU, and add up through shared
// memory.
#include "fp4.cuh"

namespace {

using namespace muon;
using namespace muon::fp4;

constexpr int kStepK = 128;          // k of a step: 32 codes a thread
constexpr int kDepth = 4;            // ring of steps of a warp
constexpr int kStepBytes = 1024 + 128;  // codes of 16 rows, then 8 bytes of scales a row
constexpr int kMaxK = 10240;         // k of X in shared memory at a time
constexpr int kXBudget = 164 * 1024; // bytes of it
constexpr int kSmemMax = 226 * 1024;
constexpr int kWindowLog = 5, kWindow = 1 << kWindowLog;  // exponents of X that one fp16 copy holds exactly
constexpr int kMxBig = 192;          // MX scale bytes from here on (2^65) are summed apart
constexpr int kMxUp = 30, kMxDown = 31;  // scales are taken times 2^30, the big ones times 2^-31

struct RowsArgs {
  const __nv_bfloat16* x;
  const uint8_t* data;
  const uint8_t* scales;
  const float* ts;
  void* out;
  int64_t ldx, ldo, pitch, atoms;
  int32_t t, n, k, out_dtype;
  int32_t ks, kc, xpitch, tg;  // k split, k per pass, bytes of a row of X in shared memory, rows of X per CTA
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same from zero
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four 8 x 16-byte matrices whose rows lie one after another: word t4 of row gr of each.
__device__ __forceinline__ void load_words(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bit 7 of every byte of four e8m0 scales that is kMxBig or more.
__device__ __forceinline__ uint32_t mx_big(uint32_t w) { return w & (w << 1) & 0x80808080u; }
// The four scales as the exponent fields that they are taken with, kMxUp above
// their own (a byte 0 is 2^-127, so this holds for all); none may be big, or a
// big one counts as 0.
__device__ __forceinline__ uint32_t mx_up(uint32_t w) { return w + kMxUp * 0x01010101u; }
__device__ __forceinline__ uint32_t mx_up_mixed(uint32_t w) {
  uint32_t r = 0u;
#pragma unroll
  for (int b = 0; b < 32; b += 8) {
    const uint32_t byte = (w >> b) & 255u;
    if (byte < kMxBig) r |= (byte + kMxUp) << b;
  }
  return r;
}
// Scale b of them.
__device__ __forceinline__ float mx_scale(uint32_t up, int b) {
  return __uint_as_float((b < 3 ? up << (23 - 8 * b) : up >> 1) & 0x7F800000u);
}

// Exponent of the power of two that is taken out of part `part` of a row of X
// with the largest magnitude a (bits).  At least -126: below, the values are
// multiples of 2^-133, times 2^126 multiples of 2^-7, exact in fp16 all the same.
__device__ __forceinline__ int exponent_of(uint32_t a, int part = 0) {
  return max(static_cast<int>(a >> 23) - 127 - 14 - kWindow * part, -126);
}
// v m 2^e for e <= 254, half of e at a time: nothing passes fp32's range that
// the result does not pass.  (Below -252 the result is 0.)
__device__ __forceinline__ float times_pow2(float v, float m, int e) {
  e = max(e, -252);
  const int h = e >> 1;
  return v * (m * pow2(h)) * pow2(e - h);
}
// Exponent field of a finite magnitude (bits); subnormals count as the least normal numbers.
__device__ __forceinline__ int field_of(uint32_t a) { return max(static_cast<int>(a >> 23), 1); }

// Two magnitudes (bf16 bits) less 2^15 + 1 each, as signed halves: a zero wraps
// to the largest, so a minimum is that of the values that are not zero.
__device__ __forceinline__ uint32_t wrapped(uint32_t two) { return (two & 0x7FFF7FFFu) + 0x7FFF7FFFu; }
// The lesser half, as its bf16 bits again (2^16 for a zero).
__device__ __forceinline__ int least_half(uint32_t w) {
  return min(static_cast<int>(w) >> 16, static_cast<int>(w << 16) >> 16) + 0x8001;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  // the rest of the 16 bytes is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// true if the lesser of `least` (wrapped) lies kWindow exponents or more below a
__device__ __forceinline__ bool spread(uint32_t a, uint32_t least) {
  return field_of(a) - (least_half(least) >> 7) >= kWindow;
}

// Where 16-byte piece p of a row of X lies: within a step of 128 the pieces lie
// in the order in which the four threads of a row take them, NV thread t4's
// i-th piece (8 values of its 32) at 4 i + t4, MX in order.
template <bool kNv>
__device__ __forceinline__ int x_place(int p) {
  return (kNv ? (p & ~15) + (p & 3) * 4 + ((p >> 2) & 3) : p) * 16;
}

// fn(p, the eight values of piece p) for a lane's pieces of a row of X with kn
// values; zeros past its end.  Four pieces are on their way at a time.
template <class Fn>
__device__ __forceinline__ void each_piece(const unsigned short* src, int kn, int pieces, const Fn& fn) {
  const bool plain = ((reinterpret_cast<uintptr_t>(src) | static_cast<uintptr_t>(2 * kn)) & 15) == 0;
#pragma unroll 1
  for (int p = threadIdx.x & 31; p < pieces; p += 128) {
    uint4 q[4];
    if (plain) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        q[u] = (p + 32 * u) * 8 < kn ? __ldg(reinterpret_cast<const uint4*>(src) + p + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = (p + 32 * u) * 8 + 2 * i;
          const uint32_t lo = at < kn ? __ldg(src + at) : 0u, hi = at + 1 < kn ? __ldg(src + at + 1) : 0u;
          v[i] = lo | (hi << 16);
        }
        q[u] = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t v[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      if (p + 32 * u < pieces) fn(p + 32 * u, v);
    }
  }
}

// Stages part `part` of X of [k0, k0 + kc); finds the rows' ranges first if
// they are not known.
template <bool kNv, int kNg, int kWarps>
__device__ __noinline__ void stage_part(const RowsArgs& g, int k0, int part, bool known, int t0, int nt, uint8_t* smem,
                                           uint32_t* amax, int* nparts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kn = min(g.kc, g.k - k0);
  const int pieces = (kn + kStepK - 1) / kStepK * (kStepK / 8);
  auto row = [&](int r) {
    return reinterpret_cast<const unsigned short*>(g.x) + static_cast<int64_t>(t0 + r) * g.ldx + k0;
  };
  if (!known) {
    if (threadIdx.x == 0) *nparts = 1;
    __syncthreads();
#pragma unroll 1
    for (int r = warp; r < nt; r += kWarps) {
      uint32_t a = 0u, least = 0x7FFF7FFFu;
      each_piece(row(r), kn, pieces, [&](int, const uint32_t (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = (v[i] << 16) & 0x7FFF0000u, hi = v[i] & 0x7FFF0000u;
          a = max(a, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
          least = __vmins2(least, wrapped(v[i]));
        }
      });
      a = __reduce_max_sync(0xffffffffu, a);
      const int low = __reduce_min_sync(0xffffffffu, least_half(least));
      if (lane == 0) {
        amax[r] = a;
        // one part for a row of zeros or without a finite value
        atomicMax(nparts, ((field_of(a) - max(low >> 7, 1)) >> kWindowLog) + 1);
      }
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int r = warp; r < nt; r += kWarps) {
    // the values whose exponents are in the part, zeros for the others; an
    // infinity is in the first (no magnitude is at or above a NaN), a NaN in all
    const float f = pow2(-exponent_of(amax[r], part));
    const int top = field_of(amax[r]) - kWindow * part, bottom = top - kWindow + 1;
    const float above = part == 0 ? __uint_as_float(0x7FFFFFFFu)
                        : top > 0 ? __uint_as_float(static_cast<uint32_t>(top + 1) << 23)
                                  : 0.0f;  // the row has no such part
    const float from = bottom > 1 ? __uint_as_float(static_cast<uint32_t>(bottom) << 23) : 0.0f;
    auto in_part = [&](uint32_t v) {
      const float x = __uint_as_float(v);
      return !(fabsf(x) < from) && !(fabsf(x) >= above) ? x * f : 0.0f;
    };
    each_piece(row(r), kn, pieces, [&](int p, const uint32_t (&v)[4]) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 c = __floats2half2_rn(in_part(v[i] << 16), in_part(v[i] & 0xFFFF0000u));
        h[i] = *reinterpret_cast<const uint32_t*>(&c);
      }
      *reinterpret_cast<uint4*>(smem + r * g.xpitch + x_place<kNv>(p)) = make_uint4(h[0], h[1], h[2], h[3]);
    });
  }
}

// One lane's outputs of a row tile: rows `row` and row + 8 of W.
template <int kNg>
__device__ __forceinline__ void store_rows(const RowsArgs& g, const float (&total)[kNg][4], int row, int t0, int nt, int t4) {
#pragma unroll
  for (int q = 0; q < kNg; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row + (i >> 1) * 8, t = 8 * q + 2 * t4 + (i & 1);
      if (r >= g.n || t >= nt) continue;
      const int64_t at = static_cast<int64_t>(t0 + t) * g.ldo + r;
      if (g.out_dtype == MUON_DT_BF16) static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(total[q][i]);
      else static_cast<float*>(g.out)[at] = total[q][i];
    }
}

// MX: the sums of a warp's row tile (its lane's rows `row` and row + 8 of W)
// over the blocks with big scales, times 2^-31; X of [k0, k0 + kc) is in shared
// memory.
template <int kNg>
__device__ __forceinline__ void big_scales(const RowsArgs& g, const uint8_t* smem, int row, int k0, int ks, int nt,
                                           float (&acc)[kNg][4]) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
  const int steps = (min(g.kc, g.k - k0) + kStepK - 1) / kStepK;
  const int chunks = static_cast<int>(g.pitch >> 4), atoms = static_cast<int>(g.atoms);
#pragma unroll 1
  for (int j = ks; j < steps; j += g.ks) {
    const int at = k0 / kStepK + j;  // step of the row, and its scale atom
    uint32_t w[2][4], sw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(row + 8 * h, g.n - 1);
      sw[h] = at < atoms ? __ldg(reinterpret_cast<const uint32_t*>(
                               g.scales + (static_cast<int64_t>(r >> 7) * g.atoms + at) * kAtomBytes + atom_byte(r, 0)))
                         : 0u;
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(g.data + static_cast<int64_t>(r) * g.pitch) + t4;
#pragma unroll
      for (int b = 0; b < 4; ++b) w[h][b] = 4 * at + b < chunks ? __ldg(codes + (4 * at + b) * 4) : 0u;
    }
    if (!__any_sync(0xffffffffu, (mx_big(sw[0]) | mx_big(sw[1])) != 0u)) continue;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t lo[4], hi[4];
      e2m1_expand8(w[0][b], lo);
      e2m1_expand8(w[1][b], hi);
      float s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t byte = (sw[h] >> 8 * b) & 255u;
        s[h] = byte == 255u ? __uint_as_float(0x7FFFFFFFu) : byte >= kMxBig ? __uint_as_float((byte - kMxDown) << 23) : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kNg; ++q) {
        const uint4 x =
            *reinterpret_cast<const uint4*>(smem + min(8 * q + gr, nt - 1) * g.xpitch + t4 * 16 + j * (kStepK * 2) + b * 64);
        float d4[4];
        mma16816_first(d4, lo[0], hi[0], lo[1], hi[1], x.x, x.y);
        mma16816(d4, lo[2], hi[2], lo[3], hi[3], x.z, x.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][i] = fmaf(s[i >> 1], d4[i], acc[q][i]);
      }
    }
  }
}

// What rows_in_parts works with, in shared memory in the place of the rings: as
// an argument by value g made a stack frame, and a kernel with one takes 1 us
// longer from stream to stream launch (28.2 instead of 26.8 us for
// 16 x 65536 x 2048); static arrays made the common path 1 to 5% slower.
struct PartsArgs {
  RowsArgs g;
  uint32_t amax[32];  // bits of the largest finite magnitude of each row of X
  int nparts;         // of the row with the most
};

// The row tiles of a CTA from group `grp` on, for an X whose rows spread over
// more exponents than an fp16 holds, and for big MX scales: each row tile once
// for each part of X, its sums in the order in which the kernel below adds
// them, so that a row of one part has the same bits from both.  Out of line, W
// straight from memory and steps not unrolled: the instructions of a call with
// few rows are a good part of its time, and its common path keeps its own
// (inlined, or sharing its code with the kernel, this cost that 5 to 13%; as it
// is, within 2%).
// Two parts take two to four times as long as one in the kernel.
template <bool kNv, int kNg, int kWarps>
__device__ __noinline__ void rows_in_parts(PartsArgs* args, int grp) {
  extern __shared__ __align__(16) uint8_t smem[];
  const RowsArgs& g = args->g;
  uint32_t* amax = args->amax;
  int* nparts = &args->nparts;
  float* sums = reinterpret_cast<float*>(smem + min(g.tg, g.t) * g.xpitch + kWarps * kDepth * kStepBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;
  const int ks = warp % g.ks, rw = warp / g.ks, per = kWarps / g.ks;
  const int t0 = blockIdx.y * g.tg;
  const int nt = min(g.tg, g.t - t0);
  const int ngroups = (g.n + 16 * per - 1) / (16 * per);
  const int chunks = static_cast<int>(g.pitch >> 4), atoms = static_cast<int>(g.atoms);  // of a row
  int eunit = -kMxUp;
  const float unit = kNv ? significand(*g.ts, eunit) : 1.0f;
  bool known = false;  // the ranges of X's rows
#pragma unroll 1
  for (; grp < ngroups; grp += gridDim.x) {
    float total[kNg][4] = {};
    const uint8_t *codes[2], *scales[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = min((grp * per + rw) * 16 + gr + 8 * h, g.n - 1);
      codes[h] = g.data + static_cast<int64_t>(row) * g.pitch;
      scales[h] = g.scales + static_cast<int64_t>(row >> 7) * g.atoms * kAtomBytes + atom_byte(row, 0);
    }
#pragma unroll 1
    for (int k0 = 0; k0 < g.k; k0 += g.kc) {
      const int steps = (min(g.kc, g.k - k0) + kStepK - 1) / kStepK;
      int part = 0;
#pragma unroll 1
      do {
        __syncthreads();
        stage_part<kNv, kNg, kWarps>(g, k0, part, part > 0 || known, t0, nt, smem, amax, nparts);
        __syncthreads();
        known = g.k <= g.kc;  // one pass: for the groups that follow too
        float acc[kNg][4] = {};
        uint32_t w[2][4], sw[2], next[2][4], snext[2], big = 0u;
        auto fetch = [&](int j) {
          const int at = k0 / kStepK + j;  // step of the row
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (kNv) {
              const int piece = 4 * at + t4, atom = 2 * at + (t4 >> 1);
              const uint4 v = piece < chunks ? __ldg(reinterpret_cast<const uint4*>(codes[h]) + piece) : make_uint4(0u, 0u, 0u, 0u);
              next[h][0] = v.x;
              next[h][1] = v.y;
              next[h][2] = v.z;
              next[h][3] = v.w;
              snext[h] = atom < atoms ? __ldg(reinterpret_cast<const unsigned short*>(
                                            scales[h] + static_cast<int64_t>(atom) * kAtomBytes + (t4 & 1) * 2))
                                      : 0u;
            } else {
#pragma unroll
              for (int b = 0; b < 4; ++b)
                next[h][b] = 4 * at + b < chunks ? __ldg(reinterpret_cast<const uint32_t*>(codes[h]) + (4 * at + b) * 4 + t4) : 0u;
              snext[h] = at < atoms ? __ldg(reinterpret_cast<const uint32_t*>(scales[h] + static_cast<int64_t>(at) * kAtomBytes)) : 0u;
            }
          }
        };
        if (ks < steps) fetch(ks);
#pragma unroll 1
        for (int j = ks; j < steps; j += g.ks) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sw[h] = snext[h];
#pragma unroll
            for (int b = 0; b < 4; ++b) w[h][b] = next[h][b];
          }
          if (j + g.ks < steps) fetch(j + g.ks);
          if (!kNv) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              big |= mx_big(sw[h]);
              sw[h] = mx_up_mixed(sw[h]);
            }
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t lo[4], hi[4];
            e2m1_expand8(w[0][b], lo);
            e2m1_expand8(w[1][b], hi);
            float s[2] = {};
            if (kNv) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const __half_raw r = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(sw[h] >> (b >> 1) * 8), __NV_E4M3);
                const uint32_t two = r.x * 0x10001u;
#pragma unroll
                for (int p = 0; p < 4; ++p) (h ? hi : lo)[p] = mul2((h ? hi : lo)[p], two);
              }
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) s[h] = mx_scale(sw[h], b);
            }
#pragma unroll
            for (int q = 0; q < kNg; ++q) {
              const uint4 x = *reinterpret_cast<const uint4*>(smem + min(8 * q + gr, nt - 1) * g.xpitch + t4 * 16 +
                                                              j * (kStepK * 2) + b * 64);
              if (kNv) {
                mma16816(acc[q], lo[0], hi[0], lo[1], hi[1], x.x, x.y);
                mma16816(acc[q], lo[2], hi[2], lo[3], hi[3], x.z, x.w);
              } else {
                float d4[4];
                mma16816_first(d4, lo[0], hi[0], lo[1], hi[1], x.x, x.y);
                mma16816(d4, lo[2], hi[2], lo[3], hi[3], x.z, x.w);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[q][i] = fmaf(s[i >> 1], d4[i], acc[q][i]);
              }
            }
          }
        }
        // undo the part's powers of two
#pragma unroll
        for (int q = 0; q < kNg; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = exponent_of(amax[min(8 * q + 2 * t4 + (i & 1), nt - 1)], part);
            total[q][i] += times_pow2(acc[q][i], unit, e + eunit);
          }
        if (!kNv && __any_sync(0xffffffffu, big != 0u)) {
          float more[kNg][4] = {};
          big_scales<kNg>(g, smem, (grp * per + rw) * 16 + gr, k0, ks, nt, more);
#pragma unroll
          for (int q = 0; q < kNg; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              total[q][i] += times_pow2(more[q][i], 1.0f,
                                        exponent_of(amax[min(8 * q + 2 * t4 + (i & 1), nt - 1)], part) + kMxDown);
        }
      } while (++part < *nparts);
    }
    if (g.ks > 1) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kNg; ++q)
        *reinterpret_cast<float4*>(sums + (warp * kNg + q) * 128 + lane * 4) =
            make_float4(total[q][0], total[q][1], total[q][2], total[q][3]);
      __syncthreads();
      if (ks != 0) continue;
#pragma unroll 1
      for (int w = 1; w < g.ks; ++w)
#pragma unroll
        for (int q = 0; q < kNg; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(sums + ((warp + w) * kNg + q) * 128 + lane * 4);
          total[q][0] += v.x;
          total[q][1] += v.y;
          total[q][2] += v.z;
          total[q][3] += v.w;
        }
    }
    store_rows(g, total, (grp * per + rw) * 16 + gr, t0, nt, t4);
  }
}

template <bool kNv, int kNg, int kWarps>
__device__ __forceinline__ void call_rows_in_parts(const RowsArgs& g, uint8_t* rings, int grp) {
  asm volatile("cp.async.wait_all;" ::: "memory");  // the loads ahead: the rings are free
  __syncthreads();
  PartsArgs* args = reinterpret_cast<PartsArgs*>(rings);
  if (threadIdx.x == 0) args->g = g;
  __syncthreads();
  rows_in_parts<kNv, kNg, kWarps>(args, grp);
}

template <bool kNv, int kNg, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) fp4_rows_kernel(const RowsArgs g) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t amax[8 * kNg];  // bits of the largest finite magnitude of each row of X
  uint8_t* rings = smem + min(g.tg, g.t) * g.xpitch;
  float* part = reinterpret_cast<float*>(rings + kWarps * kDepth * kStepBytes);  // [warp][16 * 8 * kNg], k split only
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;
  const int ks = warp % g.ks, rw = warp / g.ks, per = kWarps / g.ks;
  const int t0 = blockIdx.y * g.tg;
  const int nt = min(g.tg, g.t - t0);
  const int ngroups = (g.n + 16 * per - 1) / (16 * per);
  const int chunks = static_cast<int>(g.pitch >> 4), atoms = static_cast<int>(g.atoms);  // of a row

  uint8_t* ring = rings + warp * kDepth * kStepBytes;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  // Where this lane copies from: piece t4 (32 codes) of a step of rows g and
  // g + 8 of the row tile, and scale words (four blocks of a row): NV two a
  // row, of atoms 2 j and 2 j + 1, MX one, of atom j.  NV: a lane reads back the
  // pieces that it copied, [h][lane].  MX: a lane needs word t4 of all four
  // pieces of its rows, which lie as [h][piece][row], so that the eight rows of
  // an access meet no bank twice.  Scales lie as [h][word][row].
  const int sh = kNv ? t4 >> 1 : t4 & 1, sword = kNv ? t4 & 1 : 0;
  const uint32_t code_dst = ring_s + (kNv ? lane : t4 * 8 + gr) * 16;
  const uint32_t scale_dst = ring_s + 1024 + (sh * 16 + sword * 8 + gr) * 4;
  const uint8_t *code0 = nullptr, *code1 = nullptr, *scale = nullptr;
  int piece_at = 0, atom_at = 0;
  auto aim = [&](int grp, int k0) {  // at the first step of this warp
    const int r0 = (grp * per + rw) * 16 + gr;
    const int row0 = min(r0, g.n - 1), row1 = min(r0 + 8, g.n - 1), rs = sh ? row1 : row0;
    const int j = k0 / kStepK + ks;
    piece_at = 4 * j + t4;
    atom_at = kNv ? 2 * j + sword : j;
    code0 = g.data + static_cast<int64_t>(row0) * g.pitch + static_cast<int64_t>(piece_at) * 16;
    code1 = g.data + static_cast<int64_t>(row1) * g.pitch + static_cast<int64_t>(piece_at) * 16;
    scale = g.scales + (static_cast<int64_t>(rs >> 7) * g.atoms + atom_at) * kAtomBytes + atom_byte(rs, 0);
  };
  auto load = [&](uint32_t slot) {  // the step aimed at; then the next one
    // past the row's end nothing is read (a size of 0) and zeros are written
    const uint32_t nb = piece_at < chunks ? 16u : 0u;
    cp_async16(code_dst + slot, nb ? code0 : g.data, nb);
    cp_async16(code_dst + slot + 512, nb ? code1 : g.data, nb);
    const uint32_t sb = atom_at < atoms ? 4u : 0u;
    if (kNv || t4 < 2) cp_async4(scale_dst + slot, sb ? scale : g.scales, sb);
    piece_at += 4 * g.ks;
    code0 += 64 * g.ks;
    code1 += 64 * g.ks;
    atom_at += (kNv ? 2 : 1) * g.ks;
    scale += (kNv ? 2 : 1) * kAtomBytes * g.ks;
  };

  // X of [k0, k0 + kc) as scaled fp16, zeros past the edges.  Few rows are each
  // spread over several warps.  `exact` turns false if a value lies 32 exponents
  // or more below its row's largest.
  bool exact = true;
  auto stage = [&](int k0) {
    const int kn = min(g.kc, g.k - k0);
    const int pieces = (kn + kStepK - 1) / kStepK * (kStepK / 8);
    const int wpr = nt > kWarps / 2 ? 1 : kWarps / (nt > 4 ? 8 : nt > 2 ? 4 : nt);  // warps per row
    const int first = warp / wpr, rstep = kWarps / wpr, p0 = (warp - first * wpr) * 32 + lane, pstep = wpr * 32;
    auto piece = [&](const unsigned short* src, bool vec, int p) {
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (vec && p * 8 + 8 <= kn) {
        q = __ldg(reinterpret_cast<const uint4*>(src) + p);
      } else if (p * 8 < kn) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned short* e = src + p * 8 + 2 * i;
          const uint32_t lo = p * 8 + 2 * i < kn ? __ldg(e) : 0u, hi = p * 8 + 2 * i + 1 < kn ? __ldg(e + 1) : 0u;
          v[i] = lo | (hi << 16);
        }
        q = make_uint4(v[0], v[1], v[2], v[3]);
      }
      return q;
    };
    uint32_t least = 0u;  // of the last row: a warp with a share of a row has no other
    if (threadIdx.x < 8 * kNg) amax[threadIdx.x] = 0u;
    __syncthreads();
    for (int r = first; r < nt; r += rstep) {
      const unsigned short* src = reinterpret_cast<const unsigned short*>(g.x) + static_cast<int64_t>(t0 + r) * g.ldx + k0;
      const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
      uint32_t a = 0u;  // two magnitudes
      least = 0x7FFF7FFFu;
      auto look = [&](const uint4& q) {
        a = __vmaxu2(__vmaxu2(a, q.x & 0x7FFF7FFFu), __vmaxu2(q.y & 0x7FFF7FFFu, __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu)));
        least = __vmins2(__vmins2(least, wrapped(q.x)), __vmins2(wrapped(q.y), __vmins2(wrapped(q.z), wrapped(q.w))));
      };
      int p = p0;
      if (vec)
        for (; (p + 7 * pstep) * 8 + 8 <= kn; p += 8 * pstep) {
          uint4 q[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) q[u] = __ldg(reinterpret_cast<const uint4*>(src) + p + u * pstep);
#pragma unroll
          for (int u = 0; u < 8; ++u) look(q[u]);
        }
#pragma unroll 4
      for (; p < pieces; p += pstep) look(piece(src, vec, p));
      a = __reduce_max_sync(0xffffffffu, max(a & 0xFFFF0000u, a << 16));
      if (a >= 0x7F800000u) {  // a NaN or an infinity: the finite values alone set the power of two
        a = 0u;
        for (int p = p0; p < pieces; p += pstep) {
          const uint4 q = piece(src, vec, p);
          const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (v[i] << 16) & 0x7FFF0000u, hi = v[i] & 0x7FFF0000u;
            a = max(a, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
          }
        }
        a = __reduce_max_sync(0xffffffffu, a);
      }
      if (lane == 0) atomicMax(&amax[r], a);
      if (wpr == 1 && spread(a, least)) exact = false;
    }
    __syncthreads();
    for (int r = first; r < nt; r += rstep) {
      const unsigned short* src = reinterpret_cast<const unsigned short*>(g.x) + static_cast<int64_t>(t0 + r) * g.ldx + k0;
      const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
      const float f = pow2(-exponent_of(amax[r]));
      uint8_t* dst = smem + r * g.xpitch;
#pragma unroll 4
      for (int p = p0; p < pieces; p += pstep) {
        const uint4 q = piece(src, vec, p);
        const uint32_t v[4] = {q.x, q.y, q.z, q.w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 c = __floats2half2_rn(__uint_as_float(v[i] << 16) * f, __uint_as_float(v[i] & 0xFFFF0000u) * f);
          h[i] = *reinterpret_cast<const uint32_t*>(&c);
        }
        *reinterpret_cast<uint4*>(dst + x_place<kNv>(p)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      if (wpr > 1 && spread(amax[r], least)) exact = false;
    }
  };

  const int npass = (g.k + g.kc - 1) / g.kc;
  // columns of the products that X has no row for read its last one; they are not written
  int xrow[kNg];
#pragma unroll
  for (int q = 0; q < kNg; ++q) xrow[q] = min(8 * q + gr, nt - 1) * g.xpitch + t4 * 16;
  const float scale_g = kNv ? *g.ts : 1.0f;
  bool staged = false;
  uint32_t big = 0u;  // MX: a big scale was met, whose sums do not count
  for (int grp = blockIdx.x; grp < ngroups; grp += gridDim.x) {
    float total[kNg][4];
#pragma unroll
    for (int q = 0; q < kNg; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[q][i] = 0.0f;
    for (int pass = 0; pass < npass; ++pass) {
      const int k0 = pass * g.kc;
      const int steps = (min(g.kc, g.k - k0) + kStepK - 1) / kStepK;
      const int ni = (steps - ks + g.ks - 1) / g.ks;  // this warp's steps: ks, ks + KS, ...
      aim(grp, k0);
#pragma unroll
      for (int d = 0; d < kDepth - 1; ++d) {
        if (d < ni) load(d * kStepBytes);
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (npass > 1 || !staged) {  // behind the first loads of W
        __syncthreads();
        stage(k0);
        if (__syncthreads_or(!exact)) {
          call_rows_in_parts<kNv, kNg, kWarps>(g, rings, grp);
          return;
        }
        staged = true;
      }
      float acc[kNg][4];
#pragma unroll
      for (int q = 0; q < kNg; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
      const uint8_t* xj = smem + ks * (kStepK * 2);
      auto step = [&](int i, int d) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");  // step i has landed
        __syncwarp();  // for every lane, and step i - 1 has been read by every lane
        const uint8_t* st = ring + d * kStepBytes;
        uint32_t w[2][4], sw[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kNv) {
            const uint4 v = *reinterpret_cast<const uint4*>(st + h * 512 + lane * 16);
            w[h][0] = v.x;
            w[h][1] = v.y;
            w[h][2] = v.z;
            w[h][3] = v.w;
            // blocks 2 t4 and 2 t4 + 1 of the step's eight: half a word
            sw[h] = *reinterpret_cast<const unsigned short*>(st + 1024 + (h * 16 + (t4 >> 1) * 8 + gr) * 4 + (t4 & 1) * 2);
          } else {
            load_words(w[h], ring_s + static_cast<uint32_t>(d * kStepBytes + h * 512 + lane * 16));
            sw[h] = *reinterpret_cast<const uint32_t*>(st + 1024 + (h * 16 + gr) * 4);
          }
        }
        if (i + kDepth - 1 < ni) load((d + kDepth - 1) % kDepth * kStepBytes);  // over step i - 1
        asm volatile("cp.async.commit_group;" ::: "memory");
        uint32_t sc[2][2];
        if (kNv) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(sw[h]), __NV_E4M3);
            const uint32_t both = static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
            sc[h][0] = __byte_perm(both, both, 0x1010);
            sc[h][1] = __byte_perm(both, both, 0x3232);
          }
        }
        if (!kNv) {
          big |= mx_big(sw[0]) | mx_big(sw[1]);
          sw[0] = mx_up(sw[0]);
          sw[1] = mx_up(sw[1]);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t lo[4], hi[4];  // rows g and g + 8
          e2m1_expand8(w[0][b], lo);
          e2m1_expand8(w[1][b], hi);
          float s0 = 0.0f, s1 = 0.0f;
          if (kNv) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              lo[p] = mul2(lo[p], sc[0][b >> 1]);
              hi[p] = mul2(hi[p], sc[1][b >> 1]);
            }
          } else {
            s0 = mx_scale(sw[0], b);
            s1 = mx_scale(sw[1], b);
          }
#pragma unroll
          for (int q = 0; q < kNg; ++q) {
            const uint4 x = *reinterpret_cast<const uint4*>(xj + xrow[q] + b * 64);
            if (kNv) {
              mma16816(acc[q], lo[0], hi[0], lo[1], hi[1], x.x, x.y);
              mma16816(acc[q], lo[2], hi[2], lo[3], hi[3], x.z, x.w);
            } else {
              float d4[4];
              mma16816_first(d4, lo[0], hi[0], lo[1], hi[1], x.x, x.y);
              mma16816(d4, lo[2], hi[2], lo[3], hi[3], x.z, x.w);
              acc[q][0] = fmaf(s0, d4[0], acc[q][0]);
              acc[q][1] = fmaf(s0, d4[1], acc[q][1]);
              acc[q][2] = fmaf(s1, d4[2], acc[q][2]);
              acc[q][3] = fmaf(s1, d4[3], acc[q][3]);
            }
          }
        }
        xj += g.ks * (kStepK * 2);
      };
      int i = 0;
      for (; i + kDepth <= ni; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) step(i + d, d);
      }
#pragma unroll
      for (int d = 0; d < kDepth - 1; ++d)
        if (i + d < ni) step(i + d, d);
      __syncwarp();  // the ring is read before the next pass or tile fills it
      // undo X's powers of two; g is split here, and kept here by the asm, since
      // nothing before needs to wait for it (ahead of the loops: 6.8 instead of
      // 6.5 us for 1 x 8192 x 2048)
      int eunit = -kMxUp;
      float gw = scale_g;
      asm volatile("" : "+f"(gw));
      const float unit = kNv ? significand(gw, eunit) : 1.0f;
#pragma unroll
      for (int q = 0; q < kNg; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = exponent_of(amax[min(8 * q + 2 * t4 + j, nt - 1)]);
          total[q][j] += times_pow2(acc[q][j], unit, e + eunit);
          total[q][j + 2] += times_pow2(acc[q][j + 2], unit, e + eunit);
        }
    }
    if (g.ks > 1) {
      // the first warp of a row tile adds the others' sums, in order
      __syncthreads();
      float* mine = part + warp * (128 * kNg);
#pragma unroll
      for (int q = 0; q < kNg; ++q)
        *reinterpret_cast<float4*>(mine + q * 128 + lane * 4) =
            make_float4(total[q][0], total[q][1], total[q][2], total[q][3]);
      __syncthreads();
      if (ks != 0) continue;
      for (int w = 1; w < g.ks; ++w)
#pragma unroll
        for (int q = 0; q < kNg; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(part + (warp + w) * (128 * kNg) + q * 128 + lane * 4);
          total[q][0] += v.x;
          total[q][1] += v.y;
          total[q][2] += v.z;
          total[q][3] += v.w;
        }
    }
#pragma unroll
    for (int q = 0; q < kNg; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (grp * per + rw) * 16 + gr + (i >> 1) * 8;
        const int t = 8 * q + 2 * t4 + (i & 1);
        if (row >= g.n || t >= nt) continue;
        const float v = total[q][i];
        const int64_t at = static_cast<int64_t>(t0 + t) * g.ldo + row;
        if (g.out_dtype == MUON_DT_BF16) static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(v);
        else static_cast<float*>(g.out)[at] = v;
      }
  }
  if (!kNv && __syncthreads_or(big != 0u)) call_rows_in_parts<kNv, kNg, kWarps>(g, rings, blockIdx.x);  // all of them again
}

template <bool kNv, int kNg, int kWarps>
cudaError_t launch_rows_w(const RowsArgs& g, int dev, int ctas, int smem, cudaStream_t st) {
  const int per = kWarps / g.ks;
  const int groups = ((g.n + 15) / 16 + per - 1) / per;
  const dim3 grid(groups < ctas ? groups : ctas, (g.t + g.tg - 1) / g.tg);
  auto kernel = fp4_rows_kernel<kNv, kNg, kWarps>;
  if (smem + 1024 > 48 * 1024) {  // with the static share
    const cudaError_t e = allow_smem<fp4_rows_kernel<kNv, kNg, kWarps>>(dev, kSmemMax);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, 32 * kWarps, smem, st>>>(g);
  return cudaGetLastError();
}

// 16 warps of 128 registers a SM: up to eight rows of X as two CTAs, whose
// copies of X are small and whose barriers overlap (65536 x 2048, NV, t = 1:
// 19.6 us against 20.3 us as one CTA; 2048 x 8192 7.2 against 8.6 us), more
// rows as one CTA, which copies X once (t = 16: 26.6 against 27.7 us, t = 32:
// 39.8 against 46.1 us); eight warps where X takes the shared memory.  (These
// pairs were measured before rows could be taken in parts; the choices made
// now take 20.2, 7.1, 26.1 and 40.2 us.)  Kernels for more than 16 rows spill
// 32 (NV) or 72 (MX) bytes, MX ones for 9 to 16 rows 28; with 24 warps of 80
// registers the spills took t = 16 to 39.9 us.
template <bool kNv, int kNg>
cudaError_t launch_rows(const RowsArgs& g, int dev, int sms, cudaStream_t st) {
  auto smem = [&](int warps) {
    return (g.t < g.tg ? g.t : g.tg) * g.xpitch + warps * (kDepth * kStepBytes + (g.ks > 1 ? 128 * kNg * 4 : 0));
  };
  const bool two = 2 * (smem(8) + 2048) <= kSmemMax;
  // fewer row tiles than 16 warps a SM take: CTAs of eight reach more SMs
  // (many rows of X are better copied by 16 warps)
  const bool few = static_cast<int64_t>((g.n + 15) / 16) * g.ks < 16 * static_cast<int64_t>(sms);
  if ((kNg == 1 && (two || few)) || smem(16) > kSmemMax) return launch_rows_w<kNv, kNg, 8>(g, dev, two ? 2 * sms : sms, smem(8), st);
  return launch_rows_w<kNv, kNg, 16>(g, dev, sms, smem(16), st);
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
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MUON_ERR_CUDA;
  const int sms = device_sms(dev);
  if (sms <= 0) return MUON_ERR_UNSUPPORTED;

  RowsArgs g{static_cast<const __nv_bfloat16*>(x), static_cast<const uint8_t*>(w->data),
             static_cast<const uint8_t*>(w->scales), w->tensor_scale, out, ldx, ldo, pitch_of(w->k),
             atoms_of(w->format, w->k), static_cast<int32_t>(t), static_cast<int32_t>(w->rows),
             static_cast<int32_t>(w->k), out_dtype, 0, 0, 0, 0};
  // k of a pass: all of it, up to what eight rows of X fit for.  Neither this
  // nor the k split depends on t, so that a row's sums have one order.
  g.kc = static_cast<int32_t>(w->k < kMaxK ? w->k : kMaxK);
  // rows of X in shared memory are 64 bytes past a multiple of 128, so that the
  // eight lanes of a 16-byte access (two rows, four pieces) meet no bank twice
  g.xpitch = (g.kc + kStepK - 1) / kStepK * kStepK * 2 + 64;
  int ng = t <= 8 ? 1 : t <= 16 ? 2 : 4;
  while (ng > 1 && 8 * ng * g.xpitch > kXBudget) ng /= 2;
  g.tg = 8 * ng;
  // k split: the fewest steps of a warp when 16 warps a SM take the row tiles in
  // rounds, a reduction counted as a step
  const int64_t tiles = (w->rows + 15) / 16;
  const int steps = (g.kc + kStepK - 1) / kStepK;
  int64_t best = 0;
  for (int ks = 1; ks <= 8; ks *= 2) {
    const int64_t rounds = (tiles * ks + 16 * sms - 1) / (16 * sms);
    const int64_t cost = rounds * ((steps + ks - 1) / ks + (ks > 1 ? 1 : 0));
    if (ks == 1 || cost < best) {
      best = cost;
      g.ks = ks;
    }
  }
  const bool nv = w->format == MUON_FP4_NV;
  cudaError_t e;
  if (ng == 1) e = nv ? launch_rows<true, 1>(g, dev, sms, st) : launch_rows<false, 1>(g, dev, sms, st);
  else if (ng == 2) e = nv ? launch_rows<true, 2>(g, dev, sms, st) : launch_rows<false, 2>(g, dev, sms, st);
  else e = nv ? launch_rows<true, 4>(g, dev, sms, st) : launch_rows<false, 4>(g, dev, sms, st);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
