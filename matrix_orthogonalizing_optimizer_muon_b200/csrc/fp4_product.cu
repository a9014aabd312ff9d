// Product of two 4-bit matrices, out[M, N] = A B^T (format: fp4.cuh), on the
// 5th-generation tensor cores: sum over blocks of s_a s_b sum over the block
// of the codes' products, block scaling done by the tensor core, fp32 sums.
//
// A tile of kCg * 128 x kBn outputs is computed by kCg CTAs (a 2-CTA pair
// sharing one tcgen05.mma.cta_group::2, or one CTA).  Per CTA:
//   warp 0       TMA producer: four lanes load a stage (256 of K: 128 bytes a
//                row) of A's codes, B's codes, A's scales and B's scales; the
//                scale atoms arrive in the order in which they are stored.
//   warp 1       TMEM allocator; in the leading CTA the warp copies a stage's
//                scale atoms to TMEM (tcgen05.cp, 32 lanes x 16 bytes, repeated
//                for the four lane quadrants) and issues its four MMAs of
//                K = 64, all from one elected lane: 17 tcgen05 instructions a
//                stage.  Issued under `lane == 0` instead, each took about 75
//                cycles and 8192^3 332 us; elected, 211 us.  A stage's scales
//                have TMEM columns of their own, so they are overwritten only
//                after the MMAs that read them have released the stage.
//   warps 2..9   epilogue: a warp takes 32 rows and half the columns, 32 x 32
//                blocks at a time, scales and converts them and stores each
//                from a staging block by TMA (added in fp32 by the TMA's
//                reduction), or, where the output's rows do not start or end
//                on 16-byte boundaries (TMA writes whole 16-byte pieces), by
//                rows of the block.  Two
//                accumulators and the scales do not fit into TMEM's 512
//                columns, so a warp takes its share into registers (packed, if
//                bf16) and releases the accumulator before it stores any.
#include "fp4.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>

namespace {

using namespace muon;
using namespace muon::fp4;

__device__ unsigned g_fp4_status;  // kStatusTimeout, sticky until muon_fp4_get_status

constexpr int kThreadsP = 320;
constexpr int kEpi0 = 2;            // first epilogue warp
constexpr int kEpiWarpsP = 8;
constexpr int kStagingBytes = 32 * 32 * 4;  // an epilogue warp's block of 32 x 32 outputs
constexpr int kStageK = 256;        // K of a stage: one 128-byte swizzle atom of codes
constexpr int kRowBytes = 128;      // codes of a row in a stage
constexpr int kMmaK = 64;           // K of one MMA

__host__ __device__ constexpr int atoms_per_stage(bool nv) { return nv ? 4 : 2; }

template <int kCg, int kBn, bool kNv>
struct Cfg {
  static constexpr int kAtoms = atoms_per_stage(kNv);
  static constexpr int kABytes = 128 * kRowBytes;
  static constexpr int kBRows = kBn / kCg;  // B rows staged by one CTA
  static constexpr int kBBytes = kBRows * kRowBytes;
  static constexpr int kSaBytes = kAtoms * kAtomBytes;
  static constexpr int kSbBytes = kAtoms * kAtomBytes * (kBn / 128);  // every CTA needs the scales of all kBn columns
  static constexpr int kStage = kABytes + kBBytes + kSaBytes + kSbBytes;
  static constexpr int kStages = 5;
  static constexpr int kEpi = kStages * kStage;
  static constexpr int kBar = kEpi + kEpiWarpsP * kStagingBytes;
  static constexpr int kMisc = kBar + (2 * kStages + 3) * 8;
  static constexpr int kSmem = kMisc + 16 + 1024;
  static constexpr uint32_t kTx = static_cast<uint32_t>(kCg) * kStage;
  // TMEM columns: accumulator, then per stage the scales of A and of B
  static constexpr int kSfStage = kAtoms * 4 * (1 + kBn / 128);
  static constexpr int kSf0 = kBn;
  static constexpr int kCols = 512;
  static_assert(kSf0 + kStages * kSfStage <= kCols, "TMEM");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kStage % 1024 == 0, "swizzle atoms");
};

struct ProdArgs {
  void* out;
  int64_t ldo;
  const float* ga;
  const float* gb;
  int32_t m, n, nk, tiles_m, tiles_n;
  int32_t out_dtype, accumulate, vec;
  uint32_t test_wait_ns;  // 0; > 0 only for the failure-detection test (muon_fp4_inject_wait_timeout)
};

template <int kCg>
__device__ __forceinline__ void tma_load(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  if (kCg == 2) {
    tma_load_pair(dst, map, x, y, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}

// true in one lane of a converged warp; the code under it keeps its operands
// in uniform registers, which tcgen05 instructions take
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0u;
}

// arrive on the barrier at this offset in every CTA of the tile once this
// thread's earlier tensor-core work is done
template <int kCg>
__device__ __forceinline__ void commit_all(uint32_t bar) {
  if (kCg == 2) tc_commit_pair(bar);
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// wait until all but this thread's last kN bulk stores have read shared memory
template <int kN>
__device__ __forceinline__ void bulk_wait_read_but() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kN) : "memory");
}

// TMA reduction of a staged box: global += shared, in fp32
__device__ __forceinline__ void tma_add_2d(const void* map, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// Scale atom (512 bytes of shared memory: 32 rows of 16 bytes) to four TMEM columns.
template <int kCg>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if (kCg == 2) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <int kCg, bool kNv>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t acc) {
#define MUON_FP4_MMA(cg, kind, vec)                                                                             \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::" cg ".kind::" kind       \
               ".block_scale.scale_vec::" vec " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                \
               "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)                                           \
               : "memory")
  if (kNv) {
    if (kCg == 2) MUON_FP4_MMA("2", "mxf4nvf4", "4X");
    else MUON_FP4_MMA("1", "mxf4nvf4", "4X");
  } else {
    if (kCg == 2) MUON_FP4_MMA("2", "mxf4", "2X");
    else MUON_FP4_MMA("1", "mxf4", "2X");
  }
#undef MUON_FP4_MMA
}

// 128-byte-swizzled K-major operand: eight rows of 128 bytes every 1024
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// unswizzled scale atom: eight rows of 16 bytes every 128
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(128 >> 4) << 32) |
         (uint64_t(1) << 46);
}

// Instruction descriptor of the 4-bit kinds: e2m1 x e2m1 (1 at bits 7 and
// 10), N / 8 at 17, scale type at 23 (1: e8m0, 0: e4m3), M / 16 at 24; the
// byte of a scale column's word from which A's and B's scales are taken at 29
// and 4.
template <int kCg, int kBn, bool kNv>
__device__ __forceinline__ uint32_t make_idesc_fp4(uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kBn >> 3) << 17) | ((kNv ? 0u : 1u) << 23) |
         (static_cast<uint32_t>((128 * kCg) >> 4) << 24) | (sf_id << 29);
}

// Tile t in an order that keeps eight rows of tiles together, so that the
// tiles in flight share operands in L2.
__device__ __forceinline__ void tile_place(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kGroup = 8;
  const int per = kGroup * tiles_n;
  const int g = t / per, first = g * kGroup;
  const int rows = min(kGroup, tiles_m - first);
  const int r = t - g * per;
  tm = first + r % rows;
  tn = r / rows;
}

__device__ __forceinline__ void give_up(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(&g_fp4_status, kStatusTimeout);
}

template <int kCg, int kBn, bool kNv>
__global__ void __launch_bounds__(kThreadsP, 1)
    fp4_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
                       const __grid_constant__ CUtensorMap map_o, const ProdArgs g) {
  using C = Cfg<kCg, kBn, kNv>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * C::kStages);
  const uint32_t tempty_bar = tfull_bar + 8u;
  const uint32_t drain_bar = tfull_bar + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kCg == 2 ? cta_rank() : 0u;
  const bool leader = rank == 0u;
  const int unit = static_cast<int>(blockIdx.x) / kCg, nunits = static_cast<int>(gridDim.x) / kCg;
  const int ntiles = g.tiles_m * g.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tempty_bar, kCg * kEpiWarpsP);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (kCg == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(C::kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(C::kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kCg == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (g.test_wait_ns != 0) {
    // Failure-detection test: one thread per CTA waits, with the short limit, on
    // a barrier on which nothing arrives before the last MMA, and gives up.  No
    // role starts, so no load or tensor-core instruction is ever issued.
    if (threadIdx.x == 0 && !wait_bounded_ns(drain_bar, 0u, nullptr, g.test_wait_ns)) give_up(abort_flag);
    __syncthreads();
  }

  if (g.test_wait_ns != 0 && *abort_flag != 0) {
    // nothing
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    const void* map = lane == 0 ? &map_a : lane == 1 ? &map_b : lane == 2 ? &map_sa : &map_sb;
    if (lane < 4) prefetch_tensormap(map);
    const uint32_t off = lane == 0 ? 0u
                         : lane == 1 ? C::kABytes
                         : lane == 2 ? C::kABytes + C::kBBytes
                                     : C::kABytes + C::kBBytes + C::kSaBytes;
    const int xstep = lane < 2 ? kRowBytes : C::kAtoms * (kAtomBytes / 8);
    const uint32_t full0 = kCg == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
    int stage = 0;
    uint32_t phase = 0;
    long fills = 0;
    for (int t = unit; t < ntiles; t += nunits) {
      int tm, tn;
      tile_place(t, g.tiles_m, g.tiles_n, tm, tn);
      const int row_block = tm * kCg + static_cast<int>(rank);
      const int y = lane == 0   ? row_block * 128
                    : lane == 1 ? tn * kBn + static_cast<int>(rank) * C::kBRows
                    : lane == 2 ? row_block
                                : tn * (kBn / 128);
      bool ok = true;
      for (int kb = 0; kb < g.nk; ++kb, ++fills) {
        int ready = 0;
        if (lane == 0) {
          ready = wait_hot(empty_bar(stage), phase ^ 1u, abort_flag) ? 1 : 0;
          if (!ready) give_up(abort_flag);
          else if (leader) mbar_arrive_expect_tx(full_bar(stage), C::kTx);
        }
        ready = __shfl_sync(0xffffffffu, ready, 0);
        if (!ready) {
          ok = false;
          break;
        }
        if (lane < 4)
          tma_load<kCg>(sbase + stage * C::kStage + off, map, kb * xstep, y, full0 + 8u * static_cast<uint32_t>(stage));
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
    }
    // both CTAs' loads complete on the leader's barriers: the last fill of
    // every stage has landed before any CTA leaves
    if (leader && lane == 0) {
      for (long f = fills > C::kStages ? fills - C::kStages : 0; f < fills; ++f)
        if (!wait_bounded(full_bar(static_cast<int>(f % C::kStages)), static_cast<uint32_t>((f / C::kStages) & 1), nullptr))
          atomicOr(&g_fp4_status, kStatusTimeout);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      const uint64_t a0 = operand_desc(sbase), b0 = operand_desc(sbase + C::kABytes);
      const uint64_t sa0 = scale_desc(sbase + C::kABytes + C::kBBytes);
      const uint64_t sb0 = scale_desc(sbase + C::kABytes + C::kBBytes + C::kSaBytes);
      int stage = 0;
      uint32_t phase = 0, tphase = 0;
      bool issued = false, ok = true;
      for (int t = unit; t < ntiles && ok; t += nunits) {
        ok = __all_sync(0xffffffffu, wait_hot(tempty_bar, tphase ^ 1u, abort_flag));
        if (!ok) break;
        tphase ^= 1u;
        tc_fence_after();
        for (int kb = 0; kb < g.nk; ++kb) {
          ok = __all_sync(0xffffffffu, wait_hot(full_bar(stage), phase, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t so = static_cast<uint64_t>((stage * C::kStage) >> 4);
            const uint32_t sfa = tmem + C::kSf0 + stage * C::kSfStage;
            const uint32_t sfb = sfa + C::kAtoms * 4;
#pragma unroll
            for (int k = 0; k < C::kAtoms; ++k) {
              copy_scales<kCg>(sfa + 4 * k, sa0 + so + (k * kAtomBytes >> 4));
#pragma unroll
              for (int r = 0; r < kBn / 128; ++r)  // the two row blocks of B side by side
                copy_scales<kCg>(sfb + k * 4 * (kBn / 128) + 4 * r,
                                 sb0 + so + ((r * C::kAtoms + k) * kAtomBytes >> 4));
            }
#pragma unroll
            for (int kk = 0; kk < kStageK / kMmaK; ++kk) {
              const int atom = kNv ? kk : kk >> 1;
              mma_fp4<kCg, kNv>(tmem, a0 + so + (kk * 32 >> 4), b0 + so + (kk * 32 >> 4),
                                make_idesc_fp4<kCg, kBn, kNv>(kNv ? 0u : (kk & 1) * 2u), sfa + 4 * atom,
                                sfb + atom * 4 * (kBn / 128), (kb | kk) != 0 ? 1u : 0u);
            }
            commit_all<kCg>(empty_bar(stage));
          }
          __syncwarp();
          issued = true;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && elect_one()) commit_all<kCg>(tfull_bar);
        __syncwarp();
      }
      if (!ok && lane == 0) give_up(abort_flag);
      if (issued) {
        if (elect_one()) {
          if (kCg == 2) tc_commit(drain_bar);
          else commit_all<1>(drain_bar);
        }
        __syncwarp();
        if (!wait_bounded(drain_bar, 0u, nullptr)) atomicOr(&g_fp4_status, kStatusTimeout);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, half = (warp - kEpi0) >> 2;
    constexpr int kPer = kBn / 2 / 32;  // 32-column blocks of a warp
    const uint32_t tempty = kCg == 2 ? map_to_rank(tempty_bar, 0) : tempty_bar;
    // g_A g_B as two factors, half of its exponent in each: both shrink or both
    // grow, so that nothing passes either end of fp32's range that the result
    // does not pass.  (Below 2^-252 a sum gives 0.)
    float ga = 1.0f, gb = 1.0f;
    if (kNv) {
      const float sa = *g.ga, sb = *g.gb;
      int ea, eb;
      ga = significand(fabsf(sa) < fabsf(sb) ? sa : sb, ea);
      gb = significand(fabsf(sa) < fabsf(sb) ? sb : sa, eb);
      const int e = max(ea + eb, -252);
      ga *= pow2(e >> 1);
      gb *= pow2(e - (e >> 1));
    }
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * (kBn / 2);
    uint8_t* stg = smem + C::kEpi + (warp - kEpi0) * kStagingBytes;
    int turn = 0;
    uint32_t tphase = 0;
    for (int t = unit; t < ntiles; t += nunits) {
      const bool ready = wait_bounded(tfull_bar, tphase, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) {  // the warp leaves as one: tcgen05.ld is aligned
        if (lane == 0) give_up(abort_flag);
        break;
      }
      tphase ^= 1u;
      tc_fence_after();
      int tm, tn;
      tile_place(t, g.tiles_m, g.tiles_n, tm, tn);
      const int row0 = (tm * kCg + static_cast<int>(rank)) * 128 + quad * 32;
      const int col0 = tn * kBn + half * (kBn / 2);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty);
      };
      if (g.out_dtype == MUON_DT_BF16) {
        uint32_t h[kPer][16];
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          uint32_t v[32];
          tmem_ld32(tq + c * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x = __uint_as_float(v[2 * i]), y = __uint_as_float(v[2 * i + 1]);
            if (kNv) {
              x = x * ga * gb;
              y = y * ga * gb;
            }
            const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
            h[c][i] = *reinterpret_cast<const uint32_t*>(&p);
          }
        }
        release();
        if (row0 >= g.m) continue;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          const int col = col0 + c * 32;
          if (col >= g.n) continue;
          if (g.vec && (col + 32 <= g.n || g.n % 8 == 0)) {
            // the halves take turns store by store (a ragged tile may store one
            // block only): the store before the last has read this one
            uint8_t* blk = stg + turn * (kStagingBytes / 2);
            turn ^= 1;
            if (lane == 0) bulk_wait_read_but<1>();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(blk + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(h[c][4 * q], h[c][4 * q + 1], h[c][4 * q + 2], h[c][4 * q + 3]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&map_o, smem_u32(blk), col, row0);
              bulk_commit();
            }
          } else {
            // rows of 17 words: a thread writes its row and reads a column without conflicts
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(g.out) + static_cast<int64_t>(row0) * g.ldo + col;
            uint32_t* w = reinterpret_cast<uint32_t*>(stg);
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[lane * 17 + i] = h[c][i];
            __syncwarp();
            const int nr = min(32, g.m - row0);
            if (col + lane < g.n)
              for (int r = 0; r < nr; ++r)
                out[r * g.ldo + lane] = reinterpret_cast<const __nv_bfloat16*>(w + r * 17)[lane];
            __syncwarp();
          }
        }
      } else {
        uint32_t v[kPer][32];
#pragma unroll
        for (int c = 0; c < kPer; ++c) tmem_ld32(tq + c * 32, v[c]);
        tmem_ld_wait();
        release();
        if (row0 >= g.m) continue;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          const int col = col0 + c * 32;
          if (col >= g.n) continue;
          if (kNv) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[c][i] = __float_as_uint(__uint_as_float(v[c][i]) * ga * gb);
          }
          if (lane == 0) bulk_wait_read();
          __syncwarp();
          if (g.vec && (col + 32 <= g.n || g.n % 4 == 0)) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_uint4(v[c][4 * q], v[c][4 * q + 1], v[c][4 * q + 2], v[c][4 * q + 3]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              if (g.accumulate) tma_add_2d(&map_o, smem_u32(stg), col, row0);
              else tma_store_2d(&map_o, smem_u32(stg), col, row0);
              bulk_commit();
            }
          } else {
            float* out = static_cast<float*>(g.out) + static_cast<int64_t>(row0) * g.ldo + col;
            uint32_t* w = reinterpret_cast<uint32_t*>(stg);
            // word i of row r at column i ^ r: conflict-free both ways
#pragma unroll
            for (int i = 0; i < 32; ++i) w[lane * 32 + (i ^ lane)] = v[c][i];
            __syncwarp();
            const int nr = min(32, g.m - row0);
            if (col + lane < g.n) {
#pragma unroll 8
              for (int r = 0; r < nr; ++r) {
                const float f = __uint_as_float(w[r * 32 + (lane ^ r)]);
                // added where it lies (one addition an element), so that no load is waited for
                if (g.accumulate) atomicAdd(out + r * g.ldo + lane, f);
                else out[r * g.ldo + lane] = f;
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // the staging blocks are read, and the stores done, before the CTA leaves
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (kCg == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (kCg == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
}

// ---------------------------------------------------------------- host
thread_local uint32_t t_test_wait_ns = 0;  // for this thread's next launch

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = []() -> EncodeFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Codes of a 4-bit matrix: boxes of 128 bytes x `rows` rows, 128-byte swizzle,
// zeros past the edges.
bool encode_codes(CUtensorMap* tm, const muon_fp4_matrix_t& m, int rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch_of(m.k)), static_cast<cuuint64_t>(m.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_of(m.k))};
  const cuuint32_t box[2] = {kRowBytes, static_cast<cuuint32_t>(rows)};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.data, dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale atoms as rows of 8-byte words: boxes of a stage's atoms x `blocks`
// row blocks, zeros (a scale of 0, or 2^-127 on codes that are 0) past the edges.
bool encode_scales(CUtensorMap* tm, const muon_fp4_matrix_t& m, int blocks) {
  const int64_t atoms = atoms_of(m.format, m.k);
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(atoms) * (kAtomBytes / 8),
                              static_cast<cuuint64_t>(row_blocks_of(m.rows))};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(atoms) * kAtomBytes};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(atoms_per_stage(m.format == MUON_FP4_NV) * (kAtomBytes / 8)),
                             static_cast<cuuint32_t>(blocks)};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, m.scales, dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output in blocks of 32 x 32, staged rows swizzled over the row's 64 or 128 bytes.
bool encode_out(CUtensorMap* tm, const ProdArgs& g) {
  const bool bf = g.out_dtype == MUON_DT_BF16;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.n), static_cast<cuuint64_t>(g.m)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.ldo) * (bf ? 2 : 4)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, g.out, dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     bf ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCg, int kBn, bool kNv>
muon_status_t launch_product(const muon_fp4_matrix_t& a, const muon_fp4_matrix_t& b, ProdArgs g, int dev, int sms,
                             cudaStream_t st) {
  using C = Cfg<kCg, kBn, kNv>;
  CUtensorMap ma, mb, msa, msb, mo = {};
  if (!encode_codes(&ma, a, 128) || !encode_codes(&mb, b, C::kBRows) || !encode_scales(&msa, a, 1) ||
      !encode_scales(&msb, b, kBn / 128) || (g.vec && !encode_out(&mo, g)))
    return MUON_ERR_CUDA;
  auto kernel = fp4_product_kernel<kCg, kBn, kNv>;
  if (allow_smem<fp4_product_kernel<kCg, kBn, kNv>>(dev, C::kSmem) != cudaSuccess) return MUON_ERR_CUDA;
  g.tiles_m = (g.m + kCg * 128 - 1) / (kCg * 128);
  g.tiles_n = (g.n + kBn - 1) / kBn;
  const int64_t tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  if (tiles > 0x3fffffff) return MUON_ERR_UNSUPPORTED;
  const int64_t units = tiles < sms / kCg ? tiles : sms / kCg;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * kCg));
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCg;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, msa, msb, mo, g) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

}  // namespace

extern "C" {

muon_status_t muon_fp4_product(const muon_fp4_matrix_t* a, const muon_fp4_matrix_t* b, void* out, int64_t ldo,
                               int32_t out_dtype, int32_t accumulate, void* stream) {
  if (a == nullptr || b == nullptr || !valid(*a) || !valid(*b)) return MUON_ERR_INVALID_ARG;
  if (out_dtype != MUON_DT_BF16 && out_dtype != MUON_DT_FP32) return MUON_ERR_INVALID_ARG;
  if ((accumulate != 0 && accumulate != 1) || (accumulate && out_dtype != MUON_DT_FP32)) return MUON_ERR_INVALID_ARG;
  if (a->k != b->k || a->format != b->format) return MUON_ERR_SHAPE_MISMATCH;
  if (a->rows == 0 || b->rows == 0) return MUON_OK;
  const int es = out_dtype == MUON_DT_BF16 ? 2 : 4;
  const uintptr_t o = reinterpret_cast<uintptr_t>(out);
  if (out == nullptr || o % es != 0 || ldo < b->rows || ldo > (int64_t(1) << 40)) return MUON_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->k == 0) {
    if (accumulate) return MUON_OK;
    return cudaMemset2DAsync(out, static_cast<size_t>(ldo) * es, 0, static_cast<size_t>(b->rows) * es,
                             static_cast<size_t>(a->rows), st) == cudaSuccess
               ? MUON_OK
               : MUON_ERR_CUDA;
  }
  RangeList reads, writes;
  add_ranges(*a, reads);
  add_ranges(*b, reads);
  writes.push_back(ByteRange{o, o + (static_cast<size_t>(a->rows - 1) * ldo + b->rows) * es});
  if (conflict(reads, writes)) return MUON_ERR_ALIAS;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MUON_ERR_CUDA;
  const int sms = device_sms(dev);
  if (sms <= 0) return MUON_ERR_UNSUPPORTED;
  if (encode_fn() == nullptr) return MUON_ERR_CUDA;
  ProdArgs g = {};
  g.out = out;
  g.ldo = ldo;
  g.ga = a->tensor_scale;
  g.gb = b->tensor_scale;
  g.m = static_cast<int32_t>(a->rows);
  g.n = static_cast<int32_t>(b->rows);
  g.nk = static_cast<int32_t>((a->k + kStageK - 1) / kStageK);
  g.out_dtype = out_dtype;
  g.accumulate = accumulate;
  // TMA stores take rows on 16-byte boundaries at most 2^40 bytes apart (one row has no pitch to speak of)
  const int64_t pitch = a->rows == 1 ? (b->rows + 7) / 8 * 8 : ldo;
  g.vec = (o % 16 == 0 && pitch * es % 16 == 0 && pitch * es < (int64_t(1) << 40)) ? 1 : 0;
  if (g.vec) g.ldo = pitch;
  g.test_wait_ns = t_test_wait_ns;
  t_test_wait_ns = 0;
  const bool nv = a->format == MUON_FP4_NV;
  // pairs where there are enough 256 x 256 tiles for them, single CTAs below
  const int64_t pair_tiles = ((a->rows + 255) / 256) * ((b->rows + 255) / 256);
  if (pair_tiles >= sms / 4)
    return nv ? launch_product<2, 256, true>(*a, *b, g, dev, sms, st)
              : launch_product<2, 256, false>(*a, *b, g, dev, sms, st);
  return nv ? launch_product<1, 128, true>(*a, *b, g, dev, sms, st)
            : launch_product<1, 128, false>(*a, *b, g, dev, sms, st);
}

muon_status_t muon_fp4_inject_wait_timeout(uint32_t wait_ns) {
  if (wait_ns < 1 || wait_ns > 1000000000u) return MUON_ERR_INVALID_ARG;
  t_test_wait_ns = wait_ns;
  return MUON_OK;
}

muon_status_t muon_fp4_get_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return MUON_ERR_CUDA;
  }
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fp4_status, sizeof(v)) != cudaSuccess ||
      (v != 0 && (cudaMemcpyToSymbol(g_fp4_status, &zero, sizeof(zero)) != cudaSuccess || !uploads_done()))) {
    cudaGetLastError();
    return MUON_ERR_CUDA;
  }
  return (v & kStatusTimeout) ? MUON_ERR_TIMEOUT : MUON_OK;
}

}  // extern "C"
