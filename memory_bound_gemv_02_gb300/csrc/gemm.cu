// C = act(alpha * sa_i sb_j (A B^T)_ij + beta * bias_j) + residual (see
// gemm_fused() in gemv_ops.h), on the fifth-generation tensor cores.
//
// The weights B take the M side of every tcgen05.mma and the vectors A the N
// side: a CTA's accumulator holds 128 rows of B (TMEM lanes) by up to 256
// vectors (columns).  So a few vectors cost a few columns and the weights still
// stream at full width, and each epilogue thread owns one output column j: its
// bias and scale are registers, and the 32 lanes of a warp write 32 neighbours
// of a row of C.
//
// Operand tiles are 128 bytes of k wide (64 16-bit or 128 8-bit elements) in
// the 128-byte swizzle, in a ring of stages.  Warp 0 fills the ring by TMA, one
// thread of warp 1 issues the matrix instructions, eight warps write the result.
// An operand whose base or row stride is not a multiple of 16 bytes is no tensor
// map's.  Many vectors: it is first copied to the workspace with rows that are
// (gemm_align_kernel).  Few: B is read in place by one tensor map for each of
// its classes of rows that start alike (ShiftedParams).  Shifting rows into place
// within the product was slower than either at every size (77 x 4099 x 7169 fp16:
// 72 us with cp.async of the covering blocks, 220 with a bulk copy per row, 37
// copied first, 22 by classes): 128-byte pieces of 128 rows are the wrong shape
// for anything but a tensor map.
//
// Two kernels:
//  * gemm_split_kernel, one tile per CTA: clusters of up to 8 CTAs share a tile
//    and split its k; their partial sums are exchanged through distributed
//    shared memory, each CTA finishing its share of the columns, in CTA order.
//  * gemm_pair_kernel, persistent: pairs of CTAs compute 256 x 256 tiles with
//    cta_group::2 instructions (each CTA loads half of both operands), two
//    accumulators in TMEM so that a tile's epilogue overlaps the next product.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ops_internal.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace gemvk {
namespace {

constexpr int kRowBytes = 128;                   // bytes of k per tile row
constexpr int kTileRows = 128;                   // rows of B per CTA
constexpr int kTileBytes = kTileRows * kRowBytes;
constexpr int kMaxStages = 8;
constexpr int kPrefetchSteps = 4;                // of B that L2 is asked for while the predecessor ends
constexpr int kMmaSteps = kRowBytes / 32;        // instructions per stage
constexpr int kPolls = kWaitPolls;               // polls of one wait before it gives up
constexpr int kEpilogueWarps = 8;                 // of gemm_pair_kernel
constexpr int kSplitThreads = 256, kAlignThreads = 256, kPairThreads = 64 + 32 * kEpilogueWarps;
constexpr int kSplitBand = 16, kPairBand = 8;    // tiles along n that run side by side
constexpr int kAccumulators = 2;                 // of gemm_pair_kernel
constexpr int kAccumulatorColumns = 256;

struct GemmParams {
  CUtensorMap map_b, map_a;
  void *C;
  int64_t ldc, ldr;
  int32_t m, n;
  int32_t steps;              // 128-byte steps of k
  int32_t cols;               // columns (vectors) per tile
  int32_t tiles_n, tiles_m;   // tiles along n and along m
  int32_t stages;
  int32_t splits;             // CTAs that share a tile's k
  float alpha, beta;
  const float *scale_a, *scale_b;
  const void *bias, *residual;
  int32_t bias_f32, act, out_type;
  int32_t pairs;              // 16-bit rows of C start on 4-byte boundaries
  uint32_t idesc;             // without the column count
  int32_t polls;              // of the waits for operands
  uint32_t *timeouts;
};

// Rows of B that start off 16 bytes, read in place: the rows j, j + classes, ..
// start at one offset within their 16 bytes, and one tensor map, based on the
// 16-byte boundary before row j, reads them.  A tile takes rows of one class,
// and the vectors come with as many zeros in front (a copy for each class).
constexpr int kMaxClasses = 16;
struct ShiftedParams : GemmParams {
  CUtensorMap map_class[kMaxClasses];
  int32_t classes;
  uint32_t base, pitch;       // of B's rows, in bytes modulo 16
};
template <bool SHIFTED>
struct SplitParams {
  typedef GemmParams type;
};
template <>
struct SplitParams<true> {
  typedef ShiftedParams type;
};

// ------------------------------------------------------------------ epilogue --

__device__ __forceinline__ float load_typed(const void *p, int64_t i, int type) {
  if (type == GEMV_TYPE_F32) return static_cast<const float *>(p)[i];
  const uint16_t v = static_cast<const uint16_t *>(p)[i];
  return type == GEMV_TYPE_F16 ? F16::to_float(v) : BF16::to_float(v);
}

template <int ACT>
__device__ __forceinline__ float activated(float y) {
  if (ACT == GEMV_ACT_RELU) return y != y ? y : fmaxf(y, 0.f);
  // __fdividef: 2 ulp; a denominator above 2^126 gives 0, where the sigmoid is below
  // 1.2e-38 and the silu within 1.1e-36 of 0
  if (ACT == GEMV_ACT_SIGMOID) return __fdividef(1.f, 1.f + expf(-y));
  if (ACT == GEMV_ACT_SILU) return __fdividef(y, 1.f + expf(-y));
  if (ACT == GEMV_ACT_LOG_SIGMOID) return fminf(y, 0.f) - log1pf(expf(-fabsf(y)));
  return y;
}
// A value that the compiler keeps in a register: what the epilogue asks for in
// every turn (a load and a branch on a kernel parameter took about 25 cycles
// each, half of the epilogue's time).
template <class T>
__device__ __forceinline__ T in_register(T v) {
  asm volatile("" : "+r"(v));
  return v;
}
template <class T>
__device__ __forceinline__ T *in_register(T *v) {
  asm volatile("" : "+l"(v));
  return v;
}

// The activation of a launch: the loops over an epilogue's columns are compiled
// for each.
template <int ACT>
struct Activation {};

// The epilogue of one launch, and of one thread's column j of C.  Pairs read the
// residual a block ahead (fetch()): in its turn 7656 x 8486 x 512 e4m3 took 164 us,
// so 135.  With one tile per CTA that gains less (959 x 960 x 8576 fp16 30 -> 27) and
// costs calls without a residual its registers and start (1024 x 1024 e4m3 4.1 -> 4.5).
struct Column {
  static constexpr int kF16 = 1, kF32 = 2, kPairs = 4;  // bits of `how`
  int32_t m, how;
  uint32_t pitch, res_pitch;
  const float *scale_a;
  char *c;
  const char *res;
  bool live, odd, together;
  float factor, shift;

  __device__ __forceinline__ void init(const GemmParams &p) {
    const uint32_t es = p.out_type == GEMV_TYPE_F32 ? 4 : 2;
    m = in_register(p.m);
    how = in_register((p.out_type == GEMV_TYPE_F16 ? kF16 : p.out_type == GEMV_TYPE_F32 ? kF32 : 0) |
                      (p.pairs ? kPairs : 0));
    scale_a = in_register(p.scale_a);
    pitch = in_register((uint32_t)p.ldc * es);
    res_pitch = in_register((uint32_t)p.ldr * es);
  }

  __device__ __forceinline__ void begin(const GemmParams &p, int64_t j) {
    const uint32_t es = how & kF32 ? 4 : 2;
    live = j < p.n;
    odd = (j & 1) != 0;
    together = (how & kPairs) && __all_sync(0xffffffffu, live);
    factor = p.alpha;
    shift = 0.f;
    c = static_cast<char *>(p.C) + j * es;
    res = p.residual ? static_cast<const char *>(p.residual) + j * es : nullptr;
    if (!live) return;
    if (p.scale_b) factor *= p.scale_b[j];
    if (p.bias) shift = p.beta * load_typed(p.bias, j, p.bias_f32 ? GEMV_TYPE_F32 : p.out_type);
  }

  // Element e of rows `pitch` bytes apart.
  template <class T>
  static __device__ __forceinline__ T *row(const char *base, uint32_t pitch, int e) {
    return reinterpret_cast<T *>(const_cast<char *>(base) + (uint64_t)pitch * (uint32_t)e);
  }

  template <class Out, int COUNT, class Convert>
  __device__ __forceinline__ void store(char *at, int rows, const float (&y)[COUNT], Convert convert) const {
#pragma unroll
    for (int e = 0; e < COUNT; ++e)
      if (e < rows) *row<Out>(at, pitch, e) = convert(y[e]);
  }

  // 16-bit rows written 4 bytes per lane: lanes of even j take the even rows and
  // their odd neighbours the odd ones, after exchanging one value of each pair
  // (needs rows of C on 4-byte boundaries and every lane's column in range).
  template <int COUNT, class Pack>
  __device__ __forceinline__ void store_pairs(char *at, int rows, const float (&y)[COUNT], Pack pack) const {
    const uint32_t pick = odd ? 0x3276u : 0x5410u;  // odd: both high halves, the neighbour's first; even: both low ones
    at += odd ? (int64_t)pitch - 2 : 0;
    if (rows == COUNT) {
#pragma unroll
      for (int e = 0; e < COUNT; e += 2) {
        const uint32_t mine = pack(y[e], y[e + 1]);  // rows e (low half) and e + 1 of this column
        *row<uint32_t>(at, pitch, e) = __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
      }
    } else {
#pragma unroll
      for (int e = 0; e < COUNT; e += 2) {
        const uint32_t mine = pack(y[e], y[e + 1]);
        const uint32_t w = __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
        if (e + odd < rows) *row<uint32_t>(at, pitch, e) = w;
      }
    }
  }

  // The residual's rows i0 .. (as write() takes them), not yet converted.
  template <int COUNT>
  __device__ __forceinline__ void fetch(int i0, uint32_t (&raw)[COUNT], int most = COUNT) const {
    if (!res || !live) return;
    const int rows = m - i0 < most ? m - i0 : most;
    const char *r = res + (int64_t)i0 * res_pitch;
    if (how & kF32) {
#pragma unroll
      for (int e = 0; e < COUNT; ++e) raw[e] = e < rows ? *row<uint32_t>(r, res_pitch, e) : 0;
    } else {
#pragma unroll
      for (int e = 0; e < COUNT; ++e) raw[e] = e < rows ? *row<uint16_t>(r, res_pitch, e) : 0;
    }
  }

  // rows i0 .. of C from their sums and the residual's: as many of the COUNT as
  // there are, at most `most`
  template <int ACT, int COUNT>
  __device__ __forceinline__ void write(Activation<ACT>, int i0, const float (&sum)[COUNT], const uint32_t (&raw)[COUNT],
                                        int most = COUNT) const {
    const int rows = m - i0 < most ? m - i0 : most;
    float y[COUNT];
    if (scale_a) {
      const float *sa = scale_a + i0;
#pragma unroll
      for (int e = 0; e < COUNT; ++e) y[e] = fmaf(sum[e], factor * (e < rows ? sa[e] : 0.f), shift);
    } else {
#pragma unroll
      for (int e = 0; e < COUNT; ++e) y[e] = fmaf(sum[e], factor, shift);
    }
#pragma unroll
    for (int e = 0; e < COUNT; ++e) y[e] = activated<ACT>(y[e]);
    if (res && live) {
      if (how & kF32) {
#pragma unroll
        for (int e = 0; e < COUNT; ++e) y[e] += __uint_as_float(raw[e]);
      } else if (how & kF16) {
#pragma unroll
        for (int e = 0; e < COUNT; ++e) y[e] += F16::to_float((uint16_t)raw[e]);
      } else {
#pragma unroll
        for (int e = 0; e < COUNT; ++e) y[e] += BF16::to_float((uint16_t)raw[e]);
      }
    }
    char *at = c + (int64_t)i0 * pitch;
    if (together) {
      if (how & kF16) store_pairs(at, rows, y, [](float a, float b) { return Elem<GEMV_TYPE_F16>::pair(a, b); });
      else store_pairs(at, rows, y, [](float a, float b) { return Elem<GEMV_TYPE_BF16>::pair(a, b); });
    } else if (live) {
      if (how & kF32) store<float>(at, rows, y, [](float v) { return v; });
      else if (how & kF16) store<uint16_t>(at, rows, y, [](float v) { return F16::from_float(v); });
      else store<uint16_t>(at, rows, y, [](float v) { return BF16::from_float(v); });
    }
  }
  // The same with the residual read in its turn.
  template <int ACT, int COUNT>
  __device__ __forceinline__ void write(Activation<ACT> act, int i0, const float (&sum)[COUNT], int most = COUNT) const {
    uint32_t raw[COUNT];
    fetch(i0, raw, most);
    write(act, i0, sum, raw, most);
  }
};

// run(Activation<act>) for the launch's activation.
template <class Run>
__device__ __forceinline__ void with_activation(int act, Run run) {
  switch (act) {
    case GEMV_ACT_RELU: run(Activation<GEMV_ACT_RELU>()); break;
    case GEMV_ACT_SIGMOID: run(Activation<GEMV_ACT_SIGMOID>()); break;
    case GEMV_ACT_SILU: run(Activation<GEMV_ACT_SILU>()); break;
    case GEMV_ACT_LOG_SIGMOID: run(Activation<GEMV_ACT_LOG_SIGMOID>()); break;
    default: run(Activation<GEMV_ACT_NONE>()); break;
  }
}

// --------------------------------------------------------------------- waits --

// Tells every role of a pair's two CTAs to give up.
__device__ __forceinline__ void fail_pair(int *failed) {
  for (uint32_t r = 0; r < 2; ++r) st_cluster(cluster_address(smem_u32(failed), r), 1);
}

// The ring's position after each step.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// Whether the next stage's operands are there already: asked before this
// stage's instructions are issued, so that the answer's latency overlaps them.
__device__ __forceinline__ bool peek(const uint64_t *full, Ring r, int stages, int polls) {
  r.next(stages);
  return polls > 0 && __all_sync(0xffffffffu, mbar_test(smem_u32(&full[r.stage]), r.phase));
}

// Tile number -> tile along n and along m: bands of `band` tiles along n,
// walked along m, so that the tiles computed at one time share few operand
// rows and the L2 serves the rest of their reads.
__device__ __forceinline__ void tile_at(int t, int tiles_n, int tiles_m, int band, int *tn, int *tm) {
  if (tiles_n <= band) {  // one band
    *tm = t / tiles_n;
    *tn = t - *tm * tiles_n;
    return;
  }
  const int64_t whole = (int64_t)band * tiles_m;
  const int number = whole > t ? 0 : t / (int)whole;  // whole fits 32 bits where t reaches it
  const int first = number * band, in = t - number * (int)whole;
  const int width = tiles_n - first < band ? tiles_n - first : band;
  *tm = in / width;
  *tn = first + in - *tm * width;
}

// -------------------------------------------------------- rows off 16 bytes --

// One operand to copy: `rows` rows of `bytes` bytes, `ld` apart, to rows of
// `pitch` (a multiple of 16) in the workspace, zeros behind each row.  For each
// class (of ShiftedParams) once, with as many zeros in front as the class has
// bytes before its rows.  A row is done in `pieces` of LOADS x 512 bytes.
struct AlignJob {
  const char *src;
  char *dst;
  int64_t ld, bytes, pitch, rows, pieces, total;  // total: classes x rows x pieces
  uint32_t class_base, class_pitch;
};
struct AlignParams {
  AlignJob job[2];
  int32_t b_in_place;  // the product reads B before this kernel's end
};

// n / d for n >= 0, d > 0: in 32 bits where both fit, in a quarter of the time.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  return ((n | d) >> 32) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}

// The bytes from .. to - 1 of 16, zeros elsewhere.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int from, int to) {  // of a word
  from = from < 0 ? 0 : from;
  if (to <= from || from >= 4) return 0;
  if (to < 4) w &= (1u << (8 * to)) - 1;
  return w & ~((1u << (8 * from)) - 1);
}
__device__ __forceinline__ uint4 keep_bytes(const uint4 &v, int from, int to) {
  return make_uint4(keep_bytes(v.x, from, to), keep_bytes(v.y, from - 4, to - 4), keep_bytes(v.z, from - 8, to - 8),
                    keep_bytes(v.w, from - 12, to - 12));
}

// 16 bytes that are read once.  The operands may be what the preceding kernel
// wrote: a coherent load, in the order that the source has it, after
// wait_for_predecessor().
__device__ __forceinline__ uint4 load_once(uintptr_t at) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at)
               : "memory");
  return v;
}

// A warp copies a piece: 512 bytes of a row at a time, read as the aligned
// 16-byte blocks that hold them (a lane's upper block is its neighbour's lower
// one).  Memory-bound for B: it reads and writes the operand once.  For A's
// copies each class has warps of its own: a warp that wrote all classes' from one
// read took twice as long (8 classes of one row of 14338 bytes: 7 us, now 4).
// LOADS: 2 spread a small copy over more warps (1 x 1001 x 999 fp16 7.3 -> 6.8 us
// for the whole call), 4 keep more in flight for a large one (512 x 4099 x 7169
// 65 -> 60).
template <int LOADS>
__global__ void __launch_bounds__(kAlignThreads, 4) gemm_align_kernel(AlignParams p) {
  // A product that reads B in place may do so once it runs: not before what
  // precedes this kernel has completed.
  if (!p.b_in_place) allow_dependents();
  wait_for_predecessor();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kAlignThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kAlignThreads / 32) + (threadIdx.x >> 5); i < p.job[0].total + p.job[1].total;
       i += warps) {
    const AlignJob &j = i < p.job[0].total ? p.job[0] : p.job[1];
    const int64_t n = i < p.job[0].total ? i : i - p.job[0].total;
    const int64_t line = quotient(n, j.pieces), piece = n - line * j.pieces;
    const int64_t number = quotient(line, j.rows), row = line - number * j.rows;
    const int lead = (int)((j.class_base + (uint32_t)number * j.class_pitch) & 15);
    // byte d of the copy is byte d - lead of the row
    const uintptr_t start = (uintptr_t)(j.src + row * j.ld), end = start + (uintptr_t)j.bytes;
    const int off = (int)((start - lead) & 15);
    const int64_t d0 = piece * (LOADS * 512) + lane * 16, bytes = lead + j.bytes;
    const uintptr_t block = start - lead - off + (uintptr_t)d0;
    uint4 lo[LOADS], up[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const uintptr_t at = block + (uintptr_t)(u * 512);
      lo[u] = at < end && at + 16 > start ? load_once(at) : zero4();
      up[u] = lane == 31 && at + 16 < end && at + 32 > start ? load_once(at + 16) : zero4();
    }
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const uint4 next = make_uint4(__shfl_down_sync(0xffffffffu, lo[u].x, 1), __shfl_down_sync(0xffffffffu, lo[u].y, 1),
                                    __shfl_down_sync(0xffffffffu, lo[u].z, 1), __shfl_down_sync(0xffffffffu, lo[u].w, 1));
      uint4 v = shifted(lo[u], lane < 31 ? next : up[u], off);
      const int64_t d = d0 + u * 512;
      if (d < lead || d + 16 > bytes)  // the row's ends: zeros outside
        v = keep_bytes(v, lead - (int)(d < 16 ? d : 16), bytes - d < 16 ? (bytes - d < 0 ? 0 : (int)(bytes - d)) : 16);
      if (d < j.pitch) *reinterpret_cast<uint4 *>(j.dst + line * j.pitch + d) = v;
    }
  }
}

// ------------------------------------------------------------- split kernel --

struct alignas(16) SplitShared {
  uint64_t full[kMaxStages], empty[kMaxStages], done;
  uint32_t tmem;
  int failed;
  int issued;  // steps whose copies were started
};

// Zeros in the first `bytes` (below 16) of 16 bytes of shared memory.
__device__ __forceinline__ void clear_front(uint32_t at, int bytes) {
  uint32_t w[4];
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int clear = bytes - 4 * i;
    w[i] = clear >= 4 ? 0u : clear <= 0 ? w[i] : w[i] & ~((1u << (8 * clear)) - 1);
  }
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}

// SHIFTED: B's rows start off 16 bytes and are read in place.
template <bool E4M3, bool SHIFTED>
__global__ void __launch_bounds__(kSplitThreads)
    gemm_split_kernel(const __grid_constant__ typename SplitParams<SHIFTED>::type p) {
  extern __shared__ char dynamic[];
  __shared__ SplitShared sh;
  const uint32_t tiles = (smem_u32(dynamic) + 1023u) & ~1023u;  // swizzled tiles start on 1024 bytes
  const uint32_t stage_bytes = kTileBytes + (uint32_t)p.cols * kRowBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.splits > 1 ? (int)cluster_rank() : 0;
  int tile_n, tile_m;
  tile_at(blockIdx.x / p.splits, p.tiles_n, p.tiles_m, kSplitBand, &tile_n, &tile_m);
  int64_t j0 = (int64_t)tile_n * kTileRows;
  const int64_t i0 = (int64_t)tile_m * p.cols;
  int64_t row0 = i0;                          // of the vectors
  int number = 0, classes = 1, lead = 0;      // class of the tile's rows, bytes before them
  if constexpr (SHIFTED) {
    classes = p.classes;
    number = tile_n % classes;
    j0 = (int64_t)(tile_n / classes) * kTileRows;
    row0 += (int64_t)number * p.m;
    lead = (int)((p.base + (uint32_t)number * p.pitch) & 15);
  }
  // this CTA's share of k, whole steps, as even as they come
  const int begin = (int)((int64_t)p.steps * split / p.splits);
  int end = (int)((int64_t)p.steps * (split + 1) / p.splits);
  const CUtensorMap *map_b = &p.map_b;
  if constexpr (SHIFTED) {
    map_b = &p.map_class[number];
    if (number + classes * j0 >= p.n) end = begin;  // the class has no rows here
  }
  const uint32_t columns = p.cols <= 32 ? 32 : p.cols <= 64 ? 64 : p.cols <= 128 ? 128 : 256;

  if (threadIdx.x == 0) {
    sh.failed = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    mbar_init(smem_u32(&sh.done), 1);
    mbar_init_fence();
    if (p.steps > 0) {
      prefetch_map(map_b);
      prefetch_map(&p.map_a);
    }
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(&sh.tmem), columns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // After the allocation: a dependent kernel that started first could hold the
  // TMEM that this one waits for.
  allow_dependents();
  // The first B tiles into L2 meanwhile (they are loaded after the wait): 1 x
  // 4096 x 4096 bf16 10.2 -> 9.8 us back to back, 8 bit 7.7 -> 7.1; with 2 steps half of it.
  if (!SHIFTED && warp == 0 && elect_one())
    for (int step = begin; step < end && step - begin < kPrefetchSteps; ++step)
      tma_prefetch(map_b, step * (E4M3 ? kRowBytes : kRowBytes / 2), (int32_t)j0);
  if (!SHIFTED || warp != 0) wait_for_predecessor();

  // All warps write C: a quarter of the lanes each (the one TMEM gives them), and
  // 16 columns in turn, or with a split a few of the CTA's share.
  constexpr int kTurns = kSplitThreads / 128, kAtOnce = 4;
  const int quarter = warp & 3, turn = warp >> 2, l = quarter * 32 + lane;
  const int share = p.cols / p.splits;
  Column col;

  if (warp == 0) {
    const bool elected = elect_one();
    Ring r;
    int step = begin, ahead = begin;
    if constexpr (SHIFTED) {
      // gemm_align_kernel does not write B, and lets this kernel start once its
      // own predecessor has completed: the ring's B tiles come meanwhile.
      for (; ahead < end && ahead - begin < p.stages; ++ahead)
        if (elected) {
          mbar_expect_tx(smem_u32(&sh.full[ahead - begin]), stage_bytes);
          tma_load<1>(tiles + (ahead - begin) * stage_bytes, map_b, ahead * (E4M3 ? kRowBytes : kRowBytes / 2), (int32_t)j0,
                      smem_u32(&sh.full[ahead - begin]));
        }
      wait_for_predecessor();
    }
    for (; step < end; ++step) {
      if (step - begin >= p.stages && !wait_for<false>(smem_u32(&sh.empty[r.stage]), r.phase ^ 1, &sh.failed, kPolls)) break;
      if (elected) {
        const uint32_t bar = smem_u32(&sh.full[r.stage]), at = tiles + r.stage * stage_bytes;
        const int32_t x = step * (E4M3 ? kRowBytes : kRowBytes / 2);
        if (!SHIFTED || step >= ahead) {
          mbar_expect_tx(bar, stage_bytes);
          tma_load<1>(at, map_b, x, (int32_t)j0, bar);
        }
        tma_load<1>(at + kTileBytes, &p.map_a, x, (int32_t)row0, bar);
      }
      r.next(p.stages);
    }
    if (elected) sh.issued = step - begin;
  } else if (warp == 1) {
    const bool elected = elect_one();
    Ring r;
    const uint32_t idesc = p.idesc | ((uint32_t)(p.cols >> 3) << 17) | ((uint32_t)(kTileRows >> 4) << 24);
    bool ready = false;
    for (int step = begin; step < end; ++step) {
      if (!ready && !wait_for<false>(smem_u32(&sh.full[r.stage]), r.phase, &sh.failed, p.polls)) break;
      tc_fence_after();
      ready = peek(sh.full, r, p.stages, p.polls);
      const uint32_t at = tiles + r.stage * stage_bytes;
      const uint64_t db = tile_descriptor(at), da = tile_descriptor(at + kTileBytes);
      if (SHIFTED && step == 0 && lead > 0) {
        // what precedes the rows is not B's (and 0 x infinity would be NaN)
        for (int row = lane; row < kTileRows; row += 32)
          clear_front(at + row * kRowBytes + ((row & 7) << 4), lead);  // the swizzle's place of a row's first 16 bytes
        fence_async_smem();
        __syncwarp();
      }
      if (elected) {
#pragma unroll
        for (int s = 0; s < kMmaSteps; ++s) tc_mma<1, E4M3>(tmem, db + 2 * s, da + 2 * s, idesc, step > begin || s > 0);
        tc_commit<1>(smem_u32(&sh.empty[r.stage]));
      }
      r.next(p.stages);
    }
    // Also after a wait that gave up: the instructions issued so far read
    // shared memory until they complete.
    if (elected) tc_commit<1>(smem_u32(&sh.done));
    int none = 0;
    wait_for<false>(smem_u32(&sh.done), 0, &none, kPolls);
    if (sh.failed && elected) atomicAdd(p.timeouts, 1u);
  }
  tc_fence_before();
  __syncthreads();  // the sums are complete; shared memory is free
  tc_fence_after();
  const float nan = __int_as_float(0x7fc00000);
  const bool empty = begin == end, failed = sh.failed != 0;
  if (failed) {  // copies in flight land before their memory is used again
    if (warp == 0) {
      int none = 0;
      Ring d;
      for (int s = 0; s < sh.issued; ++s, d.next(p.stages))
        if (s + p.stages >= sh.issued && !wait_for<false>(smem_u32(&sh.full[d.stage]), d.phase, &none, kPolls) &&
            lane == 0)
          atomicOr(p.timeouts, kDrainTimeoutBit);
    }
    __syncthreads();
  }
  if (p.splits > 1) cluster_sync();

  const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16);
  if (p.splits == 1) {
    col.init(p);
    col.begin(p, number + classes * (j0 + l));
    with_activation(p.act, [&](auto act) {
#pragma unroll 1
      for (int c = turn * 16; c < p.cols && i0 + c < p.m; c += 16 * kTurns) {
        float v[16];
        tmem_load16(from + c, v);
        if (empty || failed) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = failed ? nan : 0.f;
        }
        col.write(act, (int)i0 + c, v);
      }
    });
  } else {
    // Column c goes to CTA c / share, as [source][column][lane].
    for (int c = turn * 16; c < p.cols; c += 16 * kTurns) {
      float v[16];
      tmem_load16(from + c, v);
      int to = c / share, at = c - to * share;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        st_cluster(cluster_address(tiles + (uint32_t)(((split * share + at) * kTileRows + l) * 4), to),
                   failed ? nan : empty ? 0.f : v[e]);
        if (++at == share) {
          at = 0;
          ++to;
        }
      }
    }
    cluster_sync();
    col.init(p);
    col.begin(p, number + classes * (j0 + l));
    const float *parts = reinterpret_cast<const float *>(dynamic + (tiles - smem_u32(dynamic))) + l;
    with_activation(p.act, [&](auto act) {
      const int first = (int)i0 + split * share;
#pragma unroll 1
      for (int c = turn * kAtOnce; c < share && first + c < p.m; c += kTurns * kAtOnce) {
        float v[kAtOnce] = {};
        for (int s = 0; s < p.splits; ++s) {
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e)
            if (c + e < share) v[e] += parts[(s * share + c + e) * kTileRows];
        }
        col.write(act, first + c, v, share - c);
      }
    });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<1>(tmem, columns);
  }
}

// -------------------------------------------------------------- pair kernel --

struct alignas(16) PairShared {
  uint64_t full[kMaxStages], empty[kMaxStages];      // full: the leader's count for both CTAs
  uint64_t sums[kAccumulators], free_[kAccumulators];  // accumulator complete; read by both epilogues (leader's)
  uint64_t done;
  int64_t issued;
  uint32_t tmem;
  int failed;
};

// Persistent over tiles of 256 rows of B by p.cols vectors.  CTA r of a pair
// holds rows 128 r .. 128 r + 127 of the tile's B and half of its vectors; the
// leader (r = 0) issues the instructions, which read both CTAs' shared memory
// and write each CTA's 128 rows of the accumulator to its own TMEM.
template <bool E4M3>
__global__ void __launch_bounds__(kPairThreads, 1) gemm_pair_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ char dynamic[];
  __shared__ PairShared sh;
  const uint32_t tiles = (smem_u32(dynamic) + 1023u) & ~1023u;
  const int half = p.cols / 2;
  const uint32_t stage_bytes = kTileBytes + (uint32_t)half * kRowBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int count = p.tiles_n * p.tiles_m, pairs = gridDim.x / 2, first = blockIdx.x / 2;

  if (threadIdx.x == 0) {
    sh.failed = 0;
    sh.issued = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int a = 0; a < kAccumulators; ++a) {
      mbar_init(smem_u32(&sh.sums[a]), 1);
      mbar_init(smem_u32(&sh.free_[a]), 2 * kEpilogueWarps);  // of both CTAs
    }
    mbar_init(smem_u32(&sh.done), 1);
    mbar_init_fence();
    prefetch_map(&p.map_b);
    prefetch_map(&p.map_a);
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(&sh.tmem), kAccumulators * kAccumulatorColumns);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  allow_dependents();  // after the allocation, as in gemm_split_kernel
  wait_for_predecessor();

  if (warp == 0) {
    const bool elected = elect_one();
    Ring r;
    int64_t issued = 0;
    bool ok = true;
    for (int t = first; ok && t < count; t += pairs) {
      int tn, tm;
      tile_at(t, p.tiles_n, p.tiles_m, kPairBand, &tn, &tm);
      const int32_t j0 = tn * (2 * kTileRows) + rank * kTileRows, i0 = tm * p.cols + rank * half;
      for (int step = 0; step < p.steps; ++step) {
        ok = issued < p.stages || wait_for<false>(smem_u32(&sh.empty[r.stage]), r.phase ^ 1, &sh.failed, kPolls);
        if (!ok) break;
        if (elected) {
          const uint32_t full = smem_u32(&sh.full[r.stage]), at = tiles + r.stage * stage_bytes;
          if (rank == 0) mbar_expect_tx(full, 2 * stage_bytes);
          const uint32_t bar = cluster_address(full, 0);
          const int32_t x = step * (E4M3 ? kRowBytes : kRowBytes / 2);
          tma_load<2>(at, &p.map_b, x, j0, bar);
          tma_load<2>(at + kTileBytes, &p.map_a, x, i0, bar);
        }
        ++issued;
        r.next(p.stages);
      }
    }
    if (elected) {
      sh.issued = issued;
      if (!ok) fail_pair(&sh.failed);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const bool elected = elect_one();
      Ring r;
      const uint32_t idesc = p.idesc | ((uint32_t)(p.cols >> 3) << 17) | ((uint32_t)(2 * kTileRows >> 4) << 24);
      bool ok = true, ready = false;
      int turn = 0;
      for (int t = first; ok && t < count; t += pairs, ++turn) {
        const int acc = turn & 1;
        const uint32_t d = tmem + (uint32_t)(acc * kAccumulatorColumns);
        ok = turn < kAccumulators ||
             wait_for<true>(smem_u32(&sh.free_[acc]), ((turn >> 1) & 1) ^ 1, &sh.failed, kPolls);
        tc_fence_after();
        for (int step = 0; ok && step < p.steps; ++step) {
          ok = ready || wait_for<false>(smem_u32(&sh.full[r.stage]), r.phase, &sh.failed, p.polls);
          if (!ok) break;
          tc_fence_after();
          ready = peek(sh.full, r, p.stages, p.polls);
          const uint32_t at = tiles + r.stage * stage_bytes;
          const uint64_t db = tile_descriptor(at), da = tile_descriptor(at + kTileBytes);
          if (elected) {
#pragma unroll
            for (int s = 0; s < kMmaSteps; ++s) tc_mma<2, E4M3>(d, db + 2 * s, da + 2 * s, idesc, step > 0 || s > 0);
            tc_commit<2>(smem_u32(&sh.empty[r.stage]));
          }
          r.next(p.stages);
        }
        if (ok && elected) tc_commit<2>(smem_u32(&sh.sums[acc]));
      }
      if (elected) {
        if (!ok) fail_pair(&sh.failed);
        // Also after a wait that gave up: the instructions issued so far read
        // both CTAs' shared memory until they complete.
        tc_commit<2>(smem_u32(&sh.done));
      }
    }
  } else {
    const int quarter = warp & 3, part = (warp - 2) >> 2, l = quarter * 32 + lane;
    const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16);
    Column col;
    col.init(p);
    with_activation(p.act, [&](auto act) {
      bool ok = true;
      int turn = 0;
      for (int t = first; t < count; t += pairs, ++turn) {
        const int acc = turn & 1;
        int tn, tm;
        tile_at(t, p.tiles_n, p.tiles_m, kPairBand, &tn, &tm);
        const int i0 = tm * p.cols, end = min(p.cols, p.m - i0);
        const bool residual = p.residual != nullptr;
        uint32_t raw[16];
        col.begin(p, (int64_t)tn * (2 * kTileRows) + rank * kTileRows + l);
        if (residual) col.fetch(i0 + part * 16, raw, end - part * 16);
        if (ok) {
          // a whole product: some polls for each of its steps
          ok = wait_for<false>(smem_u32(&sh.sums[acc]), (turn >> 1) & 1, &sh.failed, kPolls + 64ll * p.steps);
          if (!ok && lane == 0) fail_pair(&sh.failed);
          tc_fence_after();
        }
        const uint32_t at = from + (uint32_t)(acc * kAccumulatorColumns);
        auto turns = [&](const bool ahead) {
#pragma unroll 1
          for (int c = part * 16; c < end; c += kEpilogueWarps * 4) {
            float v[16];
            uint32_t next[16];
            if (ahead) col.fetch(i0 + c + kEpilogueWarps * 4, next, end - c - kEpilogueWarps * 4);
            tmem_load16(at + c, v);
            if (!ok) {
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __int_as_float(0x7fc00000);
            }
            if (ahead) {
              col.write(act, i0 + c, v, raw);
#pragma unroll
              for (int e = 0; e < 16; ++e) raw[e] = next[e];
            } else {
              col.write(act, i0 + c, v);
            }
          }
        };
        if (residual) turns(true);
        else turns(false);
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive_cluster(cluster_address(smem_u32(&sh.free_[acc]), 0));
      }
    });
  }
  __syncthreads();
  // Every instruction issued has completed, in both CTAs' view.
  if (warp == 1) {
    int none = 0;
    wait_for<false>(smem_u32(&sh.done), 0, &none, kPolls);
  }
  __syncthreads();
  cluster_sync();
  if (rank == 0 && warp == 0) {
    const int other_failed = ld_cluster(cluster_address(smem_u32(&sh.failed), 1));
    if (sh.failed || other_failed) {
      if (lane == 0) atomicAdd(p.timeouts, 1u);
      // Copies in flight land before the CTAs leave: the barriers of the last
      // steps are completed by what each CTA did start.
      const int64_t mine = sh.issued, other = ld_cluster64(cluster_address(smem_u32(&sh.issued), 1));
      const int64_t most = mine > other ? mine : other;
      Ring d;
      for (int64_t s = 0; s < most; ++s, d.next(p.stages)) {
        if (s + p.stages < most) continue;
        const uint32_t bar = smem_u32(&sh.full[d.stage]);
        if (lane == 0 && s >= mine) mbar_expect_tx(bar, stage_bytes);
        else if (lane == 0 && s >= other) mbar_complete_tx(bar, stage_bytes);
        int none = 0;
        if (!wait_for<false>(bar, d.phase, &none, kPolls) && lane == 0) atomicOr(p.timeouts, kDrainTimeoutBit);
      }
    }
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_free<2>(tmem, kAccumulators * kAccumulatorColumns);
}

// ---------------------------------------------------------------------- host --

// A (rows, k) operand with `ld_bytes` between rows, in boxes of 128 bytes of k
// by `box_rows` rows; what lies outside reads as zero.
bool encode(CUtensorMap *map, const void *p, int dtype, int64_t rows, int64_t k, int64_t ld_bytes, int box_rows) {
  const int es = type_bytes(dtype);
  if (rows == 1) ld_bytes = (k * es + 15) / 16 * 16;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / es), (cuuint32_t)box_rows};
  return encode_map(map, p, dtype, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool tma_ok(const void *p, int64_t rows, int64_t ld_bytes) {
  return (uintptr_t)p % 16 == 0 && (rows == 1 || (ld_bytes % 16 == 0 && ld_bytes < (1ll << 40)));
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kSmemHalf = 112 * 1024;   // dynamic shared memory that leaves room for two CTAs per SM
constexpr int kSmemAlone = 225 * 1024;  // and for one
constexpr int kMinStages = 3;

// The launch that gemm_plan() chooses.
struct GemmPlan {
  bool pair;
  int cols, tiles_m, tiles_n, splits, stages;
  int64_t smem;
  double us;  // estimated
};

// Kernel, tile width, split and ring for m x n x steps, by estimated time: the
// operands' stream at 6.2 TB/s and the waves of CTAs times their steps, the
// larger of the two and a quarter of the other, plus what a call costs besides.
// The constants are a fit to 110 shapes of both operand widths (m = 1 .. 2048,
// n x k = 1024 x 1024 .. 28672 x 8192), each measured in every form with cold
// weights (us):
//   gemm_split_kernel   0.13 + 0.00085 cols per step alone on its SM, 1.75
//                       times that with a second CTA beside it; 0.008 per
//                       column written; 3 per call, with a split 4.2 and 0.02
//                       per column exchanged
//   gemm_pair_kernel    0.286 per step of 256 columns, no less than 0.2; 6 per
//                       call
// Clusters are only taken where all run at once, with a seventh of the slots
// left for where they do not fit (256 x 28672 x 8192 bf16, 256 columns over 2
// CTAs in several waves: 121 against 94 in pairs).  Some of the shapes (bf16,
// measured): 512 x 4096 x 4096 pairs of 128 columns 18.6, of 256
// 23.0; 256 x 14336 x 4096 pairs 27.5, one tile per CTA 33.7; 256 x 1024 x 1024
// 64 columns 6.8, 256 columns 12.0.
GemmPlan gemm_plan(int64_t m, int64_t n, int64_t steps, int64_t operand_bytes, int sms, bool split_only) {
  GemmPlan best = {};
  best.us = 1e30;
  const double stream = (double)operand_bytes / 6.2e6;
  auto take = [&](GemmPlan p, double work, double call) {
    p.us = (work > stream ? work + 0.25 * stream : stream + 0.25 * work) + call;
    if (p.us < best.us) best = p;
  };
  const int64_t fewest = cdiv64(m, kAccumulatorColumns);
  for (int64_t t = fewest; t < fewest + 8; ++t) {
    GemmPlan p = {};
    p.cols = (int)(cdiv64(cdiv64(m, t), 16) * 16);
    p.tiles_m = (int)cdiv64(m, p.cols);
    p.tiles_n = (int)cdiv64(n, kTileRows);
    if (p.tiles_m < t) break;  // 16 columns already
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    const int stage = kTileBytes + p.cols * kRowBytes;
    for (int alone = 0; alone < 2; ++alone) {
      const int room = alone ? kSmemAlone : kSmemHalf;
      p.stages = (room - 1024) / stage < kMaxStages ? (room - 1024) / stage : kMaxStages;
      if (p.stages < kMinStages) continue;
      for (p.splits = 1; p.splits <= 8; p.splits *= 2) {
        if (p.splits > 1 && steps / p.splits < 4) break;
        const int64_t ctas = tiles * p.splits;
        const int64_t ring = (int64_t)p.stages * stage;
        const int64_t exchange = p.splits > 1 ? (int64_t)p.cols * kTileRows * 4 : 0;
        if (exchange > room - 1024) break;
        p.smem = (ring > exchange ? ring : exchange) + 1024;
        if (p.splits > 1 && 7 * ctas > 6 * (alone ? sms : 2 * sms)) break;
        const bool shared = !alone && ctas > sms;
        const double step = (0.13 + 0.00085 * p.cols) * (shared ? 1.75 : 1.0);
        const double waves = (double)cdiv64(ctas, shared ? 2 * sms : sms);
        const double work = waves * (cdiv64(steps, p.splits) * step + 0.008 * p.cols / p.splits);
        // a deeper ring where it costs nothing
        take(p, work, (p.splits > 1 ? 4.2 + 0.02 * p.cols : 3.0) + (alone ? 0.0 : 0.2));
      }
    }
  }
  if (steps == 0 || split_only) return best;
  for (int64_t t = fewest; t < fewest + 4; ++t) {
    GemmPlan p = {};
    p.pair = true;
    p.splits = 1;
    p.cols = (int)(cdiv64(cdiv64(m, t), 32) * 32);
    p.tiles_m = (int)cdiv64(m, p.cols);
    p.tiles_n = (int)cdiv64(n, 2 * kTileRows);
    if (p.tiles_m < t) break;
    const int stage = kTileBytes + p.cols / 2 * kRowBytes;
    p.stages = (kSmemAlone - 1024) / stage < kMaxStages ? (kSmemAlone - 1024) / stage : kMaxStages;
    p.smem = (int64_t)p.stages * stage + 1024;
    const double step = 0.286 * p.cols / 256 > 0.2 ? 0.286 * p.cols / 256 : 0.2;
    const double work = (double)cdiv64((int64_t)p.tiles_m * p.tiles_n, sms / 2) * steps * step;
    take(p, work, 6.0);
  }
  return best;
}

}  // namespace
}  // namespace gemvk

using namespace gemvk;

namespace {

int64_t aligned_pitch(int64_t k_bytes) { return (k_bytes + 15) / 16 * 16; }

// B off 16 bytes, read in place (ShiftedParams): the row classes, and the copies
// of A that they take.
struct Shifted {
  int classes;      // 0: B is aligned, or is copied
  int lead;         // the most bytes before a class's rows
  int64_t pitch;    // of A's copies
};

// In place where reading B twice and writing it once costs more than the copies
// of A, the rows of C written 16 bytes apart and each class's last tile.  Measured
// with cold weights, in place / copied (us): fp16 n x k = 4099 x 7169, m = 1 16 / 33,
// 77 22 / 39, 256 54 / 69, 512 80 / 60; 18433 x 4095, m = 1 30 / 72, 128 44 / 83,
// 256 65 / 84, 512 127 / 106; 1001 x 999, m = 1 6.8 / 7.9, 128 10.8 / 8.9.  8 bits (twice the
// classes, half the copy): 4099 x 7169, m = 1 15 / 20, 77 20 / 23, 128 31 / 27;
// 18433 x 4095, m = 16 20 / 35, 77 38 / 41, 128 43 / 42, 256 88 / 43.
Shifted shifted_rows(const void *B, int64_t n, int64_t ldb_bytes, int64_t m, int64_t k, int es) {
  const int64_t k_bytes = k * es;
  Shifted s = {};
  if (n == 0 || k_bytes == 0 || tma_ok(B, n, ldb_bytes)) return s;
  int classes = 1;
  while (n > 1 && ldb_bytes * classes % 16 != 0) classes *= 2;
  if (n * k_bytes < (1 << 20) || classes * m > n || classes * m > 1280 * es) return s;
  if (ldb_bytes * classes >= (1ll << 40) || m * classes > INT32_MAX) return s;
  s.classes = classes;
  for (int j = 0; j < classes; ++j) {
    const int lead = (int)(((uintptr_t)B + (uintptr_t)(j * ldb_bytes)) & 15);
    if (lead > s.lead) s.lead = lead;
  }
  s.pitch = aligned_pitch(s.lead + k_bytes);
  return s;
}

// Workspace for one operand: 0 where TMA reads it in place.
int64_t operand_space(const void *p, int64_t rows, int64_t k_bytes, int64_t ld_bytes) {
  if (rows == 0 || k_bytes == 0 || tma_ok(p, rows, ld_bytes)) return 0;
  return (rows * aligned_pitch(k_bytes) + 255) / 256 * 256;
}

// The copies of unaligned operands that come before a product.
struct GemmCopies {
  AlignParams p;
  int64_t blocks;  // 0: none
  int loads;
};

// The copies and the product, once nothing but the launches can fail.
template <class P>
int launch_gemm(void (*fn)(P), const P &p, int64_t grid, const GemmPlan &plan, const GemmCopies &copies,
                cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlone);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_failure((int)e);
  }
  if (copies.blocks > 0) {
    const int st = launch_op(copies.loads == 4 ? gemm_align_kernel<4> : gemm_align_kernel<2>,
                             dim3((unsigned)copies.blocks), kAlignThreads, 0, 1, stream, copies.p);
    if (st != GEMV_OK) return st;
  }
  return launch_op(fn, dim3((unsigned)grid), plan.pair ? kPairThreads : kSplitThreads, (size_t)plan.smem,
                   plan.pair ? 2 : plan.splits, stream, p);
}

int64_t workspace_of(const Shifted &s, const void *B, int64_t ldb_bytes, const void *A, int64_t lda_bytes, int64_t m,
                     int64_t n, int64_t k_bytes) {
  if (s.classes) return (s.classes * m * s.pitch + 255) / 256 * 256;
  return operand_space(B, n, k_bytes, ldb_bytes) + operand_space(A, m, k_bytes, lda_bytes);
}

int check_sizes(int64_t ldb, int64_t lda, int64_t m, int64_t n, int64_t k, int dtype) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_E4M3) return GEMV_ERR_DTYPE;
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > INT32_MAX || k > INT32_MAX) return GEMV_ERR_ARG;
  if (ldb < k || lda < k || !span_fits(n, ldb) || !span_fits(m, lda)) return GEMV_ERR_ARG;
  return GEMV_OK;
}

}  // namespace

extern "C" int gemm_workspace(const void *B, int64_t ldb, const void *A, int64_t lda, int64_t m, int64_t n, int64_t k,
                              int dtype, int64_t *bytes) {
  const int st = check_sizes(ldb, lda, m, n, k, dtype);
  if (st != GEMV_OK) return st;
  if (bytes == nullptr) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype);
  *bytes = m == 0 || n == 0 ? 0
                            : workspace_of(shifted_rows(B, n, ldb * es, m, k, es), B, ldb * es, A, lda * es, m, n, k * es);
  return GEMV_OK;
}

extern "C" int gemm_fused(const void *B, int64_t ldb, const void *A, int64_t lda, void *C, int64_t ldc, int64_t m,
                          int64_t n, int64_t k, int dtype, int out_dtype, const gemm_epilogue *epilogue,
                          void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
  int st = check_sizes(ldb, lda, m, n, k, dtype);
  if (st != GEMV_OK) return st;
  if (out_dtype != GEMV_TYPE_F32 && out_dtype != GEMV_TYPE_F16 && out_dtype != GEMV_TYPE_BF16) return GEMV_ERR_DTYPE;
  if (dtype != GEMV_TYPE_E4M3 && out_dtype != dtype && out_dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (ldc < n || !span_fits(m, ldc)) return GEMV_ERR_ARG;
  gemm_epilogue ep = {};
  ep.alpha = 1.f;
  if (epilogue != nullptr) ep = *epilogue;
  if (!ep.residual) ep.ldr = n;  // means nothing then
  if (ep.activation < GEMV_ACT_NONE || ep.activation > GEMV_ACT_LOG_SIGMOID) return GEMV_ERR_ARG;
  if (ep.bias && ep.bias_dtype != GEMV_TYPE_F32 && ep.bias_dtype != out_dtype) return GEMV_ERR_ARG;
  if (ep.residual && (ep.ldr < n || !span_fits(m, ep.ldr))) return GEMV_ERR_ARG;
  if (m == 0 || n == 0) return GEMV_OK;
  if (!C || (k > 0 && (!A || !B))) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype), oe = type_bytes(out_dtype);
  if (m > 1 && (ldc > ep.ldr ? ldc : ep.ldr) * oe > (int64_t)UINT32_MAX) return GEMV_ERR_ARG;
  const int be = ep.bias && ep.bias_dtype == GEMV_TYPE_F32 ? 4 : oe;
  if (k > 0 && ((uintptr_t)A | (uintptr_t)B) % (uintptr_t)es) return GEMV_ERR_ALIGN;
  if (((uintptr_t)C | (uintptr_t)ep.residual) % (uintptr_t)oe || (uintptr_t)ep.bias % (uintptr_t)be ||
      ((uintptr_t)ep.scale_a | (uintptr_t)ep.scale_b) % 4u)
    return GEMV_ERR_ALIGN;
  const Shifted shift = shifted_rows(B, n, ldb * es, m, k, es);
  const int64_t space = workspace_of(shift, B, ldb * es, A, lda * es, m, n, k * es);
  if (space > 0) {
    if (workspace == nullptr || workspace_bytes < space) return GEMV_ERR_SCRATCH;
    if ((uintptr_t)workspace % 16u) return GEMV_ERR_ALIGN;
  } else {
    workspace = nullptr;
  }
  const Rows RC{C, m, n * oe, ldc * oe}, RR{ep.residual, m, n * oe, ep.ldr * oe}, RW{workspace, 1, space, space};
  const Rows inputs[] = {{k > 0 ? A : nullptr, m, k * es, lda * es}, {k > 0 ? B : nullptr, n, k * es, ldb * es},
                         {ep.bias, 1, n * be, n * be}, {ep.scale_a, 1, m * 4, m * 4}, {ep.scale_b, 1, n * 4, n * 4}};
  for (const Rows &r : inputs)
    if (rows_overlap(RC, r) || rows_overlap(RW, r)) return GEMV_ERR_ALIAS;
  if (rows_overlap(RW, RC) || rows_overlap(RW, RR)) return GEMV_ERR_ALIAS;
  if (rows_overlap(RC, RR) && !(ep.residual == C && ep.ldr == ldc)) return GEMV_ERR_ALIAS;
  int dev = -1, sms = 0;
  st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {k > 0 ? A : nullptr, k > 0 ? B : nullptr, C, ep.scale_a, ep.scale_b, ep.bias, ep.residual,
                       workspace}))
    return GEMV_ERR_DEVICE;
  if (m == 1) ldc = ep.ldr = n;
  ShiftedParams p = {};
  p.C = C;
  p.ldc = ldc; p.ldr = ep.ldr;
  p.m = (int32_t)m; p.n = (int32_t)n;
  p.steps = (int32_t)cdiv64(shift.lead + k * es, kRowBytes);
  p.alpha = ep.alpha; p.beta = ep.beta;
  p.scale_a = ep.scale_a; p.scale_b = ep.scale_b; p.bias = ep.bias; p.residual = ep.residual;
  p.bias_f32 = ep.bias_dtype == GEMV_TYPE_F32 ? 1 : 0;
  p.act = ep.activation; p.out_type = out_dtype;
  p.pairs = oe == 2 && shift.classes <= 1 && ((uintptr_t)C | (uintptr_t)(ldc * oe)) % 4 == 0 ? 1 : 0;
  // fp32 accumulators (bit 4); operand types in bits 7 and 10: 0 fp16 or e4m3, 1 bf16
  p.idesc = (1u << 4) | (dtype == GEMV_TYPE_BF16 ? (1u << 7) | (1u << 10) : 0u);
  p.polls = take_wait_budget(kPolls);
  st = wait_counter(dev, &p.timeouts);
  if (st != GEMV_OK) return st;
  const bool e4m3 = dtype == GEMV_TYPE_E4M3;
  // rows of B as tiles hold them: each class ends in a tile of its own
  const int64_t tiled = shift.classes ? shift.classes * cdiv64(cdiv64(n, shift.classes), kTileRows) * kTileRows : n;
  const GemmPlan plan = gemm_plan(m, tiled, p.steps, (m + n) * k * es, sms, shift.classes != 0);
  const bool pair = plan.pair;
  p.cols = plan.cols; p.tiles_m = plan.tiles_m; p.tiles_n = plan.tiles_n;
  p.splits = plan.splits; p.stages = plan.stages;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles * p.splits > INT32_MAX / 2) return GEMV_ERR_ARG;
  p.classes = shift.classes;
  p.base = (uint32_t)(uintptr_t)B & 15;
  p.pitch = (uint32_t)(ldb * es) & 15;
  // operands that TMA cannot read in place, copied with rows that it can
  int64_t ldb_bytes = ldb * es, lda_bytes = lda * es;
  GemmCopies copies = {};
  if (space > 0) {
    AlignParams &ap = copies.p;
    char *to = static_cast<char *>(workspace);
    int jobs = 0;
    const int loads = copies.loads = space > (16 << 20) ? 4 : 2;
    auto copy = [&](const void **from, int64_t rows, int64_t *ld, int64_t pitch, int times) {
      AlignJob &job = ap.job[jobs++];
      job = {static_cast<const char *>(*from), to, *ld, k * es, pitch, rows, cdiv64(pitch, loads * 512), 0, 0, 0};
      job.total = times * rows * job.pieces;
      if (shift.classes) {
        job.class_base = p.base;
        job.class_pitch = p.pitch;
      }
      *from = to;
      *ld = pitch;
      to += (times * rows * pitch + 255) / 256 * 256;
    };
    if (shift.classes) {
      copy(&A, m, &lda_bytes, shift.pitch, shift.classes);
    } else {
      if (operand_space(B, n, k * es, ldb_bytes)) copy(&B, n, &ldb_bytes, aligned_pitch(k * es), 1);
      if (operand_space(A, m, k * es, lda_bytes)) copy(&A, m, &lda_bytes, aligned_pitch(k * es), 1);
    }
    const int64_t blocks = cdiv64(ap.job[0].total + ap.job[1].total, kAlignThreads / 32);
    ap.b_in_place = shift.classes ? 1 : 0;
    copies.blocks = blocks < 64ll * sms ? blocks : 64ll * sms;
  }
  bool mapped = true;
  if (shift.classes) {
    for (int j = 0; j < shift.classes; ++j) {
      const char *row = static_cast<const char *>(B) + j * ldb_bytes;
      const int lead = (int)((uintptr_t)row & 15);
      mapped = mapped && encode(&p.map_class[j], row - lead, dtype, cdiv64(n - j, shift.classes), k + lead / es,
                                ldb_bytes * shift.classes, kTileRows);
    }
    mapped = mapped && encode(&p.map_a, A, dtype, m * shift.classes, shift.pitch / es, lda_bytes, p.cols);
  } else if (k > 0) {
    mapped = encode(&p.map_b, B, dtype, n, k, ldb_bytes, kTileRows) &&
             encode(&p.map_a, A, dtype, m, k, lda_bytes, pair ? p.cols / 2 : p.cols);
  }
  if (!mapped) return cuda_failure((int)cudaErrorNotSupported);
  int64_t grid = tiles * p.splits;
  if (pair) grid = 2 * (tiles < sms / 2 ? tiles : sms / 2);
  if (shift.classes)
    return launch_gemm(e4m3 ? gemm_split_kernel<true, true> : gemm_split_kernel<false, true>, p, grid, plan, copies, stream);
  if (pair)
    return launch_gemm<GemmParams>(e4m3 ? gemm_pair_kernel<true> : gemm_pair_kernel<false>, p, grid, plan, copies, stream);
  return launch_gemm<GemmParams>(e4m3 ? gemm_split_kernel<true, false> : gemm_split_kernel<false, false>, p, grid, plan,
                                 copies, stream);
}
