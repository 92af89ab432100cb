// moe_product.cu -- the experts' products on the fifth-generation tensor cores.
//
// Rank's rows are sorted by expert; with R_e the rows of expert e,
//   forward      y[R_e]  = x[R_e] w_e^T     out[row][n] = sum_k w[e][n][k] x[row][k]
//   grad_input   dx[R_e] = dy[R_e] w_e      out[row][k] = sum_n w[e][n][k] dy[row][n]
//   grad_weight  dw_e    = dy[R_e]^T x[R_e] out[n][k]   = sum_row x[row][k] dy[row][n]
// One kernel computes all three as D[m][c] = sum_q A[m][q] B[c][q], with m the
// output's contiguous axis (a TMEM lane per m, so a warp's stores are
// contiguous whatever the alignment) and c the rows (or n): the tensor core's
// N, which may be any multiple of 32.  An expert's rows are cut into equal
// tiles of at most 256, so a ragged expert wastes less than 32 columns, and a
// handful of rows costs a handful of columns: the weights' stream bounds it.
//
// A pair of CTAs (one cluster) owns a 256 x 256 tile at a time, a persistent
// grid of one pair per two SMs: each CTA stages 128 rows of A and half of B's
// columns (tcgen05.mma.cta_group::2 reads both halves, which halves shared
// memory traffic for B), in stages of 64 contraction elements.  Roles by warp:
//   0-7  epilogue: TMEM -> registers -> global, double buffered (2 x 256
//        columns) against the next tile's products
//   8    TMA: one thread issues the stage's bulk tensor copies
//   9    MMA: one thread of the even CTA issues for the pair
//   10-  loaders: what TMA cannot do -- operands that do not sit on 16 bytes
//        (16 warps), by whole 16-byte loads, shifted and masked; and
//        grad_weight's last rows, which must read as zero where the next
//        expert begins (2 warps of them clear those where TMA reads the rest)
// Every wait is bounded: one that runs out sets the device error word.
//
// Measured on bf16 operands (one GB300; 1944 TFLOP/s is the library's rate on
// one large product in a burst, 6.78 TB/s a copy's):
//   32 experts x 1024 rows, 2048 <- 7168: forward 525 us (1.83 PFLOP/s), input
//     gradient 530, fp32 weight gradient 650.  The tensor pipe bounds the first
//     two (92 % of cycles).  The last takes 532 without its 1.9 GB of stores,
//     which delay the loads; a quarter fewer loads gained 4 %, and tiles of two
//     or four experts under way at a time lost 5 %.  bf16 weight gradient 590.
//   32 experts x 512 rows: weight gradient 415 us, bf16 355; without rows, 1.9 GB
//     of zeros, 287 us (6.5 TB/s).
//   32 experts x 4 rows on average, the weights' stream: 153 us, 6.2 TB/s.
//   operands off the grid (2047 x 7167): 3.3 ms forward, 2.5 ms backward; the
//     loaders' instructions bound them.
//   1 expert of 66 columns by 5376 contraction elements: 25 us, 84 stages one
//     behind the other in a single pair.
#include <cuda.h>  // CUtensorMap and its enums; nothing links the driver

#include <atomic>
#include <climits>

#include "device_common.cuh"
#include "realign.cuh"

namespace ccl {
namespace {

constexpr int kTile = 256;         // outputs per pair: 256 x at most 256
constexpr int kStep = 64;          // contraction elements per stage (128 bytes: one swizzle row)
constexpr int kStages = 6;
constexpr int kOperandBytes = 128 * kStep * 2;  // one CTA's share of A or B in a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMaxGroups = 2048;   // (rank, expert) pairs per launch
constexpr int kLaunchRanks = 8;    // keeps the parameter block under 4 KB
constexpr int kEpilogueWarps = 8;  // two per 32 TMEM lanes
constexpr int kTmaWarp = kEpilogueWarps, kMmaWarp = kTmaWarp + 1, kLoaderWarp = kMmaWarp + 1;
// REGS (fp32 weight gradients, see kMostF32): the epilogue's threads hold
// 128 running sums each, for which the other warps give registers up; TMA
// reads both operands, so that two warps are enough to clear last rows.
// The shares add up to what the block is launched with.
template <bool REGS>
struct Crew {
  static constexpr int kLoaders = REGS ? 64 : 512;  // loader threads
  static constexpr int kThreads = kLoaderWarp * 32 + kLoaders;
  static constexpr int kLaunchRegs = 168, kEpilogueRegs = 216, kOtherRegs = 72;  // a thread
  static_assert(!REGS || (kEpilogueWarps * 32 * kEpilogueRegs + (kThreads - kEpilogueWarps * 32) * kOtherRegs == kThreads * kLaunchRegs &&
                          kThreads % 128 == 0 && kThreads * kLaunchRegs <= 65536),
                "register shares");
};
constexpr int kSmallBox = 16;      // rows of B's small box
constexpr uint32_t kTmemColumns = 512;
// The tensor core cuts its fp32 sums at the last bit instead of rounding them,
// towards zero, once per 16 contraction elements: 1e-6 of the result after
// 1024 of them, 1.9e-5 after 16384, and so on, where rounded sums stay at 2e-7
// to 4e-7.  So long sums are made in parts, which the epilogue adds up, rounded.
// fp32 outputs, the weight gradients: parts of at most so many rows (5e-7), added
// up in registers, or, where loaders fill the stages and set the pace, in the
// output (32 experts of 1024 rows by TMA took 948 us that way, 650 in registers).
constexpr int kMostF32 = 512;
// bf16 outputs round to 4e-3 and hide 1.9e-5, but not what a million rows would
// come to, always towards zero: parts of at most so many, added up in tensor
// memory.  The first part stays in its buffer and the others take turns in the
// other one, so that the tensor core waits while each of them is added (8 experts
// of 1024 rows, 2048 <- 32768: 641 -> 647 us).
constexpr int kMostBF16 = 16384;
// Two seconds without a stage: a wait for a whole tile, or for the next stage
// that the loaders have a part in, may take any number of stages (10^9 rows of
// one expert are 16 million: five seconds), so it runs out only where no stage
// was issued for so long.
constexpr long long kWaitCycles = 1ll << 32;

__device__ unsigned int g_product_error;  // nonzero: a bounded wait ran out
std::atomic<bool> g_launched{false};      // in this process; never taken back, since a captured graph may run at any time

struct PairArgs {
  CUtensorMap a[kLaunchRanks], b[kLaunchRanks], b_small[kLaunchRanks];
  const void* pa[kLaunchRanks];
  const void* pb[kLaunchRanks];
  void* out[kLaunchRanks];
  const int32_t* offsets[kLaunchRanks];
  uint32_t rows[kLaunchRanks];
  uint32_t n, contract;
  int p, num_experts;
  int tma_a, tma_b;
  int whole_a, whole_b;  // the operand's contiguous axis is whole chunks of 64: both of a stage in one copy
};
static_assert(sizeof(PairArgs) <= 4096, "product parameters exceed 4 KB");

// What a waiting warp looks at.
struct Watch {
  uint32_t dead;      // a wait of the CTA ran out
  uint32_t progress;  // stages that its TMA warp has issued
};
struct Shared {
  alignas(8) uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t go[kStages];  // to the loaders: the stage is free to fill, or its last rows have landed
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint32_t tmem;
  Watch watch;
  uint32_t scan[Crew<false>::kThreads / 32];
  uint32_t first[kMaxGroups + 1];  // row tiles before each (rank, expert)
  int32_t lo[kMaxGroups];          // its first row
  int32_t count[kMaxGroups];       // and its rows
};
constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(kStages) * kStageBytes + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "product shared memory");

// ------------------------------------------------------------------ barriers
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// On a barrier of either CTA of the pair.  Released to it is what lies in this
// CTA's shared memory: what the loaders have written, behind a proxy fence of the
// writers and a barrier among them; the epilogue has read tensor memory, which its
// own fence orders.  Only that: a release at cluster scope of all of a thread's
// memory takes 700 ns, a loader's with its loads on the way a microsecond, the
// epilogue's with its stores longer (fp32 weight gradients of 32 experts of 512
// rows 489 us instead of 437).
__device__ __forceinline__ void mbar_arrive(uint32_t cluster_bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive_own(uint32_t bar, uint32_t count = 1) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(done)
               : "r"(bar), "r"(parity)
               : "memory");
  return done != 0;
}
// False once this or another wait of the CTA ran out.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile Watch* watch, long long cycles = kWaitCycles) {
  if (mbar_try(bar, parity)) return true;
  long long t0 = clock64();
  uint32_t seen = watch->progress;
  while (!mbar_try(bar, parity)) {
    if (watch->dead) return false;
    if (clock64() - t0 <= cycles) continue;
    const uint32_t now = watch->progress;
    if (now == seen) {
      watch->dead = 1;
      atomicExch(&g_product_error, kProductError);
      return false;
    }
    seen = now;
    t0 = clock64();
  }
  return true;
}

// ------------------------------------------------------------ tensor memory
__device__ __forceinline__ uint64_t descriptor(uint32_t addr, uint32_t lead_bytes) {
  // 128-byte swizzle; 1024 bytes between groups of 8 lines
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(lead_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tma(uint32_t dst, const CUtensorMap* map, int x, int line, int chunk, int z, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
      "%4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(line), "r"(chunk), "r"(z), "r"(cluster_bar)
      : "memory");
}

// One lane of the warp, the same for every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}

// A place in the ring of stages and the parity of the pass over it.
struct Ring {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// -------------------------------------------------------------------- tiles
struct Tile {
  int rank, expert;
  int lo;       // first row of the expert
  int depth;    // contraction elements
  int segment;  // of them per part of the sum: a multiple of kStep, or depth
  int c0;       // first column: a row of the rank, or an n
  int cols;     // columns that are stored
  int width;    // columns that are computed: a multiple of 32
  int m0;       // first m of the pair
};

// The same value in every lane, and known to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Sums of more than MOST contraction elements are made in parts.
template <int KIND, int MOST>
__device__ __forceinline__ Tile tile_at(const PairArgs& a, const Shared& s, int groups, uint32_t index, uint32_t mt) {
  const uint32_t rt = index / mt;
  Tile t;
  t.m0 = static_cast<int>(index - rt * mt) * kTile;
  int g;
  if constexpr (KIND == kProductGradWeight) {
    const uint32_t nt = (a.n + kTile - 1) / kTile;
    g = static_cast<int>(rt / nt);
    t.lo = uniform(s.lo[g]);
    t.c0 = static_cast<int>(rt - g * nt) * kTile;
    t.cols = min(kTile, static_cast<int>(a.n) - t.c0);
    t.depth = uniform(s.count[g]);
  } else {
    int lo = 0, hi = groups - 1;  // the last group that begins at or before rt
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.first[mid] <= rt) lo = mid;
      else hi = mid - 1;
    }
    g = uniform(lo);
    t.lo = uniform(s.lo[g]);
    const int rows = uniform(s.count[g]), tiles = (rows + kTile - 1) / kTile;
    const int each = ((rows + tiles - 1) / tiles + 31) & ~31;
    const int at = static_cast<int>(rt - uniform(s.first[g])) * each;
    t.c0 = t.lo + at;
    t.cols = min(each, rows - at);
    t.depth = static_cast<int>(KIND == kProductForward ? a.contract : a.n);
  }
  t.rank = g / a.num_experts;
  t.expert = g - t.rank * a.num_experts;
  t.width = (t.cols + 31) & ~31;
  t.segment = t.depth;
  if (t.depth > MOST) {
    const int parts = (t.depth - 1) / MOST + 1;
    t.segment = ((t.depth - 1) / parts + kStep) / kStep * kStep;
  }
  return t;
}

// ------------------------------------------------------------------ loaders
// `v` with the elements from `valid` on zero.
__device__ __forceinline__ uint4 keep(const uint4 v, int valid) {
  uint32_t o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = 2 * i + 1 < valid ? o[i] : 2 * i < valid ? (o[i] & 0xFFFFu) : 0u;
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A barrier among the loaders, and whether any of them says so.
template <int THREADS>
__device__ __forceinline__ bool any_loader(bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "n"(THREADS)
      : "memory");
  return r != 0;
}

// What a loader thread fetches of an operand's share of a stage: unit u (8
// elements) of lines l0 and l0 + 64, of 64 elements each.  COLUMNS: line l is
// contraction row l mod 64 of 64-element chunk l / 64.
template <bool COLUMNS>
struct Fetch {
  const __nv_bfloat16* p;  // unit u of line l0 in the tile's first stage
  int64_t apart;           // elements from there to line l0 + 64
  int extent;              // COLUMNS: elements of the row from the unit on; else lines from l0 on
};
// 16-byte granules in flight: the lower and the upper one of each unit.
struct Units {
  uint4 lo[2], hi[2];
  int phase[2], valid[2];  // bytes of the lower one before the unit; elements
};
template <bool COLUMNS>
__device__ __forceinline__ void fetch_units(const Fetch<COLUMNS>& f, const __nv_bfloat16* p, int left, int l0, int u, Units& v) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = COLUMNS ? (l0 < left ? f.extent - 64 * j : 0) : 64 * j < f.extent ? left - 8 * u : 0;
    v.valid[j] = min(max(n, 0), 8);
    const uintptr_t at = reinterpret_cast<uintptr_t>(p + j * f.apart), base = at & ~static_cast<uintptr_t>(15);
    v.phase[j] = static_cast<int>(at - base);
    v.lo[j] = load16_if(base, v.valid[j] > 0);
    v.hi[j] = load16_if(base + 16, v.valid[j] > 0 && v.phase[j] + 2 * v.valid[j] > 16);
  }
}
__device__ __forceinline__ void put_units(char* dst, int lines, int l0, int u, const Units& v) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int l = l0 + 64 * j;
    if (l >= lines) continue;
    uint4 x = shift16(v.lo[j], v.hi[j], v.phase[j]);
    if (v.valid[j] < 8) x = keep(x, v.valid[j]);
    *reinterpret_cast<uint4*>(dst + l * 128 + ((u ^ (l & 7)) << 4)) = x;
  }
}

// Zeros in the lines of contraction rows from `left` on: line l holds row l mod 64.
__device__ __forceinline__ void clear_lines(char* dst, int lines, int left, int tid, int threads) {
  for (int i = tid; i < lines * 8; i += threads)
    if (((i >> 3) & 63) >= left) *reinterpret_cast<uint4*>(dst + i * 16) = make_uint4(0, 0, 0, 0);
}

// ----------------------------------------------------------------- epilogue
// This lane's column of the tile in 32 rows of the output, `ld` bytes apart:
// v[j] goes to p + j * ld while j < count.  `even` (bf16): neighbouring lanes
// swap halves of two rows, so that the even lane holds two outputs of row j
// and the odd one two of row j + 1, and half as many stores carry them.
template <int OUT, bool ALL>
__device__ __forceinline__ void store_rows(char* p, uint64_t ld, const uint32_t* v, int count, bool live, bool even) {
  if constexpr (OUT == kF32) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (live && (ALL || j < count)) st_stream4(p + j * ld, v[j]);
  } else {
    const int odd = threadIdx.x & 1;
    if (even) {
      p += odd * (ld - 2);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        const uint32_t mine = *reinterpret_cast<const uint32_t*>(&h);
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
        const uint32_t both = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
        if (live && (ALL || j + odd < count)) *reinterpret_cast<uint32_t*>(p + j * ld) = both;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (live && (ALL || j < count)) *reinterpret_cast<__nv_bfloat16*>(p + j * ld) = __float2bfloat16_rn(__uint_as_float(v[j]));
    }
  }
}
template <int OUT>
__device__ __forceinline__ void store_columns(char* p, uint64_t ld, const uint32_t* v, int count, bool live, bool even) {
  if (count >= 32) store_rows<OUT, true>(p, ld, v, count, live, even);
  else store_rows<OUT, false>(p, ld, v, count, live, even);
}

// As store_rows<kF32>, added to what the thread itself has stored there.
__device__ __forceinline__ void add_rows(char* p, uint64_t ld, const uint32_t* v, int count, bool live) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (live && j < count) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p + j * ld), "f"(__uint_as_float(v[j])) : "memory");
}

// Adds a part to the sum of those before it, both in tensor memory: this warp's columns.
__device__ __forceinline__ void add_part(uint32_t sum, uint32_t part, int c0, int width) {
  for (int c = c0; c < width; c += 64) {
#pragma unroll
    for (int h = 0; h < 32; h += 8) {
      uint32_t u[8], v[8];
      tmem_load8(sum + c + h, u);
      tmem_load8(part + c + h, v);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(__fadd_rn(__uint_as_float(u[j]), __uint_as_float(v[j])));
      tmem_store8(sum + c + h, u);
    }
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------------- kernel
// HELD: sums of a bf16 output may have several parts.  A variant of its own: in
// one kernel with the others, the code for it cost short sums up to 4 % (32
// experts of 512 rows, bf16 weight gradient: 358 -> 373 us).
template <int KIND, int OUT, bool REGS, bool HELD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Crew<REGS>::kThreads, 1)
    product_kernel(const __grid_constant__ PairArgs a) {
  constexpr bool kAColumns = KIND != kProductForward;     // A's contiguous axis is m
  constexpr bool kBColumns = KIND == kProductGradWeight;  // B's contiguous axis is c
  constexpr int kMost = OUT == kF32 ? kMostF32 : HELD ? kMostBF16 : INT_MAX;
  using CREW = Crew<REGS>;
  static_assert(OUT == kBF16 || kBColumns, "weight gradients alone are fp32");
  static_assert(!REGS || OUT == kF32, "parts of fp32 outputs alone are added up in registers");
  static_assert(!HELD || OUT == kBF16, "and parts of bf16 outputs in tensor memory");
  extern __shared__ char dynamic[];
  char* stages = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
  Shared& s = *reinterpret_cast<Shared*>(stages + static_cast<size_t>(kStages) * kStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cta = blockIdx.x & 1;
  const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const bool loaders = kBColumns || !a.tma_a || !a.tma_b;
  const int groups = a.p * a.num_experts;
  const uint32_t M = KIND == kProductForward ? a.n : a.contract;  // the output's contiguous axis
  const uint32_t mt = (M + kTile - 1) / kTile;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      // of the even CTA: its TMA thread, and both CTAs' loaders
      mbar_init(smem_addr(&s.full[i]), loaders ? 3 : 1);
      mbar_init(smem_addr(&s.empty[i]), 1);
      mbar_init(smem_addr(&s.go[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s.tmem_full[i]), 1);
      mbar_init(smem_addr(&s.tmem_empty[i]), 2 * kEpilogueWarps);  // the epilogue's warps of both CTAs
    }
    s.watch.dead = s.watch.progress = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_enter();

  // rows of every (rank, expert), cut to what the buffer holds, and a running
  // count of their row tiles: each thread counts a run of groups, then a scan
  {
    const int per = (groups + CREW::kThreads - 1) / CREW::kThreads;
    const int g0 = min(tid * per, groups), g1 = min(g0 + per, groups);
    uint32_t mine = 0;
    for (int g = g0; g < g1; ++g) {
      const int r = g / a.num_experts, e = g - r * a.num_experts;
      const int rows = static_cast<int>(a.rows[r]);
      const int32_t* off = a.offsets[r];
      const int lo = rows == 0 ? 0 : min(max(off[e], 0), rows);
      const int hi = rows == 0 ? 0 : min(max(off[e + 1], lo), rows);
      s.lo[g] = lo;
      s.count[g] = hi - lo;
      mine += (hi - lo + kTile - 1) / kTile;
    }
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s.scan[warp] = incl;
    __syncthreads();
    uint32_t run = incl - mine;
    for (int w = 0; w < warp; ++w) run += s.scan[w];
    for (int g = g0; g < g1; ++g) {
      s.first[g] = run;
      run += (s.count[g] + kTile - 1) / kTile;
    }
    if (tid == CREW::kThreads - 1) s.first[groups] = run;
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s.tmem;
  // 32 bits serve: 2^32 tiles of full size are 2^49 bytes of output, and at most
  // groups * 2^14 + rows / 256 are not
  const uint32_t tiles = (KIND == kProductGradWeight ? groups * ((a.n + kTile - 1) / kTile) : s.first[groups]) * mt;
  volatile Watch* watch = &s.watch;

  if (warp >= kEpilogueWarps) {
    if constexpr (REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CREW::kOtherRegs));
    if (warp == kTmaWarp) {
      // ------------------------------------------------------------------ TMA
      // The whole warp walks the stages, so that addresses and coordinates are
      // uniform; one lane issues.
      const bool issuer = elect_one();
      Ring ring;
      const uint32_t even = in_cta(smem_addr(s.full), 0);
      const uint32_t own = smem_addr(s.full), empty = smem_addr(s.empty), data = smem_addr(stages);
      uint32_t issued = 0;
      bool ok = true;
      for (uint32_t i = pair; ok && i < tiles; i += pairs) {
        const Tile t = tile_at<KIND, kMost>(a, s, groups, i, mt);
        const int half = t.width >> 1;
        const int c = t.c0 + static_cast<int>(cta) * half, m = t.m0 + static_cast<int>(cta) * 128;
        const int boxes = kBColumns ? (half + 63) / 64 : half > 64 ? 1 : (half + kSmallBox - 1) / kSmallBox;
        const uint32_t box_bytes = kBColumns ? kStep * 128 : half > 64 ? kOperandBytes : kSmallBox * 128;
        const CUtensorMap* map_a = &a.a[t.rank];
        const CUtensorMap* map_b = !kBColumns && half <= 64 ? &a.b_small[t.rank] : &a.b[t.rank];
        const CUtensorMap* map_small = &a.b_small[t.rank];
        const int z = KIND == kProductGradWeight ? 0 : t.expert;
        for (int k = 0; k < t.depth; k += kStep) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty + 8 * ring.stage, ring.phase ^ 1, watch))) {
            ok = false;
            break;
          }
          ++issued;
          if (issuer) {
            watch->progress = issued;
            // the even CTA's barrier counts both CTAs' copies; its own TMA
            // thread alone arrives, for the bytes of both
            uint32_t bar = even + 8 * ring.stage;
            const bool tail = kBColumns && k + kStep > t.depth;
            const bool do_a = a.tma_a, do_b = a.tma_b;
            const uint32_t bytes = (do_a ? kOperandBytes : 0) + (do_b ? boxes * box_bytes : 0);
            const bool loaded = tail || !do_a || !do_b;  // the loaders have a part in the stage
            const uint32_t go = smem_addr(&s.go[ring.stage]);
            if (loaded) mbar_arrive_tx(go, tail ? bytes : 0);
            if (cta == 0) {
              if (loaders && !loaded) mbar_arrive_own(own + 8 * ring.stage, 2);  // in the loaders' place
              mbar_arrive_tx(own + 8 * ring.stage, tail ? 0 : 2 * bytes);
            }
            if (tail) bar = go;  // the loaders clear what lies behind the last row
            const uint32_t sa = data + ring.stage * kStageBytes, sb = sa + kOperandBytes;
            if (do_a) {
              if constexpr (!kAColumns) {
                tma(sa, map_a, k, m, 0, z, bar);
              } else {
                const int line = KIND == kProductGradInput ? k : t.lo + k;
                if (a.whole_a) {
                  tma(sa, map_a, 0, line, m >> 6, z, bar);
                } else {
                  tma(sa, map_a, m, line, 0, z, bar);
                  tma(sa + kStep * 128, map_a, m + 64, line, 0, z, bar);
                }
              }
            }
            if (do_b) {
              if constexpr (kBColumns) {
                // of 192 columns, the odd CTA's half begins inside a chunk
                if (a.whole_b && boxes > 1 && (c & 63) == 0) {
                  tma(sb, map_b, 0, t.lo + k, c >> 6, 0, bar);
                } else {
                  tma(sb, map_small, c, t.lo + k, 0, 0, bar);
                  if (boxes > 1) tma(sb + kStep * 128, map_small, c + 64, t.lo + k, 0, 0, bar);
                }
              } else {
                tma(sb, map_b, k, c, 0, 0, bar);
                for (int q = 1; q < boxes; ++q) tma(sb + q * kSmallBox * 128, map_b, k, c + q * kSmallBox, 0, 0, bar);
              }
            }
          }
          ring.next();
        }
      }
      // every stage given back: no signal of the tensor core is on its way to a
      // CTA that has left
      for (int j = 0; ok && j < kStages; ++j, ring.next())
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + 8 * ring.stage, ring.phase ^ 1, watch));
      if (!ok) {  // copies in flight still write this CTA's shared memory
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 22)) {
        }
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------------ MMA
      if (cta == 0) {
        const bool issuer = elect_one();
        Ring ring;
        uint32_t buf = 0, uses = 0;  // the next part's buffer; a bit for each: whether it was used an odd number of times
        const uint32_t full = smem_addr(s.full), empty = smem_addr(s.empty);
        // descriptors of stage 0; a stage, and 16 contraction elements, further on
        const uint64_t a0 = descriptor(smem_addr(stages), kAColumns ? kStep * 128 : 16);
        const uint64_t b0 = descriptor(smem_addr(stages) + kOperandBytes, kBColumns ? kStep * 128 : 16);
        constexpr uint64_t kNextA = (kAColumns ? 2048 : 32) >> 4, kNextB = (kBColumns ? 2048 : 32) >> 4;
        bool ok = true;
        for (uint32_t i = pair; ok && i < tiles; i += pairs) {
          const Tile t = tile_at<KIND, kMost>(a, s, groups, i, mt);
          const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (kAColumns ? 1u << 15 : 0u) | (kBColumns ? 1u << 16 : 0u) |
                                 (static_cast<uint32_t>(t.width >> 3) << 17) | (16u << 24);
          const bool held = HELD && t.segment < t.depth;
          int k0 = 0;
          do {  // a part, also of an expert without rows
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&s.tmem_empty[buf]), ((uses >> buf) & 1) ^ 1, watch))) {
              ok = false;
              break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + buf * kTile;
            const int k1 = t.depth - k0 > t.segment ? k0 + t.segment : t.depth;
            for (int k = k0; k < k1; k += kStep) {
              const uint32_t bar = full + 8 * ring.stage;
              if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar, ring.phase, watch))) {
                ok = false;
                break;
              }
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              if (issuer) {
                const uint64_t da = a0 + ring.stage * (kStageBytes >> 4), db = b0 + ring.stage * (kStageBytes >> 4);
                const int left = k1 - k;  // contraction elements from here
                mma(d, da, db, idesc, k != k0);
                if (left > 16) mma(d, da + kNextA, db + kNextB, idesc, 1);
                if (left > 32) mma(d, da + 2 * kNextA, db + 2 * kNextB, idesc, 1);
                if (left > 48) mma(d, da + 3 * kNextA, db + 3 * kNextB, idesc, 1);
                commit_pair(empty + 8 * ring.stage);
              }
              ring.next();
            }
            if (ok && issuer) commit_pair(smem_addr(&s.tmem_full[buf]));
            __syncwarp();
            uses ^= 1u << buf;
            if (!held || k0 == 0) buf ^= 1;
            k0 = k1;
          } while (ok && k0 < t.depth);
        }
      }
    } else {
      // -------------------------------------------------------------- loaders
      if (loaders) {
        const int ltid = tid - kLoaderWarp * 32;
        Ring ring;
        // parity of each stage's next `go`.  The loaders skip stages, so they
        // could not follow `empty` by its parity: several of its phases may pass
        // between two of theirs, while `go` moves on only once they have filled.
        uint32_t parity = 0;
        bool ok = true;
        for (uint32_t i = pair; ok && i < tiles; i += pairs) {
          const Tile t = tile_at<KIND, kMost>(a, s, groups, i, mt);
          const int half = t.width >> 1;
          const int64_t c = t.c0 + static_cast<int>(cta) * half, m = t.m0 + static_cast<int>(cta) * 128;
          const int64_t N = a.n, K = a.contract, rows = a.rows[t.rank];
          const int lines_b = kBColumns ? (half + 63) & ~63 : half;
          const int l0 = ltid >> 3, u = ltid & 7;
          Fetch<kAColumns> fa;
          Fetch<kBColumns> fb;
          const int64_t ld_a = K, ld_b = KIND == kProductForward ? K : N;
          if constexpr (!REGS) {
            const __nv_bfloat16* pa = static_cast<const __nv_bfloat16*>(a.pa[t.rank]);
            const __nv_bfloat16* pb = static_cast<const __nv_bfloat16*>(a.pb[t.rank]);
            fa.apart = kAColumns ? 64 : 64 * ld_a;
            fb.apart = kBColumns ? 64 : 64 * ld_b;
            if constexpr (KIND == kProductForward) {
              fa.p = pa + (static_cast<int64_t>(t.expert) * N + m + l0) * K + 8 * u;
              fa.extent = static_cast<int>(N - m) - l0;
            } else {
              fa.p = pa + ((KIND == kProductGradInput ? static_cast<int64_t>(t.expert) * N : t.lo) + l0) * K + m + 8 * u;
              fa.extent = static_cast<int>(K - m) - 8 * u;
            }
            if constexpr (kBColumns) {
              fb.p = pb + (static_cast<int64_t>(t.lo) + l0) * N + c + 8 * u;
              fb.extent = static_cast<int>(N - c) - 8 * u;
            } else {
              fb.p = pb + (c + l0) * ld_b + 8 * u;
              fb.extent = static_cast<int>(rows - c) - l0;
            }
          }
          for (int k = 0; k < t.depth; k += kStep, ring.next()) {
            const uint32_t st = ring.stage;
            const bool tail = kBColumns && k + kStep > t.depth;
            if (a.tma_a && a.tma_b && !tail) continue;
            const int left = t.depth - k;  // contraction elements from here
            // the loads do not wait for the stage to be free
            Units va, vb;
            if constexpr (!REGS) {
              if (!a.tma_a) fetch_units<kAColumns>(fa, fa.p + (kAColumns ? k * ld_a : k), left, l0, u, va);
              if (!a.tma_b) fetch_units<kBColumns>(fb, fb.p + (kBColumns ? k * ld_b : k), left, l0, u, vb);
            }
            const bool here = mbar_wait(smem_addr(&s.go[st]), (parity >> st) & 1, watch);
            parity ^= 1u << st;
            char* sa = stages + static_cast<size_t>(st) * kStageBytes;
            char* sb = sa + kOperandBytes;
            if (here) {
              if constexpr (!REGS) {
                if (!a.tma_a) put_units(sa, 128, l0, u, va);
                if (!a.tma_b) put_units(sb, lines_b, l0, u, vb);
              }
              if (tail) {  // rows behind the expert's last: the next expert's, or nobody's
                if (a.tma_a) clear_lines(sa, 128, left, ltid, CREW::kLoaders);
                if (a.tma_b) clear_lines(sb, lines_b, left, ltid, CREW::kLoaders);
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (any_loader<CREW::kLoaders>(!here)) {  // one answer for all of them
              ok = false;
              break;
            }
            if (ltid == 0) mbar_arrive(in_cta(smem_addr(&s.full[st]), 0));
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    if constexpr (REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CREW::kEpilogueRegs));
    uint32_t buf = 0, uses = 0;  // as the tensor core's warp counts them
    bool ok = true;
    const uint32_t quarter = warp & 3;  // the 32 lanes that this warp can read
    constexpr int kBytes = Elem<OUT>::kBytes;
    for (uint32_t i = pair; ok && i < tiles; i += pairs) {
      const Tile t = tile_at<KIND, kMost>(a, s, groups, i, mt);
      const uint32_t m = t.m0 + cta * 128 + quarter * 32 + lane;
      const uint64_t at = (KIND == kProductGradWeight ? static_cast<uint64_t>(t.expert) * a.n + t.c0 : static_cast<uint64_t>(t.c0)) * M + m;
      // bf16 outputs two by two: where every row starts on four bytes
      const bool even = OUT == kBF16 && (M & 1) == 0 && (reinterpret_cast<uintptr_t>(a.out[t.rank]) & 3) == 0;
      char* out = static_cast<char*>(a.out[t.rank]) + at * kBytes;
      const uint64_t ld = static_cast<uint64_t>(M) * kBytes;
      const int c0 = (warp >> 2) * 32;  // every other 32 columns are this warp's
      float sum[REGS ? kTile / 64 : 1][32];  // this thread's columns
      if constexpr (REGS) {
#pragma unroll
        for (int q = 0; q < kTile / 64; ++q)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[q][j] = 0.0f;
      }
      const bool held = HELD && t.segment < t.depth;
      int k0 = 0;
      do {  // a part
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&s.tmem_full[buf]), (uses >> buf) & 1, watch))) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t lanes = tmem + (quarter << 21);  // lane 32 * quarter
        const uint32_t to = held && k0 > 0 ? buf ^ 1 : buf;  // where the parts are added up
        const uint32_t from = lanes + to * kTile;
        const bool last = t.depth - k0 <= t.segment;
        if constexpr (REGS) {
          if (t.depth > 0) {
#pragma unroll
            for (int q = 0; q < kTile / 64; ++q) {
              if (c0 + q * 64 < t.width) {
                uint32_t v[32];
                tmem_load32(from + c0 + q * 64, v);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[q][j] += __uint_as_float(v[j]);
              }
            }
          }
        } else {
          if (held && k0 > 0) add_part(from, lanes + buf * kTile, c0, t.width);
          for (int c = c0; c < t.width && (last || !held); c += 64) {
            uint32_t v[32];
            if (t.depth > 0) {
              tmem_load32(from + c, v);
              asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0;
            }
            char* p = out + static_cast<uint64_t>(c) * ld;
            if (OUT == kF32 && k0 > 0) add_rows(p, ld, v, t.cols - c, m < M);
            else store_columns<OUT>(p, ld, v, t.cols - c, m < M, even);
            __syncwarp();
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (!held || k0 > 0) mbar_arrive(in_cta(smem_addr(&s.tmem_empty[buf]), 0));
          if (held && last) mbar_arrive(in_cta(smem_addr(&s.tmem_empty[to]), 0));
        }
        uses ^= 1u << buf;
        if (!held || k0 == 0) buf ^= 1;
        k0 = last ? t.depth : k0 + t.segment;
      } while (k0 < t.depth);
      if constexpr (REGS) {
#pragma unroll
        for (int q = 0; q < kTile / 64; ++q) {
          const int c = c0 + q * 64;
          if (ok && c < t.cols)
            store_columns<OUT>(out + static_cast<uint64_t>(c) * ld, ld, reinterpret_cast<const uint32_t*>(sum[q]), t.cols - c, m < M, even);
        }
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  // neither CTA leaves while the other may still signal its barriers
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns));
  }
}

// Self-test of the bounded wait: a barrier that nothing completes, stages that
// nobody issues.
__global__ void __launch_bounds__(32) product_wait_probe_kernel(long long cycles) {
  __shared__ alignas(8) uint64_t bar;
  __shared__ Watch watch;
  if (threadIdx.x != 0) return;
  watch.dead = watch.progress = 0;
  mbar_init(smem_addr(&bar), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  mbar_wait(smem_addr(&bar), 0, &watch, cycles);
}

// ---------------------------------------------------------------- host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A [depth][height][width] bf16 tensor in boxes of `lines` lines x 64 elements;
// `chunks` > 1: the width, a multiple of 64, as an axis of its own in chunks of
// 64, so many of them per box.
bool encode(CUtensorMap* map, const void* p, uint64_t width, uint64_t height, uint64_t depth, uint32_t lines, uint32_t chunks = 1) {
  const EncodeFn fn = encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {chunks > 1 ? 64 : width, height, chunks > 1 ? width / 64 : 1, depth};
  const cuuint64_t strides[3] = {width * 2, chunks > 1 ? 128 : width * height * 2, width * height * 2};
  const cuuint32_t boxes[4] = {kStep, lines, chunks, 1}, ones[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, boxes, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether TMA can read rows of `width` bf16 elements at p.
bool on_grid(const void* p, uint64_t width) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && width % 8 == 0; }

template <int KIND, int OUT, bool REGS = false, bool HELD = false>
cudaError_t launch_pairs(const PairArgs& a, uint64_t most_tiles, cudaStream_t s) {
  const auto kernel = product_kernel<KIND, OUT, REGS, HELD>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err != cudaSuccess) return err;
  if (REGS) {  // a block launched with fewer registers would wait for its shares for ever
    static thread_local int regs = 0;
    if (regs == 0) {
      cudaFuncAttributes attr;
      err = cudaFuncGetAttributes(&attr, kernel);
      if (err != cudaSuccess) return err;
      regs = attr.numRegs;
    }
    if (regs < Crew<REGS>::kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  uint64_t pairs = static_cast<uint64_t>(current_sm_count() / 2);
  if (most_tiles < pairs) pairs = most_tiles;
  if (pairs == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(Crew<REGS>::kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  g_launched.store(true, std::memory_order_relaxed);
  err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace

cudaError_t launch_product_wait_probe(cudaStream_t s) {
  g_launched.store(true, std::memory_order_relaxed);
  product_wait_probe_kernel<<<1, 32, 0, s>>>(1ll << 14);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
}

cudaError_t read_product_error(unsigned int* flag, bool clear) {
  *flag = 0;
  if (!g_launched.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t err = cudaMemcpyFromSymbol(flag, g_product_error, sizeof(unsigned int));
  if (err == cudaSuccess && clear && *flag != 0) {
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbol(g_product_error, &zero, sizeof(zero));
  }
  return err;
}

cudaError_t launch_moe_product(int kind, int out_dt, const ProductArgs& args, cudaStream_t s) {
  const int E = args.num_experts;
  const int most_ranks = kMaxGroups / E < kLaunchRanks ? kMaxGroups / E : kLaunchRanks;
  const uint64_t n = args.n, k = args.contract;
  for (int r0 = 0; r0 < args.p; r0 += most_ranks) {
    PairArgs a = {};
    a.p = args.p - r0 < most_ranks ? args.p - r0 : most_ranks;
    a.num_experts = E;
    a.n = static_cast<uint32_t>(n);
    a.contract = static_cast<uint32_t>(k);
    const uint64_t a_width = k, b_width = kind == kProductForward ? k : n;
    a.tma_a = a.tma_b = 1;
    a.whole_a = a_width % 64 == 0 && a_width >= 128;
    a.whole_b = b_width % 64 == 0 && b_width >= 128;
    uint64_t rows = 0;
    uint64_t most_depth = kind == kProductForward ? k : kind == kProductGradInput ? n : 0;  // that a sum may have
    for (int i = 0; i < a.p; ++i) {
      a.pa[i] = args.a[r0 + i];
      a.pb[i] = args.b[r0 + i];
      a.out[i] = args.out[r0 + i];
      a.offsets[i] = args.offsets[r0 + i];
      a.rows[i] = args.rows[r0 + i];
      rows += (a.rows[i] + kTile - 1) / kTile + (a.rows[i] != 0 ? E : 0);
      if (kind == kProductGradWeight && a.rows[i] > most_depth) most_depth = a.rows[i];
      if (a.rows[i] == 0) continue;
      a.tma_a = a.tma_a && on_grid(a.pa[i], a_width);
      a.tma_b = a.tma_b && on_grid(a.pb[i], b_width);
    }
    for (int i = 0; i < a.p; ++i) {
      if (a.rows[i] == 0) continue;
      bool ok = true;
      if (a.tma_a) {
        ok = kind == kProductForward     ? encode(&a.a[i], a.pa[i], k, n, E, 128)
             : kind == kProductGradInput ? encode(&a.a[i], a.pa[i], k, n, E, kStep, a.whole_a ? 2 : 1)
                                         : encode(&a.a[i], a.pa[i], k, a.rows[i], 1, kStep, a.whole_a ? 2 : 1);
      }
      if (ok && a.tma_b) {
        if (kind == kProductGradWeight)
          ok = encode(&a.b_small[i], a.pb[i], n, a.rows[i], 1, kStep) &&
               (!a.whole_b || encode(&a.b[i], a.pb[i], n, a.rows[i], 1, kStep, 2));
        else
          ok = encode(&a.b[i], a.pb[i], b_width, a.rows[i], 1, 128) &&
               encode(&a.b_small[i], a.pb[i], b_width, a.rows[i], 1, kSmallBox);
      }
      if (!ok) return cudaErrorInvalidValue;
    }
    const uint64_t mt = ((kind == kProductForward ? n : k) + kTile - 1) / kTile;
    const uint64_t most_tiles = (kind == kProductGradWeight ? static_cast<uint64_t>(a.p) * E * ((n + kTile - 1) / kTile) : rows) * mt;
    cudaError_t err;
    if (out_dt == kF32)
      err = a.tma_a && a.tma_b ? launch_pairs<kProductGradWeight, kF32, true>(a, most_tiles, s)
                               : launch_pairs<kProductGradWeight, kF32>(a, most_tiles, s);
    else if (most_depth > kMostBF16)
      err = kind == kProductForward     ? launch_pairs<kProductForward, kBF16, false, true>(a, most_tiles, s)
            : kind == kProductGradInput ? launch_pairs<kProductGradInput, kBF16, false, true>(a, most_tiles, s)
                                        : launch_pairs<kProductGradWeight, kBF16, false, true>(a, most_tiles, s);
    else
      err = kind == kProductForward     ? launch_pairs<kProductForward, kBF16>(a, most_tiles, s)
            : kind == kProductGradInput ? launch_pairs<kProductGradInput, kBF16>(a, most_tiles, s)
                                        : launch_pairs<kProductGradWeight, kBF16>(a, most_tiles, s);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace ccl
