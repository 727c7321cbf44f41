// wgrad.cu -- weight and bias gradient of the stride-1 convs (k = 1, 3) from
// dy and an 8-bit checkpoint x~ of the conv's input, on tcgen05.
//
//   dw[o][c][ky][kx] = sum_p dy[p][o] x~[p + (ky, kx) - k/2][c]
//
// A GEMM per tap whose reduction runs over the pixels: M = 128 input channels,
// N = 64 output channels in two parts. Pixels are flattened over rows of w + 1
// positions: the extra one, zero in both operands, is the padding on the right of
// its row and on the left of the next, so any 128 consecutive positions make a
// tile whatever w is. x~ goes to tensor memory (lane = channel, two positions a
// column). dy goes to shared memory as it comes, pixel by pixel with channels next
// to each other (M/N-major): an octet of channels is a run of 16-byte pieces, one
// per position, and the tap kx is the same tile read 16 kx bytes apart, so that
// one staged tile serves three taps (three accumulators in TMEM). ky moves dy's
// row: it is one of the grid's units. With both operands in shared memory its
// bandwidth would bound the kernel: at N = 128 the MMA alone reads 128 bytes a
// clock (measured: 64.2 clocks a step, N = 64 no less than 53.6).
//
// Precision. x~ is e4m3 times a power of two: a half holds it exactly once the
// block scales are taken relative to the largest of their 32 channels (blocks
// 2^22 below it round at 2^-24 of the largest). dy is scaled per output
// channel by a power of two to below 2^15 and split into two halves, hi + lo,
// 22 significant bits. The MMA reads [hi | lo] as 128 columns next to one A
// operand, so the two parts have accumulators of their own. The tensor core's
// accumulator truncates: measured on GB300, a sum is off by about 1e-8 of its
// value per step. So a chain of MMAs ends after kChain stages; its sums move to
// FP32 registers, rounded to nearest.
//
// Schedule. (unit, stage) pairs, unit = (input-channel tile, output-channel
// tile, ky), are cut into equal contiguous ranges, one per SM, so that work
// stays balanced for any shape; every (unit, SM) piece writes a partial tile
// and a last pass adds a unit's pieces in order and undoes the scaling: the
// same inputs give the same bits.
//
// Eight warps bring x~ (global -> registers -> halves -> TMEM), eight bring dy
// (global -> registers -> halves -> shared memory), each thread loading the next
// stage's piece where it has just converted this one's; all sixteen drain the
// accumulators. Three warps turn positions into pixel indexes and block scales
// ahead of them, one thread issues the MMAs.
#include "ptx.cuh"
#include "silu.cuh"
#include "wgrad.cuh"

namespace vae {

namespace {

constexpr int kTM = 128;           // input channels of a tile (TMEM lanes)
constexpr int kTN = 64;            // output channels
constexpr int kPos = 128;          // positions of a stage
constexpr int kStagesA = 2;        // x~ in TMEM, 64 columns each
constexpr int kStagesB = 4;        // dy in shared memory
constexpr int kTables = 4;
constexpr int kChain = 16;         // stages between two drains: 2048 positions
constexpr int kStagers = 512;      // staging threads: eight warps for x~, eight for dy
constexpr int kDyThreads = 256;
constexpr int kTableWarps = 3;     // each makes every third table
constexpr int kMmaThreads = kStagers + 128;  // one more warpgroup issues and makes tables
// Registers: the launch gives every thread kLaunchRegs (65536 / 640, rounded
// down to a multiple of 8); the last warpgroup hands its share to the staging
// ones, which hold the accumulators and a raw stage.
constexpr int kLaunchRegs = 96, kStageRegs = 104, kIssueRegs = 64;
static_assert(4 * kStageRegs + kIssueRegs <= 5 * kLaunchRegs, "the split fits the launch");
// Positions between two octets of dy: odd, so that 16-byte pieces of neighbouring
// octets fall into different banks.
constexpr int kSlots = kPos + 3;
constexpr uint32_t kSbo = kSlots * 16;
constexpr uint32_t kLo = kTN / 8 * kSbo;               // from an octet's hi to its lo
constexpr uint32_t kStageBytes = 2 * kTN / 8 * kSbo;
// A stage's table: the x~ pixel of each position (-1: a zero), the scales of the
// four 32-channel blocks (a pair of halves per two positions), the dy pixel of
// each slot (-1: a zero) and its sample.
constexpr int kTabX = 0, kTabScale = kPos, kTabDy = kTabScale + 4 * (kPos / 2),
              kTabImg = kTabDy + kPos + 4, kTableInts = kTabImg + kPos + 4;
constexpr size_t kSmem = kStagesB * kStageBytes + kTables * kTableInts * 4 + 256;
static_assert(kSmem <= 227 * 1024, "stages fit an SM");
static_assert(kStageBytes % 16 == 0 && kTableInts % 4 == 0, "aligned");
constexpr int kSMs = 152;

struct WgradParams {
  const float *dy;
  const uint8_t *xq, *xs;
  const unsigned *amax;   // [cout] largest |dy| bits
  const unsigned *emax;   // [cp / 32] largest scale byte below 255
  float *part;            // [pieces][taps kx][kTN][kTM]
  int cin, cp, cout, n, h, w, wp;  // wp: positions per row
  unsigned positions;     // n * h * wp
  unsigned long long wp_magic, h_magic;
  int wp_shift, h_shift;
  int co_tiles, kys, stages;       // stages per unit
  long long total;                 // units * stages
  int *err;
  unsigned long long wait_ns;
};

// q / d for q < 2^30: (q * ceil(2^shift / d)) >> shift, shift = 32 + floor(log2 d).
__device__ __forceinline__ unsigned fast_div(unsigned q, unsigned long long magic, int shift) {
  return static_cast<unsigned>(q * magic >> shift);
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) {
  return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// The power of two that brings a channel's largest |dy| to [2^14, 2^15), as a
// float (2^127 at most); 1 for a channel with a non-finite value.
__device__ __forceinline__ int dy_exponent(unsigned amax_bits) {
  if (amax_bits >= 0x7f800000u) return 0;
  const int e = 141 - static_cast<int>(amax_bits >> 23);
  return e > 127 ? 127 : e;
}
__device__ __forceinline__ float exp2i(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

struct Unit {
  int ci0, co0, ky;
};
__device__ __forceinline__ Unit unit_at(const WgradParams &p, int u) {
  Unit t;
  t.ky = u % p.kys;
  u /= p.kys;
  t.co0 = u % p.co_tiles * kTN;
  t.ci0 = u / p.co_tiles * kTM;
  return t;
}

// Walks an SM's (unit, stage) range.
struct Cursor {
  int unit, stage;
  __device__ __forceinline__ bool next(int stages) {  // true on a new unit
    if (++stage < stages) return false;
    stage = 0;
    ++unit;
    return true;
  }
};
// Ends a chain with its kChain stages, its unit or the range.
struct Chain {
  int length = 0;
  __device__ __forceinline__ bool ends(bool piece_end) {
    if (!piece_end && ++length < kChain) return false;
    length = 0;
    return true;
  }
};

// One warp makes a stage's table. dy slot j is position q0 - 1 + j for a 3x3
// conv (tap kx pairs x~'s position k with slot k + 2 - kx), q0 + j for a 1x1.
template <int K>
__device__ __forceinline__ void make_table(const WgradParams &p, unsigned q0, const Unit &un,
                                           const uint32_t *etop, int lane, int *table) {
  const int nb = p.cp >> 5, b0 = un.ci0 >> 5;
  const bool words = (nb & 3) == 0;  // four blocks' scale bytes in one load
  const unsigned rows = static_cast<unsigned>(p.n) * p.h;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int pair = lane + 32 * i;
    uint32_t four[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned pos = q0 + 2 * pair + h;
      const unsigned row = fast_div(pos, p.wp_magic, p.wp_shift);
      const int x = static_cast<int>(pos - row * p.wp);
      const int pix = row < rows && x < p.w ? static_cast<int>(row) * p.w + x : -1;
      table[kTabX + 2 * pair + h] = pix;
      four[h] = 0;
      if (pix >= 0) {
        const uint8_t *src = p.xs + static_cast<size_t>(pix) * nb + b0;
        if (words) {
          four[h] = __ldg(reinterpret_cast<const uint32_t *>(src));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (b0 + k < nb) four[h] |= static_cast<uint32_t>(__ldg(src + k)) << (8 * k);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // 2^(7 - d), d binades below the largest block, as halves (zero under
      // 2^-25; whatever a block of NaNs is multiplied by, it stays NaN)
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 134 + static_cast<int>(four[h] >> (8 * k) & 255u) - static_cast<int>(etop[k]);
        f[h] = __uint_as_float(static_cast<uint32_t>(min(max(e, 0), 254)) << 23);
      }
      table[kTabScale + k * (kPos / 2) + pair] =
          static_cast<int>(h2_bits(__floats2half2_rn(f[0], f[1])));
    }
  }
  for (int slot = lane; slot < kPos + K - 1; slot += 32) {
    const unsigned pos = q0 + slot - (K == 3);  // (wraps below the first position)
    const unsigned row = fast_div(pos & 0x3fffffffu, p.wp_magic, p.wp_shift);
    const int x = static_cast<int>(pos - row * p.wp);
    const int img = static_cast<int>(fast_div(row, p.h_magic, p.h_shift));
    const int y = static_cast<int>(row) - img * p.h + (K == 3 ? 1 - un.ky : 0);
    const bool in = pos < p.positions && x < p.w && y >= 0 && y < p.h;
    table[kTabDy + slot] =
        in ? (static_cast<int>(row) + (K == 3 ? 1 - un.ky : 0)) * p.w + x : -1;
    table[kTabImg + slot] = img;
  }
}

// One of the 256 threads that bring x~. Warp w fills TMEM lanes 32 (w % 4) ..,
// one 32-channel block, for positions 64 (w / 4) ..; thread t of it takes four
// channels 4 (t / 4) + j, which land in lanes t / 4 + 8 j of the quadrant, at
// two positions in eight.
struct XStager {
  const WgradParams &p;
  const int quad, pair0;  // of the first of its pairs; eight of them, 4 apart
  const uint8_t *src = nullptr;
  uint32_t raw[16];

  __device__ explicit XStager(const WgradParams &params)
      : p(params), quad(threadIdx.x >> 5 & 3),
        pair0(32 * (threadIdx.x >> 7) + (threadIdx.x & 3)) {}
  __device__ void set_load_unit(const Unit &un) {
    const int ch = un.ci0 + 32 * quad + (threadIdx.x >> 2 & 7) * 4;
    src = ch < p.cp ? p.xq + ch : nullptr;
  }
  __device__ __forceinline__ void load(int i, const int *table) {
    const int2 pix = *reinterpret_cast<const int2 *>(table + kTabX + 2 * (pair0 + 4 * i));
    raw[2 * i] = raw[2 * i + 1] = 0;
    if (src) {
      if (pix.x >= 0)
        raw[2 * i] = __ldg(reinterpret_cast<const uint32_t *>(
            src + static_cast<unsigned long long>(static_cast<unsigned>(pix.x)) *
                      static_cast<unsigned>(p.cp)));
      if (pix.y >= 0)
        raw[2 * i + 1] = __ldg(reinterpret_cast<const uint32_t *>(
            src + static_cast<unsigned long long>(static_cast<unsigned>(pix.y)) *
                      static_cast<unsigned>(p.cp)));
    }
  }
  // Pair i as halves: channel j of the two positions in out[j].
  __device__ __forceinline__ void convert(int i, const int *table, uint32_t *out) const {
    const uint32_t two =
        static_cast<uint32_t>(table[kTabScale + quad * (kPos / 2) + pair0 + 4 * i]);
    const __half2 sc = *reinterpret_cast<const __half2 *>(&two);
    const uint32_t a = __byte_perm(raw[2 * i], raw[2 * i + 1], 0x5140);
    const uint32_t b = __byte_perm(raw[2 * i], raw[2 * i + 1], 0x7362);
    out[0] = h2_bits(__hmul2(e4m3x2_half2(a & 0xffffu), sc));
    out[1] = h2_bits(__hmul2(e4m3x2_half2(a >> 16), sc));
    out[2] = h2_bits(__hmul2(e4m3x2_half2(b & 0xffffu), sc));
    out[3] = h2_bits(__hmul2(e4m3x2_half2(b >> 16), sc));
  }
};

// One of the 256 threads that bring dy: an octet of output channels at slots
// first + 32 j. A 3x3 conv's stage has 130 slots, whose first two are the last
// two of the stage before; the threads of the last two carry them over.
template <int K, bool NHWC, bool WIDE>
struct DyStager {
  const WgradParams &p;
  const int co8, first;
  const float *src = nullptr;
  int valid = 0;  // channels of the octet
  Oct raw[4];
  float scale[8];

  __device__ explicit DyStager(const WgradParams &params)
      : p(params), co8(NHWC ? threadIdx.x & 7 : (threadIdx.x & 255) >> 5),
        first((NHWC ? (threadIdx.x & 255) >> 3 : threadIdx.x & 31) + (K - 1)) {}
  __device__ void set_load_unit(const Unit &un) {
    const int co = un.co0 + 8 * co8;
    valid = p.cout - co;
    src = p.dy + (NHWC ? static_cast<size_t>(co) : static_cast<size_t>(co) * p.h * p.w);
  }
  __device__ void set_unit(const Unit &un) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int co = un.co0 + 8 * co8 + i;
      scale[i] = co < p.cout ? exp2i(dy_exponent(__ldg(p.amax + co))) : 0.f;
    }
  }
  __device__ __forceinline__ void load_slot(Oct &r, int slot, const int *table) const {
    const int pix = table[kTabDy + slot];
    if (NHWC) {
      r = load_oct<WIDE, false>(src + static_cast<unsigned long long>(static_cast<unsigned>(pix)) *
                                          static_cast<unsigned>(p.cout),
                                pix < 0 ? 0 : valid);
      return;
    }
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (pix >= 0) {
      const size_t hw = static_cast<size_t>(p.h) * p.w;
      const float *q = src + static_cast<size_t>(table[kTabImg + slot]) * (p.cout - 1) * hw + pix;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (valid > i) v[i] = __ldg(q + i * hw);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = pk2(v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ uint32_t at(uint32_t stage, int slot) const {
    return stage + co8 * kSbo + slot * 16;
  }
  __device__ __forceinline__ void store_slot(uint32_t stage, int slot, const Oct &r) const {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (the scaling is exact, so the difference is what hi dropped)
      const uint64_t s = mul2(r.v[i], pk2(scale[2 * i], scale[2 * i + 1]));
      const __half2 h = __floats2half2_rn(lo2(s), hi2(s));
      const float2 f = __half22float2(h);
      const uint64_t rest = fma2(pk2(f.x, f.y), pk2(-1.f, -1.f), s);
      hi[i] = h2_bits(h);
      lo[i] = h2_bits(__floats2half2_rn(lo2(rest), hi2(rest)));
    }
    st_shared16(at(stage, slot), make_uint4(hi[0], hi[1], hi[2], hi[3]));
    st_shared16(at(stage, slot) + kLo, make_uint4(lo[0], lo[1], lo[2], lo[3]));
  }
  // Slots 0 and 1 of a 3x3 stage, by the threads of slots 128 and 129.
  __device__ __forceinline__ void carry(uint32_t stage, uint32_t before, bool contiguous,
                                        const int *table) const {
    if (K == 1 || first + 96 < kPos) return;
    const int slot = first + 96 - kPos;
    if (contiguous) {
      st_shared16(at(stage, slot), ld_shared16(at(before, kPos + slot)));
      st_shared16(at(stage, slot) + kLo, ld_shared16(at(before, kPos + slot) + kLo));
    } else {
      Oct r;
      load_slot(r, slot, table);
      store_slot(stage, slot, r);
    }
  }
};

// First (unit, stage) of SM range c.
__host__ __device__ __forceinline__ long long range_start(long long total, int grid, int c) {
  return total * c / grid;
}

template <int K, bool NHWC, bool WIDE>
__global__ void __launch_bounds__(kMmaThreads, 1) wgrad_mma(const WgradParams p) {
  constexpr int TAPS = K;  // kx
  constexpr uint32_t kAcc = TAPS * 2 * kTN;  // TMEM columns of the accumulators
  constexpr uint32_t kCols = TAPS == 1 ? 256 : 512;
  static_assert(kAcc + kStagesA * (kPos / 2) <= kCols, "TMEM holds both");
  extern __shared__ __align__(128) uint8_t smem[];
  int *tables = reinterpret_cast<int *>(smem + kStagesB * kStageBytes);
  uint64_t *a_full = reinterpret_cast<uint64_t *>(tables + kTables * kTableInts);
  uint64_t *a_empty = a_full + kStagesA, *b_full = a_empty + kStagesA;
  uint64_t *b_empty = b_full + kStagesB, *tab_full = b_empty + kStagesB;
  uint64_t *tab_empty = tab_full + kTables, *acc_done = tab_empty + kTables;
  uint64_t *acc_free = acc_done + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStagesA; ++i) {
      mbar_init(a_full + i, (kStagers - kDyThreads) / 32);
      mbar_init(a_empty + i, 1);
    }
    for (int i = 0; i < kStagesB; ++i) {
      mbar_init(b_full + i, kDyThreads / 32);
      mbar_init(b_empty + i, 1);
    }
    for (int i = 0; i < kTables; ++i) {
      mbar_init(tab_full + i, 1);
      mbar_init(tab_empty + i, kStagers / 32);
    }
    mbar_init(acc_done, 1);
    mbar_init(acc_free, kStagers / 32);
    *abort = 0u;
    fence_mbarrier_init();
  }
  if (warp == kStagers / 32) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long g0 = range_start(p.total, gridDim.x, blockIdx.x);
  const int count = static_cast<int>(range_start(p.total, gridDim.x, blockIdx.x + 1) - g0);
  const Cursor start{static_cast<int>(g0 / p.stages), static_cast<int>(g0 % p.stages)};
  auto give_up = [&]() {
    *abort = 1u;
    atomicCAS(p.err, 0, static_cast<int>(VAE_EDEVICE_TIMEOUT));
  };

  if (warp < kStagers / 32) {
    setmaxnreg_inc<kStageRegs>();
    bool ok = true;
    // Waits agree across the warp, so that a timeout leaves it converged.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, p.wait_ns));
    };

    // This warp drains TMEM lanes 32 (warp % 4) .., output channels 16 (warp / 4) ..
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    float acc[TAPS][16];
#pragma unroll
    for (int k = 0; k < TAPS; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[k][i] = 0.f;
    uint32_t chains = 0;
    Cursor dr = start;  // the stage whose chain end is looked at next
    Chain dr_chain;
    // Looks at stage `i`; called one stage behind, when the next chain's first
    // stage is on its way.
    auto drain = [&](int i) {
      const bool piece_end = i == count - 1 || dr.stage == p.stages - 1;
      const int unit = dr.unit;
      dr.next(p.stages);
      if (!dr_chain.ends(piece_end)) return;
      ok = wait(acc_done, chains & 1);
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < TAPS; ++k) {
        float v[16];
        tmem_ld_16cols(t_lane + (warp >> 2) * 16 + k * 2 * kTN, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[k][j] += v[j];
        tmem_ld_16cols(t_lane + (warp >> 2) * 16 + k * 2 * kTN + kTN, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[k][j] += v[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free);
      ++chains;
      if (piece_end) {
        // TMEM lane r of a quadrant is channel 4 (r % 8) + r / 8
        const size_t piece = static_cast<size_t>(unit) + blockIdx.x;
        float *o = p.part + piece * (TAPS * kTN * kTM) + (warp >> 2) * 16 * kTM +
                   (warp & 3) * 32 + 4 * (lane & 7) + (lane >> 3);
#pragma unroll
        for (int k = 0; k < TAPS; ++k)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[(k * kTN + j) * kTM] = acc[k][j];
            acc[k][j] = 0.f;
          }
      }
    };

    Cursor ld = start;  // the stage that is loaded next
    if (warp < (kStagers - kDyThreads) / 32) {
      XStager st(p);
      st.set_load_unit(unit_at(p, ld.unit));
      ok = wait(tab_full, 0);
      if (ok)
#pragma unroll
        for (int k = 0; k < 8; ++k) st.load(k, tables);
#pragma unroll 1
      for (int i = 0; i < count && ok; ++i) {
        const int *table = tables + (i % kTables) * kTableInts;
        const bool more = i + 1 < count;
        const int *ahead = tables + ((i + 1) % kTables) * kTableInts;
        if (ld.next(p.stages) && more) st.set_load_unit(unit_at(p, ld.unit));
        if (more) ok = wait(tab_full + (i + 1) % kTables, ((i + 1) / kTables) & 1);
        if (ok && i >= kStagesA)
          ok = wait(a_empty + i % kStagesA, (i / kStagesA - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dst = t_lane + kAcc + (i % kStagesA) * (kPos / 2) + (warp >> 2) * 32;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          uint32_t low[8], high[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
            st.convert(k + j, table, o);
            low[2 * j] = o[0];
            low[2 * j + 1] = o[1];
            high[2 * j] = o[2];
            high[2 * j + 1] = o[3];
            if (more) st.load(k + j, ahead);
          }
          tmem_st_16x16(dst + 4 * k, low);
          tmem_st_16x16(dst + 4 * k + (16u << 16), high);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(a_full + i % kStagesA);
          mbar_arrive(tab_empty + i % kTables);
        }
        if (i > 0) drain(i - 1);
      }
    } else {
      DyStager<K, NHWC, WIDE> st(p);
      const uint32_t base = smem_u32(smem);
      st.set_load_unit(unit_at(p, ld.unit));
      st.set_unit(unit_at(p, ld.unit));
      Cursor cv = start;  // the stage that is converted
      bool contiguous = false;
      ok = wait(tab_full, 0);
      if (ok)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.load_slot(st.raw[j], st.first + 32 * j, tables);
#pragma unroll 1
      for (int i = 0; i < count && ok; ++i) {
        const int *table = tables + (i % kTables) * kTableInts;
        const bool more = i + 1 < count;
        const int *ahead = tables + ((i + 1) % kTables) * kTableInts;
        const uint32_t stage = base + (i % kStagesB) * kStageBytes;
        const uint32_t before = base + ((i + kStagesB - 1) % kStagesB) * kStageBytes;
        if (i >= kStagesB) ok = wait(b_empty + i % kStagesB, (i / kStagesB - 1) & 1);
        if (ok && more) ok = wait(tab_full + (i + 1) % kTables, ((i + 1) / kTables) & 1);
        if (!ok) break;
        st.carry(stage, before, contiguous, table);
        if (ld.next(p.stages) && more) st.set_load_unit(unit_at(p, ld.unit));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          st.store_slot(stage, st.first + 32 * j, st.raw[j]);
          if (more) st.load_slot(st.raw[j], st.first + 32 * j, ahead);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_full + i % kStagesB);
          mbar_arrive(tab_empty + i % kTables);
        }
        contiguous = !cv.next(p.stages);
        if (!contiguous && more) st.set_unit(unit_at(p, cv.unit));
        if (i > 0) drain(i - 1);
      }
    }
    if (ok) drain(count - 1);
    if (!ok) give_up();
  } else {
    setmaxnreg_dec<kIssueRegs>();
    if (threadIdx.x == kStagers) {
      constexpr uint32_t idesc = idesc_f16_tmem_a(kTM, 2 * kTN);
      const uint32_t base = smem_u32(smem);
      uint32_t chains = 0;
      bool fresh = true, ok = true;
      Cursor at = start;
      Chain chain;
      for (int i = 0; i < count && ok; ++i) {
        const int sa = i % kStagesA, sb = i % kStagesB;
        if (fresh && chains > 0) ok = mbar_wait(acc_free, (chains - 1) & 1, abort, p.wait_ns);
        if (ok) ok = mbar_wait(a_full + sa, (i / kStagesA) & 1, abort, p.wait_ns);
        if (ok) ok = mbar_wait(b_full + sb, (i / kStagesB) & 1, abort, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tmem + kAcc + sa * (kPos / 2);
        const uint64_t b = mn_major_desc(base + sb * kStageBytes, 128, kSbo);
#pragma unroll
        for (int k = 0; k < kPos / 16; ++k)
#pragma unroll
          for (int tap = 0; tap < TAPS; ++tap)
            umma_f16_tmem_a(tmem + tap * 2 * kTN, a + 8 * k, b + 16 * k + (TAPS - 1 - tap), idesc,
                            !fresh || k > 0);
        fresh = false;
        umma_commit(a_empty + sa);
        umma_commit(b_empty + sb);
        const bool piece_end = i == count - 1 || at.stage == p.stages - 1;
        at.next(p.stages);
        if (chain.ends(piece_end)) {
          umma_commit(acc_done);
          ++chains;
          fresh = true;
        }
      }
      if (!ok) {
        give_up();
        // the MMAs issued so far finish before TMEM is freed
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {}
      }
    } else if (warp > kStagers / 32) {
      const int first = warp - kStagers / 32 - 1;
      Cursor at = start;
      for (int i = 0; i < first; ++i) at.next(p.stages);
      int unit = -1;
      Unit un{};
      uint32_t etop[4];
      bool ok = true;
      for (int i = first; i < count && ok; i += kTableWarps) {
        const int s = i % kTables;
        if (i >= kTables)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(tab_empty + s, (i / kTables - 1) & 1, abort, p.wait_ns));
        if (!ok) break;
        if (at.unit != unit) {
          unit = at.unit;
          un = unit_at(p, unit);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            etop[k] = (un.ci0 >> 5) + k < p.cp >> 5 ? __ldg(p.emax + (un.ci0 >> 5) + k) : 0u;
        }
        make_table<K>(p, static_cast<unsigned>(at.stage) * kPos, un, etop, lane,
                      tables + s * kTableInts);
        __syncwarp();
        if (lane == 0) mbar_arrive(tab_full + s);
        for (int k = 0; k < kTableWarps; ++k) at.next(p.stages);
      }
      if (!ok) give_up();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kStagers / 32) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------- before and after
constexpr int kScanThreads = 256;

// Largest scale byte below 255 of each 32-channel block; a share per block. A
// thread steps over the bytes, as words, in strides of nb words, so that byte k
// of its words always belongs to the same channel block.
__device__ __forceinline__ void scan_scales(const uint8_t *__restrict__ xs, long long rows,
                                            int nb, unsigned *emax, unsigned *sm, int blk,
                                            int nblk) {
  for (int i = threadIdx.x; i < nb; i += kScanThreads) sm[i] = 0u;
  __syncthreads();
  const long long bytes = rows * nb, words = bytes / 4;
  const int per = kScanThreads / nb * nb;  // (nb <= 128)
  const long long strides = (words + per - 1) / per;
  const long long w1 = min(words, strides * (blk + 1) / nblk * per);
  long long w = strides * blk / nblk * per + threadIdx.x;
  if (threadIdx.x < per && w < w1) {
    const uint32_t *src = reinterpret_cast<const uint32_t *>(xs);
    unsigned m = 0;
    const int first = static_cast<int>(4 * w % nb);
    auto add = [&](uint32_t v) { m = __vmaxu4(m, v & ~__vcmpeq4(v, 0xffffffffu)); };
    for (; w + 3 * per < w1; w += 4 * per) {
      uint32_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = __ldg(src + w + u * per);
#pragma unroll
      for (int u = 0; u < 4; ++u) add(v[u]);
    }
    for (; w < w1; w += per) add(__ldg(src + w));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (m >> (8 * k) & 255u) atomicMax(sm + (first + k) % nb, m >> (8 * k) & 255u);
  }
  if (blk == 0 && threadIdx.x < (bytes & 3)) {
    const long long i = bytes - 1 - threadIdx.x;
    const unsigned v = xs[i];
    if (v != 255u) atomicMax(sm + static_cast<int>(i % nb), v);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nb; i += kScanThreads)
    if (sm[i]) atomicMax(emax + i, sm[i]);
}

// grid (slabs, ceil(cout / 1024)): sums [slab][cout] and the largest |dy| of
// each output channel. The blocks are those resident at a time and sweep the
// rows side by side. The maxima do not depend on the order of the atomics.
template <bool WIDE>
__global__ void __launch_bounds__(kScanThreads, 2)
    wgrad_scan_nhwc(const float *__restrict__ dy, long long rows, int cout,
                    const uint8_t *__restrict__ xs, int nb, float *__restrict__ psum,
                    unsigned *__restrict__ amax, unsigned *__restrict__ emax) {
  constexpr int kDepth = 4;  // rows in flight
  __shared__ unsigned sm[128];
  __shared__ float4 rs[2 * kScanThreads], rm[2 * kScanThreads];  // [row of a sweep][channel]
  const int c0 = blockIdx.y * 1024, cols = min(1024, cout - c0), octs = (cols + 7) / 8;
  const int per = kScanThreads / octs, q = threadIdx.x % octs, l = threadIdx.x / octs;
  const int left = l < per ? cols - 8 * q : 0;
  const long long step = static_cast<long long>(gridDim.x) * per;
  Oct s = {{0, 0, 0, 0}};
  float m[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const float *src = dy + c0 + 8 * q;
  for (long long r = static_cast<long long>(blockIdx.x) * per + l; r < rows; r += kDepth * step) {
    Oct v[kDepth];
#pragma unroll
    for (int u = 0; u < kDepth; ++u)
      v[u] = load_oct<WIDE, false>(src + (r + u * step) * cout, r + u * step < rows ? left : 0);
#pragma unroll
    for (int u = 0; u < kDepth; u += 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s.v[i] = add2(s.v[i], add2(v[u].v[i], v[u + 1].v[i]));
        m[2 * i] = max_abs3(m[2 * i], lo2(v[u].v[i]), lo2(v[u + 1].v[i]));
        m[2 * i + 1] = max_abs3(m[2 * i + 1], hi2(v[u].v[i]), hi2(v[u + 1].v[i]));
      }
  }
  if (l < per) {
    const int at = 2 * (l * octs + q);
    rs[at] = oct_lo(s);
    rs[at + 1] = oct_hi(s);
    rm[at] = make_float4(m[0], m[1], m[2], m[3]);
    rm[at + 1] = make_float4(m[4], m[5], m[6], m[7]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += kScanThreads) {
    float sum = 0.f, top = 0.f;
#pragma unroll 4
    for (int k = 0; k < per; ++k) {
      sum += reinterpret_cast<const float *>(rs)[k * octs * 8 + c];
      const float t = reinterpret_cast<const float *>(rm)[k * octs * 8 + c];
      top = max_abs3(top, t, t);
    }
    psum[static_cast<size_t>(blockIdx.x) * cout + c0 + c] = sum;
    atomicMax(amax + c0 + c, __float_as_uint(top));
  }
  if (blockIdx.y == 0) scan_scales(xs, rows, nb, emax, sm, blockIdx.x, gridDim.x);
}

// grid (slabs, cout): slab of the n planes of one channel.
__global__ void __launch_bounds__(kScanThreads)
    wgrad_scan_nchw(const float *__restrict__ dy, int n, long long hw, int cout,
                    const uint8_t *__restrict__ xs, int nb, float *__restrict__ psum,
                    unsigned *__restrict__ amax, unsigned *__restrict__ emax) {
  __shared__ unsigned sm[128];
  __shared__ float rs[kScanThreads / 32];
  __shared__ unsigned rm[kScanThreads / 32];
  const int co = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long p0 = hw * blockIdx.x / gridDim.x, p1 = hw * (blockIdx.x + 1) / gridDim.x;
  float s = 0.f;
  unsigned m = 0;
  for (int i = 0; i < n; ++i) {
    const float *src = dy + (static_cast<long long>(i) * cout + co) * hw;
    for (long long q = p0 + threadIdx.x; q < p1; q += kScanThreads) {
      const float v = __ldg(src + q);
      s += v;
      m = max(m, abs_bits(v));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (lane == 0) {
    rs[warp] = s;
    rm[warp] = m;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kScanThreads / 32; ++k) {
      s += rs[k];
      m = max(m, rm[k]);
    }
    psum[static_cast<size_t>(blockIdx.x) * cout + co] = s;
    atomicMax(amax + co, m);
  }
  const int blk = blockIdx.y * gridDim.x + blockIdx.x;
  if (blk < kSMs)
    scan_scales(xs, n * hw, nb, emax, sm, blk,
                min(kSMs, static_cast<int>(gridDim.x * gridDim.y)));
}

// grid (input-channel tiles + 1, cout): adds a unit's pieces in order, undoes
// the scaling and writes the taps of 128 input channels, contiguous in dw, through
// shared memory; the last column of blocks adds up dbias.
template <int K>
__global__ void __launch_bounds__(kTM)
    wgrad_reduce(const WgradParams p, int grid, const float *__restrict__ psum, int slabs,
                 float *__restrict__ dw, float *__restrict__ dbias) {
  __shared__ float out[kTM * K * K];
  const int co = blockIdx.y;
  if (blockIdx.x == gridDim.x - 1) {
    if (!dbias || threadIdx.x >= 32) return;
    float s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < slabs; i += 32) s += psum[static_cast<size_t>(i) * p.cout + co];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) dbias[co] = s;
    return;
  }
  const int ci0 = blockIdx.x * kTM, ci = ci0 + threadIdx.x;
  const int e = ci < p.cin ? static_cast<int>(p.emax[ci >> 5]) - 127 - 7 - dy_exponent(p.amax[co])
                           : 0;
#pragma unroll 1
  for (int ky = 0; ky < K; ++ky) {
    const int u = (static_cast<int>(blockIdx.x) * p.co_tiles + co / kTN) * K + ky;
    // the SM ranges that hold the unit's first and last stage
    const long long a = static_cast<long long>(u) * p.stages, b = a + p.stages - 1;
    const int c0 = static_cast<int>(((a + 1) * grid - 1) / p.total);
    const int c1 = static_cast<int>(((b + 1) * grid - 1) / p.total);
    float v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const float *src = p.part + static_cast<size_t>(u + c) * (K * kTN * kTM) +
                         (co % kTN) * kTM + threadIdx.x;
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += src[k * kTN * kTM];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) out[threadIdx.x * (K * K) + ky * K + k] = scalbnf(v[k], e);
  }
  __syncthreads();
  const int count = min(kTM, p.cin - ci0) * K * K;
  float *o = dw + (static_cast<size_t>(co) * p.cin + ci0) * (K * K);
  for (int i = threadIdx.x; i < count; i += kTM) o[i] = out[i];
}

int floor_log2(unsigned d) {
  int l = 0;
  while (d >> (l + 1)) ++l;
  return l;
}

struct WgradWs {
  float *psum, *part;
  unsigned *maxima;  // amax [cout], emax [cp / 32]
  int slabs, grid, units, stages;  // slabs: at most, of the scan
};

WgradWs carve_wgrad(Carver &cv, int n, int cin, int h, int w, int cout, int k) {
  WgradWs ws{};
  const long long rows = static_cast<long long>(n) * h * w;
  ws.slabs = static_cast<int>(std::max(1ll, std::min<long long>(2 * kSMs, rows / 8)));
  const long long positions = static_cast<long long>(n) * h * (w + (k == 3));
  ws.stages = ceil_div(positions, kPos);
  ws.units = ceil_div(cin, kTM) * ceil_div(cout, kTN) * k;
  // Whole slices of the pixels per SM where that leaves few SMs idle: the units
  // then walk the same pixels at the same time and share them in L2.
  const int slices = std::min(kSMs / ws.units, ws.stages);
  ws.grid = slices * ws.units >= kSMs * 9 / 10
                ? slices * ws.units
                : static_cast<int>(std::min<long long>(
                      kSMs, static_cast<long long>(ws.units) * ws.stages));
  ws.psum = cv.take<float>(static_cast<size_t>(ws.slabs) * cout);
  ws.maxima = cv.take<unsigned>(cout + ckpt_cp(cin) / 32);
  ws.part = cv.take<float>(static_cast<size_t>(ws.units + ws.grid - 1) * k * kTN * kTM);
  return ws;
}

template <int K, bool NHWC, bool WIDE>
int launch_mma(const WgradParams &p, int grid, cudaStream_t s) {
  // (the register split waits for what the launch did not bring)
  static const int regs = [] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, wgrad_mma<K, NHWC, WIDE>) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs != kLaunchRegs) return VAE_ECUDA;
  VAE_CUDA_TRY(cudaFuncSetAttribute(wgrad_mma<K, NHWC, WIDE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem)));
  wgrad_mma<K, NHWC, WIDE><<<grid, kMmaThreads, kSmem, s>>>(p);
  VAE_LAUNCH_CHECK();
  return VAE_OK;
}

template <int K>
int launch_mma(const WgradParams &p, int nhwc, bool wide, int grid, cudaStream_t s) {
  if (!nhwc) return launch_mma<K, false, false>(p, grid, s);
  return wide ? launch_mma<K, true, true>(p, grid, s) : launch_mma<K, true, false>(p, grid, s);
}

}  // namespace

size_t wgrad_ws_bytes(int n, int cin, int h, int w, int cout, int k) {
  Carver cv(nullptr, 0);
  carve_wgrad(cv, n, cin, h, w, cout, k);
  return cv.used;
}

int wgrad(const float *dy, CkptView x, int n, int cin, int h, int w, int nhwc, int cout, int k,
          float *dw, float *dbias, void *workspace, cudaStream_t s) {
  Carver cv(workspace, ~size_t(0));
  const WgradWs ws = carve_wgrad(cv, n, cin, h, w, cout, k);
  const int cp = ckpt_cp(cin), nb = cp / 32;
  const long long hw = static_cast<long long>(h) * w, rows = n * hw;
  WgradParams p{};
  p.dy = dy;
  p.xq = x.q;
  p.xs = x.scale;
  p.amax = ws.maxima;
  p.emax = ws.maxima + cout;
  p.part = ws.part;
  p.cin = cin;
  p.cp = cp;
  p.cout = cout;
  p.n = n;
  p.h = h;
  p.w = w;
  p.wp = w + (k == 3);
  p.positions = static_cast<unsigned>(n) * h * p.wp;
  p.wp_shift = 32 + floor_log2(p.wp);
  p.h_shift = 32 + floor_log2(h);
  p.wp_magic = ((1ull << p.wp_shift) + p.wp - 1) / p.wp;
  p.h_magic = ((1ull << p.h_shift) + h - 1) / h;
  p.co_tiles = ceil_div(cout, kTN);
  p.kys = k;
  p.stages = ws.stages;
  p.total = static_cast<long long>(ws.units) * ws.stages;
  p.err = device_error_word();
  if (!p.err) return VAE_ECUDA;
  p.wait_ns = wait_limit_ns();
  VAE_CUDA_TRY(cudaMemsetAsync(ws.maxima, 0, (cout + nb) * sizeof(unsigned), s));
  const bool wide = wide_ok(cout, dy);
  int slabs;
  if (nhwc) {
    const int per = kScanThreads / std::min(128, ceil_div(cout, 8));  // rows of a block's sweep
    slabs = static_cast<int>(std::max(1ll, std::min<long long>(ws.slabs, rows / (4 * per))));
    (wide ? wgrad_scan_nhwc<true> : wgrad_scan_nhwc<false>)<<<
        dim3(slabs, ceil_div(cout, 1024)), kScanThreads, 0, s>>>(
        dy, rows, cout, x.scale, nb, ws.psum, ws.maxima, ws.maxima + cout);
  } else {
    slabs = std::max(1, std::min(ws.slabs, 8 * kSMs / cout));
    wgrad_scan_nchw<<<dim3(slabs, cout), kScanThreads, 0, s>>>(
        dy, n, hw, cout, x.scale, nb, ws.psum, ws.maxima, ws.maxima + cout);
  }
  VAE_LAUNCH_CHECK();
  VAE_TRY((k == 3 ? launch_mma<3> : launch_mma<1>)(p, nhwc, wide, ws.grid, s));
  const dim3 rg(ceil_div(cin, kTM) + 1, cout);
  if (k == 3)
    wgrad_reduce<3><<<rg, kTM, 0, s>>>(p, ws.grid, ws.psum, slabs, dw, dbias);
  else
    wgrad_reduce<1><<<rg, kTM, 0, s>>>(p, ws.grid, ws.psum, slabs, dw, dbias);
  VAE_LAUNCH_CHECK();
  count_launches(3);
  return VAE_OK;
}

}  // namespace vae
