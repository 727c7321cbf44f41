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
// block scales are taken relative to the largest of their 32 channels, which is
// put at 2^7 (its largest numbers are 224 to 448 times that). A block whose scale is
// d binades lower holds multiples of 2^(-2 - d): exact to d = 22, rounded to
// multiples of 2^-24 to d = 31 (2^-39 of the largest number), zero from d = 32 on
// (2^-31 of it at most). It shows only where dy is next to nothing wherever the
// activations are large; bf16 operands would hold any range, but take dy in three
// parts, half as many MMAs again. dy is scaled per output
// channel by a power of two to below 2^15 and split into two halves, hi + lo,
// 22 significant bits. The MMA reads [hi | lo] as 128 columns next to one A
// operand, so the two parts have accumulators of their own. The tensor core's
// accumulator truncates: measured on GB300, a sum is off by about 1e-8 of its
// value per step. So a chain of MMAs ends after kChain stages; its sums are added
// to the piece's FP32 numbers in global memory, rounded to nearest. Each of those
// belongs to one thread, whose additions keep their order.
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
// ahead of them. Three threads issue the MMAs, one per tap: a thread takes 80
// clocks to issue one, the tensor core 64 to run it.
//
// Bound: the tensor core (24 MMAs of 64 clocks a stage), then what the staging
// warps and barriers add (dy's loop takes 2300 clocks a stage; a chain's end 3700,
// for 768 reductions of 128 bytes). 128 to 128 channels at 512^2: 113 us, 12300
// stages of 128 positions on 150 SMs, 65 us of them the MMAs' (154 GFLOP; 1.36
// PFLOP/s); with the scan (25 us) and the reduction 145 us.
// Measured on the way at this size: one issuing thread 142 us, sums in registers
// with the spills of prefetched data that they bring 187 us, 128-bit loads of dy
// (each sector twice) 40 us more; sixteen warps for x~ at 64 registers 179 us,
// sixteen for dy 115 us.
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
constexpr int kXGroups = 2;        // of four warps each, for a share of the positions
constexpr int kXWarps = 4 * kXGroups, kDyWarps = 8;
constexpr int kStageWarps = kXWarps + kDyWarps;
constexpr int kTableWarps = 3;     // each makes every third table
constexpr int kIssueWarp = kStageWarps, kTableWarp = kStageWarps + 3;  // one issuer per tap
constexpr int kMmaThreads = 32 * (kTableWarp + kTableWarps);
// Positions between two octets of dy: odd, so that 16-byte pieces of neighbouring
// octets fall into different banks.
constexpr int kSlots = kPos + 3;
constexpr uint32_t kSbo = kSlots * 16;
constexpr uint32_t kLo = kTN / 8 * kSbo;               // from an octet's hi to its lo
constexpr uint32_t kStageBytes = 2 * kTN / 8 * kSbo;
// A stage's table: its unit and flags, the x~ pixel of each position (-1: a
// zero), the scales of the four 32-channel blocks (a pair of halves per two
// positions), the dy pixel of each slot (-1: a zero) and, NCHW, its sample.
constexpr int kTabUnit = 0, kTabFlags = 1, kTabX = 4, kTabScale = kTabX + kPos,
              kTabDy = kTabScale + 4 * (kPos / 2), kTabImg = kTabDy + kPos + 4,
              kTableInts = kTabImg + kPos + 4;
enum : int {
  kNewUnit = 1,     // the stage before is another unit's
  kChainEnd = 2,    // its MMAs end a chain
  kFirstChain = 4,  // which is the first of its (unit, SM) piece
};
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
// Loads where `at` is not negative, else zeros: predicated, where a branch around
// each would cost the staging warps more than the loads.
__device__ __forceinline__ uint32_t load4_if(int at, const uint8_t *p) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ge.s32 q, %1, 0;\n\tmov.b32 %0, 0;\n\t"
      "@q ld.global.nc.b32 %0, [%2];\n\t}"
      : "=r"(v)
      : "r"(at), "l"(p));
  return v;
}
__device__ __forceinline__ Oct load32_if(int at, const float *p) {
  Oct o;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ge.s32 q, %4, 0;\n\t"
      "mov.b64 %0, 0;\n\tmov.b64 %1, 0;\n\tmov.b64 %2, 0;\n\tmov.b64 %3, 0;\n\t"
      "@q ld.global.L1::no_allocate.v4.b64 {%0, %1, %2, %3}, [%5];\n\t}"
      : "=&l"(o.v[0]), "=&l"(o.v[1]), "=&l"(o.v[2]), "=&l"(o.v[3])
      : "r"(at), "l"(p));
  return o;
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
template <int K, bool NHWC>
__device__ __forceinline__ void make_table(const WgradParams &p, unsigned q0, const Unit &un,
                                           const uint32_t *etop, int lane, int *table) {
  const int nb = p.cp >> 5, b0 = un.ci0 >> 5;
  const bool words = (nb & 3) == 0;  // four blocks' scale bytes in one load
  const int up = K == 3 ? 1 - un.ky : 0;
  // x~'s pixel at a position (-1: none), and dy's in its slot
  auto place = [&](unsigned pos, int slot) {
    const unsigned row = fast_div(pos & 0x3fffffffu, p.wp_magic, p.wp_shift);
    const int x = static_cast<int>(pos - row * p.wp);
    const int img = static_cast<int>(fast_div(row, p.h_magic, p.h_shift));
    const int y = static_cast<int>(row) - img * p.h + up;
    const int pix = pos < p.positions && x < p.w ? static_cast<int>(row) * p.w + x : -1;
    table[kTabDy + slot] = pix >= 0 && y >= 0 && y < p.h ? pix + up * p.w : -1;
    if (!NHWC) table[kTabImg + slot] = img;
    return pix;
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int pair = lane + 32 * i;
    uint32_t four[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pix = place(q0 + 2 * pair + h, 2 * pair + h + (K == 3));
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
  if (K == 3 && lane < 2) place(lane ? q0 + kPos : q0 - 1, lane * (kPos + 1));
}

// One of the threads that bring x~. Warp w fills TMEM lanes 32 (w % 4) .., one
// 32-channel block, for a group's share of the positions; thread t of it takes
// four channels 4 (t / 4) + j, which land in lanes t / 4 + 8 j of the quadrant, at
// two positions in eight.
struct XStager {
  const WgradParams &p;
  static constexpr int kPairs = kPos / 8 / kXGroups;  // a thread's, four apart
  const int quad, pair0;  // of the first
  const uint8_t *src = nullptr;
  int none = 0;  // -1 behind the last channel
  uint32_t raw[2 * kPairs];

  __device__ explicit XStager(const WgradParams &params)
      : p(params), quad(threadIdx.x >> 5 & 3),
        pair0(4 * kPairs * (threadIdx.x >> 7) + (threadIdx.x & 3)) {}
  __device__ void set_load_unit(const Unit &un) {
    const int ch = un.ci0 + 32 * quad + (threadIdx.x >> 2 & 7) * 4;
    none = ch < p.cp ? 0 : -1;
    src = p.xq + ch;
  }
  __device__ __forceinline__ void load(int i, const int *table, int skip) {
    const int2 pix = *reinterpret_cast<const int2 *>(table + kTabX + 2 * (pair0 + 4 * i));
    const unsigned cp = static_cast<unsigned>(p.cp);
    raw[2 * i] = load4_if(pix.x | skip, src + static_cast<unsigned long long>(
                                                  static_cast<unsigned>(pix.x)) * cp);
    raw[2 * i + 1] = load4_if(pix.y | skip, src + static_cast<unsigned long long>(
                                                      static_cast<unsigned>(pix.y)) * cp);
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

// One of the threads that bring dy: an octet of output channels at slots
// first + kStep j. A 3x3 conv's stage has 130 slots, whose first two are the last
// two of the stage before; the threads of the last two carry them over.
template <int K, bool NHWC, bool WIDE>
struct DyStager {
  const WgradParams &p;
  static constexpr int kStep = 4 * kDyWarps, kCount = kPos / kStep;
  const int co8, first;
  const float *src = nullptr;
  int valid = 0;  // channels of the octet
  Oct raw[kCount];
  uint64_t scale[4];

  __device__ DyStager(const WgradParams &params, int t)
      : p(params), co8(NHWC ? t & 7 : t >> 5 & 7),
        first((NHWC ? t >> 3 : (t & 31) + (t >> 8) * 32) + (K - 1)) {}
  __device__ void set_load_unit(const Unit &un) {
    const int co = un.co0 + 8 * co8;
    valid = p.cout - co;
    src = p.dy + (NHWC ? static_cast<size_t>(co) : static_cast<size_t>(co) * p.h * p.w);
  }
  __device__ void set_unit(const Unit &un) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int co = un.co0 + 8 * co8 + i;
      f[i] = co < p.cout ? exp2i(dy_exponent(p.amax[co])) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) scale[i] = pk2(f[2 * i], f[2 * i + 1]);
  }
  // skip: -1 to load nothing (zeros)
  __device__ __forceinline__ void load_slot(Oct &r, int slot, const int *table, int skip) const {
    const int pix = table[kTabDy + slot] | skip;
    if (WIDE) {
      r = load32_if(valid > 0 ? pix : -1,
                    src + static_cast<unsigned long long>(static_cast<unsigned>(pix)) *
                              static_cast<unsigned>(p.cout));
      return;
    }
    if (NHWC) {
      r = load_oct<false, false>(src + static_cast<unsigned long long>(static_cast<unsigned>(pix)) *
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
      const uint64_t s = mul2(r.v[i], scale[i]);
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
    const int slot = first - kStep;
    if (K == 1 || slot < 0) return;
    if (contiguous) {
      st_shared16(at(stage, slot), ld_shared16(at(before, kPos + slot)));
      st_shared16(at(stage, slot) + kLo, ld_shared16(at(before, kPos + slot) + kLo));
    } else {
      Oct r;
      load_slot(r, slot, table, 0);
      store_slot(stage, slot, r);
    }
  }
};

// First (unit, stage) of SM range c.
__host__ __device__ __forceinline__ long long range_start(long long total, int grid, int c) {
  return total * c / grid;
}

// The SM range that holds stage g, the largest c with total * c < (g + 1) * grid:
// guessed in FP32 (c < 152, so at most one off) and put right.
__device__ __forceinline__ int range_of(long long total, int grid, long long g) {
  const long long bound = (g + 1) * grid;
  int c = static_cast<int>(__fdividef(static_cast<float>(bound), static_cast<float>(total)));
  while (total * c >= bound) --c;
  while (total * (c + 1) < bound) ++c;
  return c;
}

// Adds to a value that only this thread writes, in its order.
__device__ __forceinline__ void red_add(float *p, float v) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
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
  grid_release();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStagesA; ++i) {
      mbar_init(a_full + i, kXWarps);
      mbar_init(a_empty + i, TAPS);
    }
    for (int i = 0; i < kStagesB; ++i) {
      mbar_init(b_full + i, kDyWarps);
      mbar_init(b_empty + i, TAPS);
    }
    for (int i = 0; i < kTables; ++i) {
      mbar_init(tab_full + i, 1);
      mbar_init(tab_empty + i, kStageWarps);
    }
    mbar_init(acc_done, TAPS);
    mbar_init(acc_free, kStageWarps);
    *abort = 0u;
    fence_mbarrier_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  const long long g0 = range_start(p.total, gridDim.x, blockIdx.x);
  const int count = static_cast<int>(range_start(p.total, gridDim.x, blockIdx.x + 1) - g0);
  const Cursor start{static_cast<int>(g0 / p.stages), static_cast<int>(g0 % p.stages)};
  bool ok = true;

  if (warp < kStageWarps) {
    // Waits agree across the warp, so that a timeout leaves it converged.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_short(bar, parity, abort, p.wait_ns));
    };
    // Two at once: a wait that finds its phase complete still takes some 300 clocks.
    auto wait_both = [&](uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1) {
      const bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1);
      return __all_sync(0xffffffffu, r0 && r1) || (wait(b0, p0) && wait(b1, p1));
    };
    // TMEM lanes 32 (warp % 4) ..
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    uint32_t chains = 0;
    // Brings a finished chain's sums to the piece; called one stage behind its
    // last, when the next chain's first stage is on its way.
    auto drain = [&](int flags, int unit) {
      if (!ok || !(flags & kChainEnd)) return;
      ok = wait(acc_done, chains & 1);
      if (!ok) return;
      ++chains;
      tc_fence_after();
      // TMEM lane r of a quadrant is channel 4 (r % 8) + r / 8
      const size_t piece = static_cast<size_t>(unit) + blockIdx.x;
      float *o = p.part + piece * (TAPS * kTN * kTM) + (warp & 3) * 32 + 4 * (lane & 7) +
                 (lane >> 3);
#pragma unroll 1
      for (int c = warp >> 2; c < TAPS * kTN / 8; c += kStageWarps / 4) {
        const uint32_t at = t_lane + (c / (kTN / 8)) * 2 * kTN + c % (kTN / 8) * 8;
        float v[8], low[8];
        tmem_ld_8cols_pair(at, at + kTN, v, low);
        float *dst = o + c * 8 * kTM;
        if (flags & kFirstChain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j * kTM] = v[j] + low[j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) red_add(dst + j * kTM, v[j] + low[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free);
    };
    int flags = 0, unit = start.unit;  // of the stage before

    if (warp < kXWarps) {
      XStager st(p);
      st.set_load_unit(unit_at(p, start.unit));
      ok = wait(tab_full, 0);
      if (ok)
#pragma unroll
        for (int k = 0; k < st.kPairs; ++k) st.load(k, tables, st.none);
#pragma unroll 1
      for (int i = 0; i < count && ok; ++i) {
        const int *table = tables + (i % kTables) * kTableInts;
        const int *ahead = tables + ((i + 1) % kTables) * kTableInts;
        const bool more = i + 1 < count;
        const int next = more ? i + 1 : i;
        ok = wait_both(tab_full + next % kTables, (next / kTables) & 1, a_empty + i % kStagesA,
                       (i / kStagesA + 1) & 1);
        if (!ok) break;
        if (more && (ahead[kTabFlags] & kNewUnit)) st.set_load_unit(unit_at(p, ahead[kTabUnit]));
        tc_fence_after();
        const int skip = more ? st.none : -1;
        const uint32_t dst = t_lane + kAcc + (i % kStagesA) * (kPos / 2) +
                             (warp >> 2) * (4 * st.kPairs);
#pragma unroll
        for (int k = 0; k < st.kPairs; k += 4) {
          uint32_t low[8], high[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
            st.convert(k + j, table, o);
            low[2 * j] = o[0];
            low[2 * j + 1] = o[1];
            high[2 * j] = o[2];
            high[2 * j + 1] = o[3];
            st.load(k + j, ahead, skip);
          }
          tmem_st_16x16(dst + 4 * k, low);
          tmem_st_16x16(dst + 4 * k + (16u << 16), high);
        }
        const int2 head = *reinterpret_cast<const int2 *>(table);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(a_full + i % kStagesA);
          mbar_arrive(tab_empty + i % kTables);
        }
        drain(flags, unit);
        unit = head.x;
        flags = head.y;
      }
    } else {
      DyStager<K, NHWC, WIDE> st(p, threadIdx.x - 32 * kXWarps);
      const uint32_t base = smem_u32(smem);
      st.set_load_unit(unit_at(p, start.unit));
      st.set_unit(unit_at(p, start.unit));
      ok = wait(tab_full, 0);
      if (ok)
#pragma unroll
        for (int j = 0; j < st.kCount; ++j)
          st.load_slot(st.raw[j], st.first + st.kStep * j, tables, 0);
#pragma unroll 1
      for (int i = 0; i < count && ok; ++i) {
        const int *table = tables + (i % kTables) * kTableInts;
        const int *ahead = tables + ((i + 1) % kTables) * kTableInts;
        const bool more = i + 1 < count;
        const uint32_t stage = base + (i % kStagesB) * kStageBytes;
        const uint32_t before = base + ((i + kStagesB - 1) % kStagesB) * kStageBytes;
        const int next = more ? i + 1 : i;
        ok = wait_both(tab_full + next % kTables, (next / kTables) & 1, b_empty + i % kStagesB,
                       (i / kStagesB + 1) & 1);
        if (!ok) break;
        const int2 head = *reinterpret_cast<const int2 *>(table);
        if (i > 0 && (head.y & kNewUnit)) st.set_unit(unit_at(p, head.x));
        st.carry(stage, before, !(head.y & kNewUnit), table);
        if (more && (ahead[kTabFlags] & kNewUnit)) st.set_load_unit(unit_at(p, ahead[kTabUnit]));
#pragma unroll
        for (int j = 0; j < st.kCount; ++j) {
          st.store_slot(stage, st.first + st.kStep * j, st.raw[j]);
          st.load_slot(st.raw[j], st.first + st.kStep * j, ahead, more ? 0 : -1);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_full + i % kStagesB);
          mbar_arrive(tab_empty + i % kTables);
        }
        drain(flags, unit);
        unit = head.x;
        flags = head.y;
      }
    }
    if (count > 0) drain(flags, unit);
  } else if (warp < kTableWarp) {
    const int tap = warp - kIssueWarp;
    if (tap < TAPS && lane == 0) {
      constexpr uint32_t idesc = idesc_f16_tmem_a(kTM, 2 * kTN);
      const uint32_t acc = tmem + tap * 2 * kTN;
      const uint32_t base = smem_u32(smem);
      uint32_t chains = 0;
      bool fresh = true;
      // What the next stage needs is asked for before this one's MMAs are done.
      bool a_ready = false, b_ready = false;
      Cursor at = start;
      Chain chain;
      for (int i = 0; i < count && ok; ++i) {
        const int sa = i % kStagesA, sb = i % kStagesB;
        if (!a_ready) ok = mbar_wait_short(a_full + sa, (i / kStagesA) & 1, abort, p.wait_ns);
        if (ok && !b_ready) ok = mbar_wait_short(b_full + sb, (i / kStagesB) & 1, abort, p.wait_ns);
        if (ok && fresh && chains > 0)
          ok = mbar_wait_short(acc_free, (chains - 1) & 1, abort, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tmem + kAcc + sa * (kPos / 2);
        const uint64_t b = mn_major_desc(base + sb * kStageBytes, 128, kSbo) + (TAPS - 1 - tap);
#pragma unroll
        for (int k = 0; k < kPos / 16; ++k)
          umma_f16_tmem_a(acc, a + 8 * k, b + 16 * k, idesc, !fresh || k > 0);
        a_ready = mbar_try_wait(a_full + (i + 1) % kStagesA, ((i + 1) / kStagesA) & 1);
        b_ready = mbar_try_wait(b_full + (i + 1) % kStagesB, ((i + 1) / kStagesB) & 1);
        umma_commit(a_empty + sa);
        umma_commit(b_empty + sb);
        const bool piece_end = i == count - 1 || at.stage == p.stages - 1;
        at.next(p.stages);
        fresh = chain.ends(piece_end);
        if (fresh) {
          umma_commit(acc_done);
          ++chains;
        }
      }
      if (!ok) {
        // the MMAs issued so far finish before TMEM is freed
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {}
      }
    }
    __syncwarp();
  } else {
    const int first = warp - kTableWarp;
    Cursor at = start;
    Chain chain;
    int unit = -1;
    bool new_chain = true;  // the stage's chain is its piece's first
    Unit un{};
    uint32_t etop[4];
    for (int i = 0; i < count && ok; ++i) {
      const bool piece_end = i == count - 1 || at.stage == p.stages - 1;
      const bool chain_end = chain.ends(piece_end);
      const int flags = (i == 0 || at.stage == 0 ? kNewUnit : 0) | (chain_end ? kChainEnd : 0) |
                        (new_chain ? kFirstChain : 0);
      if (i % kTableWarps == first) {
        const int s = i % kTables;
        int *table = tables + s * kTableInts;
        if (i >= kTables)
          ok = __all_sync(0xffffffffu, mbar_wait_short(tab_empty + s, (i / kTables - 1) & 1, abort,
                                                       p.wait_ns));
        if (!ok) break;
        if (at.unit != unit) {
          unit = at.unit;
          un = unit_at(p, unit);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            etop[k] = (un.ci0 >> 5) + k < p.cp >> 5 ? p.emax[(un.ci0 >> 5) + k] : 0u;
        }
        if (lane == 0) *reinterpret_cast<int2 *>(table) = make_int2(unit, flags);
        make_table<K, NHWC>(p, static_cast<unsigned>(at.stage) * kPos, un, etop, lane, table);
        __syncwarp();
        if (lane == 0) mbar_arrive(tab_full + s);
      }
      at.next(p.stages);
      if (chain_end) new_chain = piece_end;
    }
  }
  if (!ok) {
    *abort = 1u;
    atomicCAS(p.err, 0, static_cast<int>(VAE_EDEVICE_TIMEOUT));
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------- before and after
constexpr int kScanThreads = 256;

// (Launched before the scan, which may start, and read, while this runs.)
__global__ void __launch_bounds__(1024) wgrad_zero(unsigned *maxima, int count) {
  grid_release();
  for (int i = threadIdx.x; i < count; i += 1024) maxima[i] = 0u;
}

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
                    const uint8_t *__restrict__ xs, int nb, float *psum, unsigned *amax,
                    unsigned *emax) {
  grid_release();
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
  grid_wait();
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
                    const uint8_t *__restrict__ xs, int nb, float *psum, unsigned *amax,
                    unsigned *emax) {
  __shared__ unsigned sm[128];
  __shared__ float rs[kScanThreads / 32];
  __shared__ unsigned rm[kScanThreads / 32];
  grid_release();
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
  grid_wait();
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

// grid (input-channel tiles + 1, cout), a group of kTM threads per ky: adds a
// unit's pieces in order, undoes the scaling and writes the taps of 128 input
// channels, contiguous in dw, through shared memory; the last column of blocks
// adds up dbias.
template <int K>
__global__ void __launch_bounds__(K *kTM)
    wgrad_reduce(const WgradParams p, int grid, const float *psum, int slabs, float *dw,
                 float *dbias) {
  __shared__ float out[kTM * K * K];
  grid_wait();
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
  const int ky = threadIdx.x / kTM, c = threadIdx.x % kTM;
  const int ci0 = blockIdx.x * kTM, ci = ci0 + c;
  const int e = ci < p.cin ? static_cast<int>(p.emax[ci >> 5]) - 127 - 7 - dy_exponent(p.amax[co])
                           : 0;
  const int u = (static_cast<int>(blockIdx.x) * p.co_tiles + co / kTN) * K + ky;
  const long long a = static_cast<long long>(u) * p.stages;
  const int c0 = range_of(p.total, grid, a), c1 = range_of(p.total, grid, a + p.stages - 1);
  const float *src = p.part + static_cast<size_t>(u + c0) * (K * kTN * kTM) + (co % kTN) * kTM + c;
  float v[K];
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll 8
  for (int i = c0; i <= c1; ++i, src += K * kTN * kTM)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += src[k * kTN * kTM];
#pragma unroll
  for (int k = 0; k < K; ++k) out[c * (K * K) + ky * K + k] = scalbnf(v[k], e);
  __syncthreads();
  const int count = min(kTM, p.cin - ci0) * K * K;
  float *o = dw + (static_cast<size_t>(co) * p.cin + ci0) * (K * K);
  for (int i = threadIdx.x; i < count; i += K * kTM) o[i] = out[i];
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
  VAE_CUDA_TRY(cudaFuncSetAttribute(wgrad_mma<K, NHWC, WIDE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem)));
  VAE_CUDA_TRY(launch_after(wgrad_mma<K, NHWC, WIDE>, grid, kMmaThreads, kSmem, s, p));
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
  wgrad_zero<<<1, 1024, 0, s>>>(ws.maxima, cout + nb);
  VAE_LAUNCH_CHECK();
  const bool wide = wide_ok(cout, dy);
  int slabs;
  if (nhwc) {
    const int per = kScanThreads / std::min(128, ceil_div(cout, 8));  // rows of a block's sweep
    slabs = static_cast<int>(std::max(1ll, std::min<long long>(ws.slabs, rows / (4 * per))));
    VAE_CUDA_TRY(launch_after(wide ? wgrad_scan_nhwc<true> : wgrad_scan_nhwc<false>,
                              dim3(slabs, ceil_div(cout, 1024)), kScanThreads, 0, s, dy, rows,
                              cout, x.scale, nb, ws.psum, ws.maxima, ws.maxima + cout));
  } else {
    slabs = std::max(1, std::min(ws.slabs, 8 * kSMs / cout));
    VAE_CUDA_TRY(launch_after(wgrad_scan_nchw, dim3(slabs, cout), kScanThreads, 0, s, dy, n, hw,
                              cout, x.scale, nb, ws.psum, ws.maxima, ws.maxima + cout));
  }
  VAE_TRY((k == 3 ? launch_mma<3> : launch_mma<1>)(p, nhwc, wide, ws.grid, s));
  VAE_CUDA_TRY(launch_after(k == 3 ? wgrad_reduce<3> : wgrad_reduce<1>,
                            dim3(ceil_div(cin, kTM) + 1, cout), k * kTM, 0, s, p, ws.grid, ws.psum,
                            slabs, dw, dbias));
  count_launches(4);
  return VAE_OK;
}

}  // namespace vae
