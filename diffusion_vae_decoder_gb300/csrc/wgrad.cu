// wgrad.cu -- weight and bias gradient of the stride-1 convs (k = 1, 3) from
// dy and an 8-bit checkpoint x~ of the conv's input, on tcgen05.
//
//   dw[o][c][ky][kx] = sum_p dy[p][o] x~[p + (ky, kx) - k/2][c]
//
// A GEMM per tap whose reduction runs over the pixels: M = 128 input channels,
// N = 64 output channels. Both operands arrive pixel by pixel with channels
// next to each other, so both are M/N-major. An octet of channels takes a run
// of 16-byte pieces, one per pixel; the tap kx is the same tile read 16 kx
// bytes further on, so one staged tile serves three taps (TMEM holds three
// accumulators). Pixels are flattened over rows of w + 1 positions: the extra
// one, zero in both operands, is the padding on the right of its row and on
// the left of the next, so any 128 consecutive positions make a tile whatever
// w is. ky moves the input row: it is one of the grid's units.
//
// Precision. x~ is e4m3 times a power of two: a half holds it exactly once the
// block scales are taken relative to the largest of their 32 channels (blocks
// 2^22 below it round at 2^-24 of the largest). dy is scaled per output
// channel by a power of two to below 2^15 and split into two halves, hi + lo,
// 22 significant bits. The MMA reads [hi | lo] as 128 columns next to one A
// operand, so the two parts have accumulators of their own. The tensor core's
// accumulator truncates: measured on GB300, the sum of K/8 steps is off by
// about 5e-9 of its value per step. So a chain of MMAs ends after kChain
// stages; its sums move to FP32 registers, rounded to nearest.
//
// Schedule. (unit, stage) pairs, unit = (input-channel tile, output-channel
// tile, ky), are cut into equal contiguous ranges, one per SM, so that work
// stays balanced for any shape; every (unit, SM) piece writes a partial tile
// and a last pass adds a unit's pieces in order and undoes the scaling: the
// same inputs give the same bits.
//
// Sixteen warps stage: each thread copies its own 48 bytes of a half stage to
// shared memory three halves ahead (cp.async, no barrier: it reads back only
// what it copied), converts them and stores the operands; they also drain the
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
constexpr int kHalf = 64;          // positions that the staging threads take at once
constexpr int kStages = 2;         // staged operands
constexpr int kRaw = 3;            // raw halves in flight
constexpr int kTables = 4;
constexpr int kChain = 16;         // stages between two drains: 2048 positions
constexpr int kProducers = 512;    // staging threads: 16 warps
constexpr int kTableWarps = 3;     // each makes every third table
constexpr int kMmaThreads = kProducers + 128;  // one more warpgroup issues and makes tables
// Registers: the launch gives every thread kLaunchRegs (65536 / 640, rounded
// down to a multiple of 8); the last warpgroup hands its share to the staging
// ones, which hold the accumulators.
constexpr int kLaunchRegs = 96, kStageRegs = 104, kIssueRegs = 64;
static_assert(4 * kStageRegs + kIssueRegs <= 5 * kLaunchRegs, "the split fits the launch");
// Positions between two octets, odd so that 16-byte pieces of neighbouring
// octets fall into different banks.
constexpr int kSlotsA = kPos + 3, kSlotsB = kPos + 1;
constexpr uint32_t kSboA = kSlotsA * 16, kSboB = kSlotsB * 16;
constexpr uint32_t kBytesA = kTM / 8 * kSboA;      // 16 octets
constexpr uint32_t kBytesB = 2 * kTN / 8 * kSboB;  // hi, then lo
constexpr uint32_t kStageBytes = (kBytesA + kBytesB + 127) / 128 * 128;
// A raw half: 32 bytes of dy and 16 of x~ per staging thread, and the two
// further positions of x~ that the taps of a 3x3 conv reach (16 threads).
constexpr uint32_t kRawX = kProducers * 32, kRawMore = kRawX + kProducers * 16;
constexpr uint32_t kRawBytes = kRawMore + 16 * 16;
// A stage's table: per A slot the checkpoint row (-1: a zero) and the scales
// of the four 32-channel blocks (pairs of halves); per B position the dy pixel
// (-1: a zero) and its sample.
constexpr int kTabX = 0, kTabScale = kPos + 4, kTabDy = kTabScale + 4 * (kPos + 2),
              kTabImg = kTabDy + kPos, kTableInts = kTabImg + kPos;
constexpr size_t kSmem =
    kStages * kStageBytes + kRaw * kRawBytes + kTables * kTableInts * 4 + 256;
static_assert(kSmem <= 227 * 1024, "stages fit an SM");
static_assert(kRawBytes % 16 == 0 && kStageBytes % 16 == 0 && kTableInts % 4 == 0, "aligned");
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
__device__ __forceinline__ float ld_shared4(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
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

// The rows and scales of a stage's positions, by one warp. A slot `slot` is
// position q0 + slot read at tap kx = 0, so one to the left.
template <int K>
__device__ __forceinline__ void make_table(const WgradParams &p, unsigned q0, const Unit &un,
                                           const uint32_t *etop, int lane, int *table) {
  constexpr int kPasses = (kPos + K - 1 + 31) / 32;
  const int nb = p.cp >> 5, b0 = un.ci0 >> 5;
  int a[kPasses];
  uint32_t byte[kPasses][4];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int slot = lane + 32 * i;
    const unsigned pos = q0 + slot;
    int b = -1, img = 0;
    a[i] = -1;
    const unsigned row = fast_div(pos, p.wp_magic, p.wp_shift);
    const int x = static_cast<int>(pos - row * p.wp);
    img = static_cast<int>(fast_div(row, p.h_magic, p.h_shift));
    if (row < static_cast<unsigned>(p.n * p.h)) {
      if (K == 1) {
        a[i] = b = static_cast<int>(pos);
      } else {
        const int y = static_cast<int>(row) - img * p.h + un.ky - 1;
        if (x > 0 && y >= 0 && y < p.h)
          a[i] = (static_cast<int>(row) + un.ky - 1) * p.w + x - 1;
        if (x < p.w) b = static_cast<int>(row) * p.w + x;
      }
    }
    if (slot < kPos) {
      table[kTabDy + slot] = b;
      table[kTabImg + slot] = img;
    }
    if (slot < kPos + K - 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        byte[i][k] = a[i] >= 0 && b0 + k < nb
                         ? __ldg(p.xs + static_cast<size_t>(a[i]) * nb + b0 + k) : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int slot = lane + 32 * i;
    if (slot >= kPos + K - 1) continue;
    table[kTabX + slot] = a[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // 2^(7 - d), d binades below the largest block, as a half (zero under
      // 2^-25; whatever a block of NaNs is multiplied by, it stays NaN)
      const int e = 134 + static_cast<int>(byte[i][k]) - static_cast<int>(etop[k]);
      const float f = __uint_as_float(static_cast<uint32_t>(min(max(e, 0), 254)) << 23);
      table[kTabScale + 4 * slot + k] = static_cast<int>(h2_bits(__float2half2_rn(f)));
    }
  }
}

// K: the conv's kernel size. NHWC: the layout of dy.
template <int K, bool NHWC>
struct Producer {
  const WgradParams &p;
  const int t;
  // A: 16 input channels (two octets) at one position; four threads cover 64
  // contiguous bytes, eight lanes store to distinct banks.
  const int c16, a_slot;
  // B: an octet of output channels at one position.
  const int co8, b_slot;

  __device__ explicit Producer(const WgradParams &params)
      : p(params), t(threadIdx.x), c16((t & 3) | ((t >> 8) << 2)), a_slot((t >> 2) & 63),
        co8(NHWC ? t & 7 : t >> 6), b_slot(NHWC ? t >> 3 : t & 63) {}

  // Where this thread's channels start, for the unit whose stages are copied.
  const uint8_t *x_src;
  const float *dy_src;
  bool x_in;
  int dy_in;  // valid channels of the octet
  __device__ void set_copy_unit(const Unit &un) {
    const int ch = un.ci0 + 16 * c16, co = un.co0 + 8 * co8;
    x_in = ch < p.cp;
    x_src = p.xq + (x_in ? ch : 0);
    dy_in = min(8, p.cout - co);
    dy_src = dy_in > 0 ? p.dy + (NHWC ? static_cast<size_t>(co)
                                      : static_cast<size_t>(co) * p.h * p.w) : p.dy;
  }

  __device__ __forceinline__ void copy_x(uint32_t dst, int pix) const {
    const bool in = pix >= 0 && x_in;
    const unsigned long long off =
        static_cast<unsigned long long>(static_cast<unsigned>(in ? pix : 0)) *
        static_cast<unsigned>(p.cp);
    cp_async16(dst, x_src + off, in);
  }

  // Half `half` of a stage.
  __device__ __forceinline__ void copy(uint32_t raw, const int *table, int half) const {
    const int b_at = b_slot + kHalf * half, a_at = a_slot + kHalf * half;
    const int pix = table[kTabDy + b_at];
    if (NHWC) {
      const bool in = pix >= 0 && dy_in > 0;
      const float *src = dy_src + static_cast<unsigned long long>(
                                      static_cast<unsigned>(in ? pix : 0)) *
                                      static_cast<unsigned>(p.cout);
      cp_async16(raw + t * 16, src, in);
      const bool in4 = in && dy_in > 4;
      cp_async16(raw + kProducers * 16 + t * 16, in4 ? src + 4 : src, in4);
    } else {
      const size_t hw = static_cast<size_t>(p.h) * p.w;
      const int img = table[kTabImg + b_at];
      const float *src = dy_src + static_cast<size_t>(img) * (p.cout - 1) * hw + max(pix, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = pix >= 0 && i < dy_in;
        cp_async4(raw + i * (kProducers * 4) + t * 4, in ? src + i * hw : p.dy, in);
      }
    }
    copy_x(raw + kRawX + t * 16, table[kTabX + a_at]);
    if (K == 3 && half == 1 && a_slot < 2)
      copy_x(raw + kRawMore + (a_slot * 8 + c16) * 16, table[kTabX + kPos + a_slot]);
  }

  // Scales of dy for the unit whose stages are converted.
  float sdy[8];
  __device__ void set_unit(const Unit &un) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int co = un.co0 + 8 * co8 + i;
      sdy[i] = co < p.cout ? exp2i(dy_exponent(__ldg(p.amax + co))) : 0.f;
    }
  }

  __device__ __forceinline__ void store_x(uint32_t a, uint32_t raw, int slot,
                                          const int *table) const {
    const uint4 v = ld_shared16(raw);
    const uint32_t two = static_cast<uint32_t>(table[kTabScale + 4 * slot + (c16 >> 1)]);
    const __half2 sc = *reinterpret_cast<const __half2 *>(&two);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = h2_bits(__hmul2(e4m3x2_half2(w[i] & 0xffffu), sc));
      o[2 * i + 1] = h2_bits(__hmul2(e4m3x2_half2(w[i] >> 16), sc));
    }
    const uint32_t at = a + 2 * c16 * kSboA + slot * 16;
    st_shared16(at, make_uint4(o[0], o[1], o[2], o[3]));
    st_shared16(at + kSboA, make_uint4(o[4], o[5], o[6], o[7]));
  }

  __device__ __forceinline__ void store(uint32_t a, uint32_t b, uint32_t raw,
                                        const int *table, int half) const {
    uint64_t v[4];
    if (NHWC) {
      const uint4 d0 = ld_shared16(raw + t * 16);
      const uint4 d1 = ld_shared16(raw + kProducers * 16 + t * 16);
      v[0] = pk2(__uint_as_float(d0.x), __uint_as_float(d0.y));
      v[1] = pk2(__uint_as_float(d0.z), __uint_as_float(d0.w));
      v[2] = pk2(__uint_as_float(d1.x), __uint_as_float(d1.y));
      v[3] = pk2(__uint_as_float(d1.z), __uint_as_float(d1.w));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = pk2(ld_shared4(raw + 2 * i * (kProducers * 4) + t * 4),
                   ld_shared4(raw + (2 * i + 1) * (kProducers * 4) + t * 4));
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (the scaling is exact, so the difference is what hi dropped)
      v[i] = mul2(v[i], pk2(sdy[2 * i], sdy[2 * i + 1]));
      const __half2 h = __floats2half2_rn(lo2(v[i]), hi2(v[i]));
      const float2 f = __half22float2(h);
      const uint64_t rest = fma2(pk2(f.x, f.y), pk2(-1.f, -1.f), v[i]);
      hi[i] = h2_bits(h);
      lo[i] = h2_bits(__floats2half2_rn(lo2(rest), hi2(rest)));
    }
    const uint32_t at = b + co8 * kSboB + (b_slot + kHalf * half) * 16;
    st_shared16(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
    st_shared16(at + kTN / 8 * kSboB, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    store_x(a, raw + kRawX + t * 16, a_slot + kHalf * half, table);
    if (K == 3 && half == 1 && a_slot < 2)
      store_x(a, raw + kRawMore + (a_slot * 8 + c16) * 16, kPos + a_slot, table);
  }
};

// First (unit, stage) of SM range c.
__host__ __device__ __forceinline__ long long range_start(long long total, int grid, int c) {
  return total * c / grid;
}

template <int K, bool NHWC>
__global__ void __launch_bounds__(kMmaThreads, 1) wgrad_mma(const WgradParams p) {
  constexpr int TAPS = K;  // kx
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *raws = smem + kStages * kStageBytes;
  int *tables = reinterpret_cast<int *>(raws + kRaw * kRawBytes);
  uint64_t *full = reinterpret_cast<uint64_t *>(tables + kTables * kTableInts);
  uint64_t *empty = full + kStages;
  uint64_t *tab_full = empty + kStages, *tab_empty = tab_full + kTables;
  uint64_t *acc_done = tab_empty + kTables, *acc_free = acc_done + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + i, kProducers / 32);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < kTables; ++i) {
      mbar_init(tab_full + i, 1);
      mbar_init(tab_empty + i, kProducers / 32);
    }
    mbar_init(acc_done, 1);
    mbar_init(acc_free, kProducers / 32);
    *abort = 0u;
    fence_mbarrier_init();
  }
  constexpr uint32_t kCols = TAPS == 1 ? 128 : 512;
  if (warp == kProducers / 32) {
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

  if (warp < kProducers / 32) {
    setmaxnreg_inc<kStageRegs>();
    Producer<K, NHWC> pr(p);
    const uint32_t base = smem_u32(smem), raw0 = smem_u32(raws);
    bool ok = true;
    // Waits agree across the warp, so that a timeout leaves it converged.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, p.wait_ns));
    };

    // This warp drains TMEM lanes 32 (warp % 4) .., output channels 16 (warp / 4) ..
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21) + (warp >> 2) * 16;
    float acc[TAPS][16];
#pragma unroll
    for (int k = 0; k < TAPS; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[k][i] = 0.f;
    int drained = 0;  // stages whose chain end has been looked at
    uint32_t chains = 0;
    Cursor dr = start;
    Chain dr_chain;
    auto drain_to = [&](int upto) {  // chains that end before stage `upto`
      for (; ok && drained < upto; ++drained) {
        const bool piece_end = drained == count - 1 || dr.stage == p.stages - 1;
        const int unit = dr.unit;
        dr.next(p.stages);
        if (!dr_chain.ends(piece_end)) continue;
        ok = wait(acc_done, chains & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < TAPS; ++k) {
          float v[16];
          tmem_ld_16cols(t_lane + k * 2 * kTN, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[k][i] += v[i];
          tmem_ld_16cols(t_lane + k * 2 * kTN + kTN, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[k][i] += v[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_free);
        ++chains;
        if (piece_end) {
          const size_t piece = static_cast<size_t>(unit) + blockIdx.x;
          float *o = p.part + piece * (TAPS * kTN * kTM) + (warp >> 2) * 16 * kTM +
                     (warp & 3) * 32 + lane;
#pragma unroll
          for (int k = 0; k < TAPS; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[(k * kTN + i) * kTM] = acc[k][i];
              acc[k][i] = 0.f;
            }
        }
      }
    };

    // Copies run three halves ahead of the conversion: halves `ahead` of stage
    // `at`, into the raw buffers in turn.
    Cursor cp = start;
    int at = 0, ahead = 0;
    uint32_t raw_in = 0, raw_out = 0;
    pr.set_copy_unit(unit_at(p, cp.unit));
    auto copy = [&]() {
      if (at < count) {
        const int s = at % kTables;
        if (!ahead) ok = wait(tab_full + s, (at / kTables) & 1);
        if (ok) pr.copy(raw0 + raw_in, tables + s * kTableInts, ahead);
        if (ahead) {
          ++at;
          if (cp.next(p.stages) && at < count) pr.set_copy_unit(unit_at(p, cp.unit));
        }
        ahead ^= 1;
      }
      cp_async_commit();
      raw_in = raw_in == (kRaw - 1) * kRawBytes ? 0 : raw_in + kRawBytes;
    };
    Cursor cv = start;  // the stage that is converted
    pr.set_unit(unit_at(p, cv.unit));
    for (int i = 0; i < kRaw && ok; ++i) copy();
#pragma unroll 1
    for (int i = 0; i < count && ok; ++i) {
      const int s = i % kStages;
      if (i >= kStages) ok = wait(empty + s, (i / kStages - 1) & 1);
      if (!ok) break;
      const uint32_t a = base + s * kStageBytes;
      const int *table = tables + (i % kTables) * kTableInts;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        cp_async_wait<kRaw - 1>();
        pr.store(a, a + kBytesA, raw0 + raw_out, table, half);
        raw_out = raw_out == (kRaw - 1) * kRawBytes ? 0 : raw_out + kRawBytes;
        copy();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full + s);
        mbar_arrive(tab_empty + i % kTables);
      }
      if (cv.next(p.stages) && i + 1 < count) pr.set_unit(unit_at(p, cv.unit));
      // One stage behind: the next chain's first stage is staged by then.
      drain_to(i);
    }
    if (ok) drain_to(count);
    cp_async_wait<0>();
    if (!ok) give_up();
  } else {
    setmaxnreg_dec<kIssueRegs>();
    if (threadIdx.x == kProducers) {
      constexpr uint32_t idesc = idesc_f16_mn(kTM, 2 * kTN);
      const uint32_t base = smem_u32(smem);
      uint32_t chains = 0;
      bool fresh = true, ok = true;
      Cursor at = start;
      Chain chain;
      for (int i = 0; i < count && ok; ++i) {
        const int s = i % kStages;
        if (fresh && chains > 0) ok = mbar_wait(acc_free, (chains - 1) & 1, abort, p.wait_ns);
        if (ok) ok = mbar_wait(full + s, (i / kStages) & 1, abort, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = mn_major_desc(base + s * kStageBytes, 128, kSboA);
        const uint64_t bd = mn_major_desc(base + s * kStageBytes + kBytesA, 128, kSboB);
#pragma unroll
        for (int k = 0; k < kPos / 16; ++k)
#pragma unroll
          for (int tap = 0; tap < TAPS; ++tap)
            umma_f16(tmem + tap * 2 * kTN, ad + 16 * k + tap, bd + 16 * k, idesc,
                     !fresh || k > 0);
        fresh = false;
        umma_commit(empty + s);
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
    } else if (warp > kProducers / 32) {
      const int first = warp - kProducers / 32 - 1;
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
  if (warp == kProducers / 32) {
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
// each output channel. The maxima do not depend on the order of the atomics.
__global__ void __launch_bounds__(kScanThreads)
    wgrad_scan_nhwc(const float *__restrict__ dy, long long rows, int cout,
                    const uint8_t *__restrict__ xs, int nb, float *__restrict__ psum,
                    unsigned *__restrict__ amax, unsigned *__restrict__ emax) {
  __shared__ unsigned sm[128];
  __shared__ float4 rs[kScanThreads], rm[kScanThreads];
  const int c0 = blockIdx.y * 1024, quads = min(1024, cout - c0) / 4;
  const int per = kScanThreads / quads, q = threadIdx.x % quads, l = threadIdx.x / quads;
  const long long r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  uint4 m = make_uint4(0, 0, 0, 0);
  if (l < per) {
    const float *src = dy + c0 + 4 * q;
    auto add = [&](float4 v) {
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
      m.x = max(m.x, abs_bits(v.x));
      m.y = max(m.y, abs_bits(v.y));
      m.z = max(m.z, abs_bits(v.z));
      m.w = max(m.w, abs_bits(v.w));
    };
    long long r = r0 + l;
    for (; r + 3 * per < r1; r += 4 * per) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = __ldg(reinterpret_cast<const float4 *>(src + (r + u * per) * cout));
#pragma unroll
      for (int u = 0; u < 4; ++u) add(v[u]);
    }
    for (; r < r1; r += per) add(__ldg(reinterpret_cast<const float4 *>(src + r * cout)));
  }
  rs[threadIdx.x] = s;
  rm[threadIdx.x] = make_float4(__uint_as_float(m.x), __uint_as_float(m.y),
                                __uint_as_float(m.z), __uint_as_float(m.w));
  __syncthreads();
  if (threadIdx.x < quads) {
    for (int k = 1; k < per; ++k) {
      const float4 a = rs[k * quads + q], b = rm[k * quads + q];
      s = make_float4(s.x + a.x, s.y + a.y, s.z + a.z, s.w + a.w);
      m = make_uint4(max(m.x, __float_as_uint(b.x)), max(m.y, __float_as_uint(b.y)),
                     max(m.z, __float_as_uint(b.z)), max(m.w, __float_as_uint(b.w)));
    }
    *reinterpret_cast<float4 *>(psum + static_cast<size_t>(blockIdx.x) * cout + c0 + 4 * q) = s;
    atomicMax(amax + c0 + 4 * q, m.x);
    atomicMax(amax + c0 + 4 * q + 1, m.y);
    atomicMax(amax + c0 + 4 * q + 2, m.z);
    atomicMax(amax + c0 + 4 * q + 3, m.w);
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

// Blocks (128 threads: input channels) x output channel x (ky, and one more
// for dbias): adds a unit's pieces in order and undoes the scaling.
template <int K>
__global__ void __launch_bounds__(kTM)
    wgrad_reduce(const WgradParams p, int grid, const float *__restrict__ psum, int slabs,
                 float *__restrict__ dw, float *__restrict__ dbias) {
  const int co = blockIdx.y;
  if (blockIdx.z == K) {
    if (blockIdx.x > 0 || !dbias || threadIdx.x >= 32) return;
    float s = 0.f;
    for (int i = threadIdx.x; i < slabs; i += 32) s += psum[static_cast<size_t>(i) * p.cout + co];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) dbias[co] = s;
    return;
  }
  const int ci = blockIdx.x * kTM + threadIdx.x, ky = blockIdx.z;
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
  if (ci >= p.cin) return;
  const int e = static_cast<int>(p.emax[ci >> 5]) - 127 - 7 - dy_exponent(p.amax[co]);
  float *o = dw + (static_cast<size_t>(co) * p.cin + ci) * (K * K) + ky * K;
#pragma unroll
  for (int k = 0; k < K; ++k) o[k] = scalbnf(v[k], e);
}

int floor_log2(unsigned d) {
  int l = 0;
  while (d >> (l + 1)) ++l;
  return l;
}

struct WgradWs {
  float *psum, *part;
  unsigned *maxima;  // amax [cout], emax [cp / 32]
  int slabs, grid, units, stages;
};

WgradWs carve_wgrad(Carver &cv, int n, int cin, int h, int w, int cout, int k) {
  WgradWs ws{};
  const long long rows = static_cast<long long>(n) * h * w;
  ws.slabs = static_cast<int>(std::max(1ll, std::min<long long>(4 * kSMs, rows / 64)));
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

template <int K, bool NHWC>
int launch_mma(const WgradParams &p, int grid, cudaStream_t s) {
  // (the register split waits for what the launch did not bring)
  static const int regs = [] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, wgrad_mma<K, NHWC>) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs != kLaunchRegs) return VAE_ECUDA;
  VAE_CUDA_TRY(cudaFuncSetAttribute(wgrad_mma<K, NHWC>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem)));
  wgrad_mma<K, NHWC><<<grid, kMmaThreads, kSmem, s>>>(p);
  VAE_LAUNCH_CHECK();
  return VAE_OK;
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
  if (nhwc) {
    wgrad_scan_nhwc<<<dim3(ws.slabs, ceil_div(cout, 1024)), kScanThreads, 0, s>>>(
        dy, rows, cout, x.scale, nb, ws.psum, ws.maxima, ws.maxima + cout);
  } else {
    const int slabs = std::max(1, std::min(ws.slabs, 8 * kSMs / cout));
    wgrad_scan_nchw<<<dim3(slabs, cout), kScanThreads, 0, s>>>(
        dy, n, hw, cout, x.scale, nb, ws.psum, ws.maxima, ws.maxima + cout);
  }
  VAE_LAUNCH_CHECK();
  const int slabs = nhwc ? ws.slabs : std::max(1, std::min(ws.slabs, 8 * kSMs / cout));
  if (k == 3)
    VAE_TRY((nhwc ? launch_mma<3, true> : launch_mma<3, false>)(p, ws.grid, s));
  else
    VAE_TRY((nhwc ? launch_mma<1, true> : launch_mma<1, false>)(p, ws.grid, s));
  const dim3 rg(ceil_div(cin, kTM), cout, k + 1);
  if (k == 3)
    wgrad_reduce<3><<<rg, kTM, 0, s>>>(p, ws.grid, ws.psum, slabs, dw, dbias);
  else
    wgrad_reduce<1><<<rg, kTM, 0, s>>>(p, ws.grid, ws.psum, slabs, dw, dbias);
  VAE_LAUNCH_CHECK();
  count_launches(3);
  return VAE_OK;
}

}  // namespace vae
