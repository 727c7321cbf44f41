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
// Eight warps stage (global -> registers -> halves -> shared memory) and drain
// the accumulators, one thread issues the MMAs.
#include "ptx.cuh"
#include "wgrad.cuh"

namespace vae {

namespace {

constexpr int kTM = 128;           // input channels of a tile (TMEM lanes)
constexpr int kTN = 64;            // output channels
constexpr int kPos = 128;          // positions of a stage
constexpr int kStages = 3;
constexpr int kChain = 16;         // stages between two drains: 2048 positions
constexpr int kProducers = 256;
constexpr int kMmaThreads = kProducers + 128;  // and a warpgroup of which one thread issues
// Registers: the launch gives every thread kLaunchRegs (65536 / 384, rounded
// down to a multiple of 8); the issuing warpgroup hands most of its share to
// the staging ones, which hold a third of the accumulators and a raw stage.
constexpr int kLaunchRegs = 168, kStageRegs = 232, kIssueRegs = 40;
static_assert(2 * kStageRegs + kIssueRegs <= 3 * kLaunchRegs, "the split fits the launch");
// Positions between two octets, odd so that 16-byte pieces of neighbouring
// octets fall into different banks.
constexpr int kSlotsA = kPos + 3, kSlotsB = kPos + 1;
constexpr uint32_t kSboA = kSlotsA * 16, kSboB = kSlotsB * 16;
constexpr uint32_t kBytesA = kTM / 8 * kSboA;      // 16 octets
constexpr uint32_t kBytesB = 2 * kTN / 8 * kSboB;  // hi, then lo
constexpr uint32_t kStageBytes = (kBytesA + kBytesB + 127) / 128 * 128;
constexpr size_t kSmem = kStages * kStageBytes + 256;
static_assert(kSmem <= 227 * 1024, "stages fit an SM");
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

// Raw data of one stage in a producer thread's registers.
struct Raw {
  float dy[4][8];
  uint4 x[5];
  uint32_t xs[5];
};

// K: the conv's kernel size. NHWC: the layout of dy.
template <int K, bool NHWC>
struct Producer {
  const WgradParams &p;
  const int t;
  // A: 16 input channels (two octets) at positions slot + 32 j; four threads
  // cover 64 contiguous bytes, eight lanes store to distinct banks.
  const int c16, a_slot;
  // B: an octet of output channels at positions b_slot + 32 j.
  const int co8, b_slot;

  __device__ explicit Producer(const WgradParams &params)
      : p(params), t(threadIdx.x), c16((t & 3) | ((t >> 7) << 2)), a_slot((t >> 2) & 31),
        co8(NHWC ? t & 7 : t >> 5), b_slot(NHWC ? t >> 3 : t & 31) {}

  __device__ void load_x(Raw &r, int j, unsigned pos, const Unit &un) const {
    const int ch = un.ci0 + 16 * c16;
    long long pix = -1;
    if (K == 1) {
      if (pos < p.positions) pix = pos;
    } else {
      const unsigned row = fast_div(pos, p.wp_magic, p.wp_shift);
      const int x = static_cast<int>(pos - row * p.wp) - 1;
      const int y = static_cast<int>(row - fast_div(row, p.h_magic, p.h_shift) * p.h) + un.ky - 1;
      if (x >= 0 && y >= 0 && y < p.h && row < static_cast<unsigned>(p.n * p.h))
        pix = (static_cast<long long>(row) + un.ky - 1) * p.w + x;
    }
    const bool in = pix >= 0 && ch < p.cp;
    r.x[j] = in ? __ldg(reinterpret_cast<const uint4 *>(p.xq + pix * p.cp + ch))
                : make_uint4(0, 0, 0, 0);
    r.xs[j] = in ? __ldg(p.xs + pix * (p.cp >> 5) + (ch >> 5)) : 0u;
  }

  __device__ void load(Raw &r, unsigned stage, const Unit &un) const {
    const unsigned q0 = stage * kPos;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned q = q0 + b_slot + 32 * j;
      const int co = un.co0 + 8 * co8;
      long long pix = -1;
      if (q < p.positions) {
        if (K == 1) {
          pix = q;
        } else {
          const unsigned row = fast_div(q, p.wp_magic, p.wp_shift);
          const int x = static_cast<int>(q - row * p.wp);
          if (x < p.w) pix = static_cast<long long>(row) * p.w + x;
        }
      }
      if (NHWC) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float *src = p.dy + pix * p.cout + co;
        const float4 a =
            pix >= 0 && co < p.cout ? __ldg(reinterpret_cast<const float4 *>(src)) : zero;
        const float4 b =
            pix >= 0 && co + 4 < p.cout ? __ldg(reinterpret_cast<const float4 *>(src) + 1) : zero;
        r.dy[j][0] = a.x;
        r.dy[j][1] = a.y;
        r.dy[j][2] = a.z;
        r.dy[j][3] = a.w;
        r.dy[j][4] = b.x;
        r.dy[j][5] = b.y;
        r.dy[j][6] = b.z;
        r.dy[j][7] = b.w;
      } else {
        const unsigned hw = static_cast<unsigned>(p.h) * p.w;
        const unsigned img = pix >= 0 ? static_cast<unsigned>(pix) / hw : 0u;
        const float *src = p.dy + (static_cast<long long>(img) * p.cout + co) * hw +
                           (pix - static_cast<long long>(img) * hw);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          r.dy[j][i] = pix >= 0 && co + i < p.cout ? __ldg(src + static_cast<long long>(i) * hw)
                                                   : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) load_x(r, j, q0 + a_slot + 32 * j, un);
    if (K == 3 && a_slot < 2) load_x(r, 4, q0 + 128 + a_slot, un);
  }

  // Scales of the unit whose stages are converted next.
  float sdy[8];
  uint32_t etop;
  __device__ void set_unit(const Unit &un) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int co = un.co0 + 8 * co8 + i;
      sdy[i] = co < p.cout ? exp2i(dy_exponent(__ldg(p.amax + co))) : 0.f;
    }
    const int ch = un.ci0 + 16 * c16;
    etop = ch < p.cp ? __ldg(p.emax + (ch >> 5)) : 0u;
  }

  // 16 channels at one position: times 2^(7 - d), d binades below the largest
  // block, as a half (below 2^-24 zero; a block of NaNs keeps them).
  __device__ void store_x(uint32_t a, const Raw &r, int j, int slot) const {
    const uint32_t d = r.xs[j] == 255u ? 7u : etop - r.xs[j];
    const uint32_t hb = d <= 21 ? (22 - d) << 10 : d <= 31 ? 1u << (31 - d) : 0u;
    const uint32_t two = hb | (hb << 16);
    const __half2 sc = *reinterpret_cast<const __half2 *>(&two);
    const uint32_t w[4] = {r.x[j].x, r.x[j].y, r.x[j].z, r.x[j].w};
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

  __device__ void store(uint32_t a, uint32_t b, const Raw &r) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = r.dy[j][2 * i] * sdy[2 * i], v1 = r.dy[j][2 * i + 1] * sdy[2 * i + 1];
        const __half2 h = __floats2half2_rn(v0, v1);
        const float2 f = __half22float2(h);
        hi[i] = h2_bits(h);
        lo[i] = h2_bits(__floats2half2_rn(v0 - f.x, v1 - f.y));
      }
      const uint32_t at = b + co8 * kSboB + (b_slot + 32 * j) * 16;
      st_shared16(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      st_shared16(at + kTN / 8 * kSboB, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) store_x(a, r, j, a_slot + 32 * j);
    if (K == 3 && a_slot < 2) store_x(a, r, 4, 128 + a_slot);
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
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);
  uint64_t *empty = full + kStages;
  uint64_t *acc_done = empty + kStages, *acc_free = acc_done + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + i, kProducers / 32);
      mbar_init(empty + i, 1);
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
  const int u0 = static_cast<int>(g0 / p.stages), s0 = static_cast<int>(g0 % p.stages);
  // Stage i of this SM: unit u0 + (s0 + i) / stages, stage (s0 + i) % stages.
  // A chain ends with its kChain stages, its unit or the range.
  auto unit_of = [&](int i) { return u0 + (s0 + i) / p.stages; };
  auto chain_end = [&](int i, bool *piece_end) {
    const int first = max(0, (s0 + i) / p.stages * p.stages - s0);  // the piece's first stage
    *piece_end = i == count - 1 || (s0 + i + 1) % p.stages == 0;
    return *piece_end || (i - first + 1) % kChain == 0;
  };
  auto give_up = [&]() {
    *abort = 1u;
    atomicCAS(p.err, 0, static_cast<int>(VAE_EDEVICE_TIMEOUT));
  };

  if (warp < kProducers / 32) {
    setmaxnreg_inc<kStageRegs>();
    Producer<K, NHWC> pr(p);
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    // This warp drains TMEM lanes 32 (warp % 4) .., output channels 32 (warp / 4) ..
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21) + (warp >> 2) * 32;
    float acc[TAPS][32];
#pragma unroll
    for (int k = 0; k < TAPS; ++k)
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[k][i] = 0.f;
    int drained = 0;     // stages whose chain end has been looked at
    uint32_t chains = 0;
    bool ok = true;
    auto drain_to = [&](int upto) {  // chains that end before stage `upto`
      for (; ok && drained < upto; ++drained) {
        bool piece_end;
        if (!chain_end(drained, &piece_end)) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(acc_done, chains & 1, abort, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < TAPS; ++k) {
          float v[32];
          tmem_ld_32cols(t_lane + k * 2 * kTN, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[k][i] += v[i];
          tmem_ld_32cols(t_lane + k * 2 * kTN + kTN, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[k][i] += v[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_free);
        ++chains;
        if (piece_end) {
          const size_t piece = static_cast<size_t>(unit_of(drained)) + blockIdx.x;
          float *o = p.part + piece * (TAPS * kTN * kTM) + (warp >> 2) * 32 * kTM +
                     (warp & 3) * 32 + lane;
#pragma unroll
          for (int k = 0; k < TAPS; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              o[(k * kTN + i) * kTM] = acc[k][i];
              acc[k][i] = 0.f;
            }
        }
      }
    };
    Raw raw;
    int unit = -1;
    if (count > 0) pr.load(raw, s0, unit_at(p, u0));
    for (int i = 0; i < count && ok; ++i) {
      const int s = i % kStages;
      if (unit_of(i) != unit) {
        unit = unit_of(i);
        pr.set_unit(unit_at(p, unit));
      }
      if (i >= kStages)
        ok = __all_sync(0xffffffffu,
                        mbar_wait(empty + s, (i / kStages - 1) & 1, abort, p.wait_ns));
      if (!ok) break;
      const uint32_t a = base + s * kStageBytes;
      pr.store(a, a + kBytesA, raw);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + s);
      if (i + 1 < count)
        pr.load(raw, (s0 + i + 1) % p.stages, unit_at(p, unit_of(i + 1)));
      // Two stages behind: by then the next chain's first stages are staged.
      drain_to(i - 1);
    }
    if (ok) drain_to(count);
    if (!ok) give_up();
  } else {
    setmaxnreg_dec<kIssueRegs>();
    if (threadIdx.x == kProducers) {
    constexpr uint32_t idesc = idesc_f16_mn(kTM, 2 * kTN);
    const uint32_t base = smem_u32(smem);
    uint32_t chains = 0;
    bool fresh = true, ok = true;
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
      bool piece_end;
      if (chain_end(i, &piece_end)) {
        umma_commit(acc_done);
        ++chains;
        fresh = true;
      }
    }
    if (!ok) {
      give_up();
      // the MMAs issued so far finish before TMEM is freed
      umma_commit(acc_done);
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000) {}
    }
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

// Largest scale byte below 255 of each 32-channel block; a share per block.
__device__ __forceinline__ void scan_scales(const uint8_t *__restrict__ xs, long long rows,
                                            int nb, unsigned *emax, unsigned *sm, int blk,
                                            int nblk) {
  for (int i = threadIdx.x; i < nb; i += kScanThreads) sm[i] = 0u;
  __syncthreads();
  const long long r0 = rows * blk / nblk, r1 = rows * (blk + 1) / nblk;
  const int per = kScanThreads / nb;  // rows at a time (nb <= 128)
  const int b = threadIdx.x % nb, l = threadIdx.x / nb;
  unsigned m = 0;
  if (l < per)
    for (long long r = r0 + l; r < r1; r += per) {
      const unsigned v = __ldg(xs + r * nb + b);
      if (v != 255u) m = max(m, v);
    }
  if (m) atomicMax(sm + b, m);
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
  ws.grid = static_cast<int>(
      std::min<long long>(kSMs, static_cast<long long>(ws.units) * ws.stages));
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
