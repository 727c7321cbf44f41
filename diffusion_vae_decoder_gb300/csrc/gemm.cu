// gemm.cu -- out = epilogue(A B^T) on the tcgen05 tensor cores, for operands of
// 16-bit numbers whose reduction runs along a row or along a column.
//
// Stages of 64 reduction indexes are copied by TMA with the 128-byte swizzle: for a
// K-major operand one box of 64 numbers a row, for the other a box of 64 rows for
// every 64 result indexes; both lie in shared memory as the tensor core reads them,
// so no operand is transposed. Numbers outside the matrices arrive as zeros, in both
// operands along the reduction.
//
// A float is the exact sum of three bf16 numbers h + m + l, each the nearest to what
// is left; the products hh, hm, mh, mm, hl, lh are added up in one accumulator, what
// is left out (ml, lm, ll) is below 2^-24 of a product. The tensor core's
// accumulator truncates (measured: about 1e-8 of the sum for every step of 16), so
// that sums that leave as floats move to registers after every 32 steps; sums that
// leave as 16-bit numbers do not need it.
#include <atomic>

#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace vae {

namespace {

constexpr int kBK = 64;     // reduction indexes of a stage
constexpr int kChain = 8;   // stages after which a float's sum leaves the accumulator

struct Params {
  long long m;
  int n;
  int its;    // stages of a tile: 64-index blocks of k times `pairs`
  int pairs;  // products of parts: 1 or 6
  int m_tiles, n_tiles;
  int slices;         // of the reduction, whose sums a later launch adds up
  bool a_k, b_k;
  bool wait;
  uint32_t idesc;
  uint32_t stage_bytes;  // that the copies of a small tile's stage bring
  uint64_t wait_ns;
  int *err;
  int inject;  // test hook: VAE_INJECT_* bits (0 in normal operation)
  int kind;
  GemmEpilogue e;
  GemmColumnSums cols;
};

// A wait ran out: the block's other waits give up as well, and a pair's other block's.
template <bool PAIR>
__device__ __forceinline__ void raise_error(const Params &p, volatile uint32_t *abort) {
  *abort = 1u;
  if constexpr (PAIR)
    st_cluster(mapa_rank(const_cast<const uint32_t *>(abort), cluster_ctarank() ^ 1), 1u);
  atomicCAS(p.err, 0, static_cast<int>(VAE_EDEVICE_TIMEOUT));
}
// Waits for products or copies that are under way before a block leaves: 10 ms at
// most, whatever limit the other waits have, where they take microseconds.
constexpr uint64_t kDrainNs = 10000000;
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kDrainNs) return;
}

// 64 reduction indexes from k0 on of 128 rows of an operand, 16 KB; `load(dst, map, c0,
// c1, c2)` issues one copy.
constexpr int kOperandBytes = 128 * kBK * 2;
template <class L>
__device__ __forceinline__ void load_operand(const CUtensorMap *map, bool k_major, int k0, int row,
                                             int part, uint8_t *dst, L &&load) {
  if (k_major) {
    load(dst, map, k0, row, part);
  } else {
    load(dst, map, row, k0, part);
    load(dst + kBK * 128, map, row + 64, k0, part);
  }
}
// What the tensor core is told of the stages: descriptors of stage 0's operands, and
// how far a step of 16 reduction indexes and a stage move them (in units of 16 bytes;
// the address is their low word's).
struct Operands {
  uint64_t a, b;
  uint32_t step_a, step_b;
};
__device__ __forceinline__ Operands operands_at(const Params &p, uint32_t sa, uint32_t sb) {
  return {p.a_k ? sw128_kmajor_desc(sa) : sw128_mnmajor_desc(sa, kBK * 128),
          p.b_k ? sw128_kmajor_desc(sb) : sw128_mnmajor_desc(sb, kBK * 128),
          (p.a_k ? 32u : 2048u) >> 4, (p.b_k ? 32u : 2048u) >> 4};
}
// The four steps of stage `s`, of `bytes` a stage.
template <bool PAIR>
__device__ __forceinline__ void multiply_stage(const Operands &o, uint32_t idesc, int s,
                                               uint32_t bytes, uint32_t acc, bool first) {
  const uint64_t a = o.a + s * (bytes >> 4), b = o.b + s * (bytes >> 4);
#pragma unroll
  for (int k = 0; k < kBK / 16; ++k)
    umma_16bit<PAIR>(acc, a + k * o.step_a, b + k * o.step_b, idesc, !(first && k == 0));
}

// A place in a ring of N stages and the parity of its round; a thread alone goes
// through it, so that a division a step would be most of its time.
template <int N>
struct Ring {
  int s = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      round ^= 1;
    }
  }
};
// After an abort, which may come when a block has asked for its last copies already, and
// a barrier of all threads: the last of the `asked` stages of a ring of N land. (Those
// before them were multiplied, or their places would not have been asked for again.)
template <int N>
__device__ __forceinline__ void drain_stages(uint64_t *full, uint64_t asked) {
  for (uint64_t i = asked > N ? asked - N : 0; i < asked; ++i)
    drain_wait(full + i % N, i / N & 1);
}
// The same on a pair's leader, whose barriers count both blocks' copies, `bytes` of each
// a stage: the stages that one block alone has asked for are put right first.
template <int N>
__device__ __forceinline__ void drain_pair(uint64_t *full, const volatile uint64_t *asked,
                                           uint32_t bytes) {
  const uint64_t mine = asked[0], theirs = asked[1];
  for (uint64_t i = mine; i < theirs; ++i) mbar_arrive_expect_tx(full + i % N, bytes);
  for (uint64_t i = theirs; i < mine; ++i) mbar_complete_tx(full + i % N, bytes);
  drain_stages<N>(full, max(mine, theirs));
}

// Floats: 64 reduction indexes are six stages of one operand's 16 KB, in the order
// A's h, B's h, m, l, A's m, l, and six products, hh, hm, hl, mh, mm, lh, so that each
// part is copied once and leaves when its last product has been issued.
template <bool PAIR, int N, class L>
__device__ __forceinline__ bool copy_parts(const Params &p, const CUtensorMap *ta,
                                           const CUtensorMap *tb, uint8_t *smem, uint64_t *full,
                                           uint64_t *empty, int block, int blocks, int withheld,
                                           int m0, int n0, bool leader, volatile uint32_t *abort,
                                           int lane, Ring<N> *r, uint64_t *asked, L &&load) {
  for (int i = 0; i < 6 * blocks - withheld; ++i, ++*asked, r->next()) {
    bool ok = mbar_wait(empty + r->s, r->round ^ 1, abort, p.wait_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0) raise_error<PAIR>(p, abort);
      return false;
    }
    const int tile = i % 6, k0 = (block + i / 6) * kBK;
    const bool is_a = tile == 0 || tile > 3;
    const int part = is_a ? max(tile - 3, 0) : tile - 1;
    if (elect_one()) {
      if (leader) mbar_arrive_expect_tx(full + r->s, (PAIR ? 2 : 1) * kOperandBytes);
      load_operand(is_a ? ta : tb, is_a ? p.a_k : p.b_k, k0, is_a ? m0 : n0, part,
                   smem + r->s * kOperandBytes,
                   [&](uint8_t *dst, const CUtensorMap *m, int c0, int c1, int c2) {
                     load(dst, m, full + r->s, c0, c1, c2);
                   });
    }
    __syncwarp();
  }
  return true;
}
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (PAIR)
    umma_commit_pair(bar, 3);
  else
    umma_commit(bar);
}
// The products of `blocks` of them, into accumulators c, c + 1, ... of kAccCols columns.
template <bool PAIR, int N, int ACC_COLS>
__device__ __forceinline__ bool multiply_parts(const Params &p, const Operands &o, uint64_t *full,
                                               uint64_t *empty, uint64_t *acc_full,
                                               uint64_t *acc_empty, uint32_t tmem, int blocks,
                                               volatile uint32_t *abort, int lane, Ring<N> *r,
                                               int *c) {
  const uint32_t idesc = p.idesc;
  int step = 0;
  for (int b = 0; b < blocks; ++b) {
#pragma unroll
    for (int q = 0; q < 6; ++q, ++step) {
      // places of the operands among the six stages, and what is new with this product
      const int ia = q < 3 ? 0 : q < 5 ? 4 : 5, ib = q < 3 ? 1 + q : q == 4 ? 2 : 1;
      const int fresh = q == 0 ? 2 : q == 4 ? 0 : 1;
      const bool first = step % kChain == 0;
      const bool last = step % kChain == kChain - 1 || (b == blocks - 1 && q == 5);
      auto stage = [&](int i) { return r->s + i < N ? r->s + i : r->s + i - N; };
      auto round = [&](int i) { return r->s + i < N ? r->round : r->round ^ 1; };
      bool ok = true;
      if (first)
        ok = mbar_wait(acc_empty + (*c & 1), (*c >> 1 & 1) ^ 1, abort, p.wait_ns);
      if (fresh == 2) ok = ok && mbar_wait(full + stage(0), round(0), abort, p.wait_ns);
      const int last_in = q < 3 ? ib : ia;
      if (fresh) ok = ok && mbar_wait(full + stage(last_in), round(last_in), abort, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) raise_error<PAIR>(p, abort);
        return false;
      }
      tc_fence_after();
      const uint64_t a = o.a + stage(ia) * (kOperandBytes >> 4);
      const uint64_t bd = o.b + stage(ib) * (kOperandBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          umma_16bit<PAIR>(tmem + (*c & 1) * ACC_COLS, a + k * o.step_a, bd + k * o.step_b, idesc,
                           !(first && k == 0));
        if (q == 2) {
          commit<PAIR>(empty + stage(0));
          commit<PAIR>(empty + stage(3));
        }
        if (q == 4) {
          commit<PAIR>(empty + stage(2));
          commit<PAIR>(empty + stage(4));
        }
        if (q == 5) {
          commit<PAIR>(empty + stage(1));
          commit<PAIR>(empty + stage(5));
        }
        if (last) commit<PAIR>(acc_full + (*c & 1));
      }
      __syncwarp();
      *c += last;
    }
    for (int i = 0; i < 6; ++i) r->next();
  }
  return true;
}

// Sums of A's columns (the result's rows), by warps that wait for the tensor core: the
// rows that the copies bring in at the same time are read once more, from L2, by one of
// the tiles that share them: on pairs of SMs tile column j takes blocks j, j + n_tiles,
// ... of 64 rows (small tiles: the first column all of them).
// Warp w of W takes every W-th pair of a block's rows of 128 numbers, a lane eight of
// them, which it copies into its own places of the warp's buffer (kColumnBytes) and
// adds up a chain of products later. (Through registers, whose loads the warp would
// have to wait for, the call took 124 us instead of 89.)
constexpr int kColumnBytes = 4096;
struct Columns {
  Oct sum = {{0, 0, 0, 0}};
  int next = 0;                // block of 64 rows
  int oldest = 0, waiting = 0;  // place and number of the blocks in the buffer
};
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
// Asks for the blocks before `end`, adding up the oldest one whenever the buffer is
// full; `rest`: what is in it as well.
template <int W, class D>
__device__ __forceinline__ void turn_blocks(const Params &p, uint8_t *buf, int end, bool rest,
                                            long long m0, int w, int lane, Columns *c) {
  constexpr int R = kBK / (2 * W), kLane = 8 * sizeof(D);  // rows of a lane's; bytes of a row
  constexpr int kBlock = R * 32 * kLane, kSlots = kColumnBytes / kBlock;
  const long long ch = m0 + 8 * (lane & 15);
  buf += 16 * lane;
  auto add_oldest = [&] {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Raw<D> v;
#pragma unroll
      for (int h = 0; h < kLane / 16; ++h)
        v.v[h] = *reinterpret_cast<const uint4 *>(buf + c->oldest * kBlock +
                                                  (i * kLane / 16 + h) * 512);
      const Oct o = oct_of(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) c->sum.v[j] = add2(c->sum.v[j], o.v[j]);
    }
    c->oldest = c->oldest + 1 == kSlots ? 0 : c->oldest + 1;
    --c->waiting;
  };
#pragma unroll 1
  for (; c->next < end; c->next += p.cols.step) {
    if (c->waiting == kSlots) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
      add_oldest();
    }
    const int slot = c->oldest + c->waiting;
    const uint32_t to = smem_u32(buf) + (slot < kSlots ? slot : slot - kSlots) * kBlock;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const long long r = static_cast<long long>(c->next) * kBK + 2 * (w + W * i) + (lane >> 4);
      const bool in = r < p.cols.rows && ch < p.m;
      const D *src = static_cast<const D *>(p.cols.src) + (in ? r * p.m + ch : 0);
#pragma unroll
      for (int h = 0; h < kLane / 16; ++h)
        copy16(to + (i * kLane / 16 + h) * 512, src + 8 / (kLane / 16) * h, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++c->waiting;
  }
  if (!rest) return;
  asm volatile("cp.async.wait_all;" ::: "memory");
  while (c->waiting) add_oldest();
}
// The blocks that stages before `it` belong to.
template <int W>
__device__ __forceinline__ void add_columns(const Params &p, uint8_t *buf, int it, bool rest,
                                            long long m0, int w, int lane, Columns *c) {
  if (!p.cols.part) return;
  const int end = p.pairs > 1 ? (it + p.pairs - 1) / p.pairs : it;
  if (p.cols.dtype == VAE_F32)
    turn_blocks<W, float>(p, buf, end, rest, m0, w, lane, c);
  else if (p.cols.dtype == VAE_BF16)
    turn_blocks<W, bf16>(p, buf, end, rest, m0, w, lane, c);
  else
    turn_blocks<W, __half>(p, buf, end, rest, m0, w, lane, c);
}
// A warp's sums, eight columns each in lanes 0 to 15.
template <int W>
__device__ __forceinline__ Oct end_columns(const Params &p, uint8_t *buf, long long m0, int w,
                                           int lane, Columns *c) {
  add_columns<W>(p, buf, 0, true, m0, w, lane, c);
  __syncwarp();  // (the buffer is the warp's again)
  Oct sum = c->sum;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    sum.v[j] = add2(sum.v[j], __shfl_xor_sync(0xffffffffu, sum.v[j], 16));
  return sum;
}

// ------------------------------------------------------------------ small tiles
// A 128 x 128 tile by a cluster of blocks that split the reduction: each adds up its
// share of the stages, puts its sums into shared memory, and finishes 128 / S rows of
// the tile from all of them, in the order of the blocks. Warp 0 copies, warp 1
// multiplies, the others take the sums out.
constexpr int kTile = 128;
constexpr int kTileStages = 6;
constexpr int kTileSlots = 2 * kTileStages;  // of one operand
constexpr int kMaxSplits = 8;  // blocks of a cluster
constexpr int kTileWarps = 8;  // that take sums out, 64 columns each
constexpr int kTileCols = 4 * kTile / kTileWarps;
constexpr int kTileThreads = 64 + 32 * kTileWarps;
constexpr int kTileStageBytes = 2 * kOperandBytes;
constexpr int kSumLd = kTile + 4;  // floats of a row of sums: 16 bytes shift the banks
constexpr size_t kTileSmem =
    kTileStages * kTileStageBytes + kTileWarps * kColumnBytes + 1024 + 256;
static_assert(kTileSmem <= 227 * 1024 && (2 * kTileSlots + 5) * 8 + 16 <= 256, "barriers");
static_assert(kTile * kSumLd * 4 <= kTileStages * kTileStageBytes, "sums lie over the stages");

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
template <class Out>
__global__ void __launch_bounds__(kTileThreads, 1)
    gemm_tile(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
              const __grid_constant__ Params p, int splits) {
  constexpr bool kFloat = sizeof(Out) == 4;
  constexpr uint32_t kTmem = kFloat ? 2 * kTile : kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kTileStages * kTileStageBytes +
                                                kTileWarps * kColumnBytes);
  uint64_t *empty = full + kTileSlots;
  uint64_t *acc_full = empty + kTileSlots, *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  volatile uint64_t *asked_of = reinterpret_cast<uint64_t *>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / splits, rank = blockIdx.x % splits;
  const int tiles = p.m_tiles * p.n_tiles, slice = unit / tiles, tile = unit - slice * tiles;
  const int m0 = tile / p.n_tiles * kTile, n0 = tile % p.n_tiles * kTile;
  const int share_of = slice * splits + rank, shares = p.slices * splits;
  const long long all = p.its / p.pairs;  // blocks of 64 reduction indexes
  const int block0 = static_cast<int>(all * share_of / shares);
  const int blocks = static_cast<int>(all * (share_of + 1) / shares) - block0;
  const int it0 = block0 * p.pairs, its = blocks * p.pairs;
  // the tiles of the first column take the sums of A's columns
  const bool columns = kFloat && p.cols.part && n0 == 0;
  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int i = 0; i < kTileSlots; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, kTileWarps + !!(p.inject & VAE_INJECT_WITHHOLD_ACCUMULATOR));
    }
    mbar_init(drain, 1);
    fence_mbarrier_init();
    *abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.wait) grid_wait();

  if (warp == 0) {
    const int withheld = !!(p.inject & VAE_INJECT_WITHHOLD_COPY);
    uint64_t asked = 0;
    if (kFloat && p.pairs > 1) {
      Ring<kTileSlots> r;
      copy_parts<false>(p, &ta, &tb, smem, full, empty, block0, blocks, withheld, m0, n0, true,
                        abort, lane, &r, &asked,
                        [](uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1,
                           int c2) { tma_load_3d(dst, m, bar, c0, c1, c2); });
    } else {
      Ring<kTileStages> r;
      int i = 0;
      for (; i < its - withheld; ++i, r.next()) {
        bool ok = mbar_wait(empty + r.s, r.round ^ 1, abort, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) raise_error<false>(p, abort);
          break;
        }
        uint64_t *bar = full + r.s;
        uint8_t *a = smem + r.s * kTileStageBytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, p.stage_bytes);
          auto load = [&](uint8_t *dst, const CUtensorMap *m, int c0, int c1, int c2) {
            tma_load_3d(dst, m, bar, c0, c1, c2);
          };
          load_operand(&ta, p.a_k, (it0 + i) * kBK, m0, 0, a, load);
          load_operand(&tb, p.b_k, (it0 + i) * kBK, n0, 0, a + kOperandBytes, load);
        }
        __syncwarp();
      }
      asked = i;
    }
    if (lane == 0) *asked_of = asked;
  } else if (warp == 1) {
    // The whole warp goes through the loop, so that descriptors stay in registers that
    // all lanes share, and one lane issues (the same one every time).
    if (kFloat && p.pairs > 1) {
      const Operands o = operands_at(p, smem_u32(smem), smem_u32(smem));
      Ring<kTileSlots> r;
      int c = 0;
      multiply_parts<false, kTileSlots, kTile>(p, o, full, empty, acc_full, acc_empty, tmem, blocks,
                                               abort, lane, &r, &c);
    } else {
      const Operands o = operands_at(p, smem_u32(smem), smem_u32(smem) + kOperandBytes);
      const uint32_t idesc = p.idesc;
      Ring<kTileStages> r;
      for (int i = 0; i < its; ++i, r.next()) {
        const int chunk = kFloat ? i / kChain : 0;
        const bool first = kFloat ? i % kChain == 0 : i == 0;
        bool ok = true;
        if (kFloat && first)
          ok = mbar_wait(acc_empty + (chunk & 1), (chunk >> 1 & 1) ^ 1, abort, p.wait_ns);
        ok = ok && mbar_wait(full + r.s, r.round, abort, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) raise_error<false>(p, abort);
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          multiply_stage<false>(o, idesc, r.s, kTileStageBytes, tmem + (chunk & 1) * kTile, first);
          umma_commit(empty + r.s);
          if (i == its - 1 || (kFloat && i % kChain == kChain - 1))
            umma_commit(acc_full + (chunk & 1));
        }
        __syncwarp();
      }
    }
    // whatever became of the sums, no product is left when tensor memory is freed
    if (elect_one()) {
      umma_commit(drain);
      drain_wait(drain, 0);
    }
  } else {
    const int col = (warp - 2) / 4 * kTileCols;
    uint8_t *buf = smem + kTileStages * kTileStageBytes + (warp - 2) * kColumnBytes;
    const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21) + col;
    const int chunks = kFloat ? (its + kChain - 1) / kChain : its > 0;
    float acc[kTileCols];
    if (kFloat || chunks == 0) {
#pragma unroll
      for (int j = 0; j < kTileCols; ++j) acc[j] = 0.f;
    }
    bool ok = true;
    Columns cols;
    cols.next = p.pairs > 1 ? (it0 + p.pairs - 1) / p.pairs : it0;
    for (int c = 0; c < chunks; ++c) {
      if (kFloat && columns)
        add_columns<kTileWarps>(p, buf, it0 + min(its, (c + 1) * kChain), false, m0, warp - 2, lane,
                                &cols);
      ok = mbar_wait(acc_full + (c & 1), c >> 1 & 1, abort, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) raise_error<false>(p, abort);
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < kTileCols; j += 32) {
        if constexpr (kFloat) {
          float v[32];
          tmem_ld_32cols(at + (c & 1) * kTile + j, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[j + i] += v[i];
        } else {
          tmem_ld_32cols(at + j, acc + j);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + (c & 1));
    }
    if (kFloat && columns) {  // into the warp's buffer, for all blocks of the cluster
      const Oct sum = end_columns<kTileWarps>(p, buf, m0, warp - 2, lane, &cols);
      if (lane < 16) {
        float4 *to = reinterpret_cast<float4 *>(buf) + 2 * lane;
        to[0] = oct_lo(sum);
        to[1] = oct_hi(sum);
      }
    }
    if (ok) {
      // every stage has been read: the last sums came after it
      float *sums = reinterpret_cast<float *>(smem) + (32 * (warp & 3) + lane) * kSumLd + col;
#pragma unroll
      for (int j = 0; j < kTileCols; j += 4)
        *reinterpret_cast<float4 *>(sums + j) =
            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (splits > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
  if (*abort) {  // what was asked for lands before the block leaves
    if (threadIdx.x == 0) {
      if (kFloat && p.pairs > 1)
        drain_stages<kTileSlots>(full, *asked_of);
      else
        drain_stages<kTileStages>(full, *asked_of);
    }
    __syncwarp();
  } else {
    const int share = kTile / splits, r0 = rank * share;
    if (columns && static_cast<int>(threadIdx.x) < share) {
      const int c = r0 + threadIdx.x;
      const float *mine =
          reinterpret_cast<const float *>(smem + kTileStages * kTileStageBytes) + c;
      float sum = 0.f;
      for (int b = 0; b < splits; ++b) {
        const uint32_t from = splits > 1 ? mapa_rank(mine, b) : smem_u32(mine);
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) sum += ld_cluster_f32(from + w * kColumnBytes);
      }
      if (m0 + c < p.m) p.cols.part[slice * p.m + m0 + c] = sum;
    }
    const int col = n0 + 4 * lane;
    const bool in = col < p.n;
    Out *out = static_cast<Out *>(p.e.out) + slice * p.m * p.n;
    Out *keep = static_cast<Out *>(p.e.keep);
    const Out *aux = static_cast<const Out *>(p.e.aux);
    Quad bias = {{0, 0}};
    if (p.e.bias && in) bias = load_quad(p.e.bias + col);
    constexpr int W = kTileThreads / 32, U = 4;
    by_kind(p.kind, [&](auto kind) {
      for (int r = warp; r < share; r += W * U) {
        Quad a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long row = m0 + r0 + r + u * W;
          a[u] = {{0, 0}};
          if (aux && in && r + u * W < share && row < p.m) a[u] = load_quad(aux + row * p.n + col);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int rr = r0 + r + u * W;
          const long long row = m0 + rr;
          if (r + u * W >= share || row >= p.m) continue;
          const float *mine = reinterpret_cast<const float *>(smem) + rr * kSumLd + 4 * lane;
          Quad sum;
          if (splits == 1) {
            sum = load_quad(mine);
          } else {
            // all in flight, added up in order
            float4 f[kMaxSplits];
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
              if (s < splits) f[s] = ld_cluster_f4(mapa_rank(mine, s));
            sum = {{pk2(f[0].x, f[0].y), pk2(f[0].z, f[0].w)}};
#pragma unroll
            for (int s = 1; s < kMaxSplits; ++s) {
              if (s >= splits) break;
              sum.v[0] = add2(sum.v[0], pk2(f[s].x, f[s].y));
              sum.v[1] = add2(sum.v[1], pk2(f[s].z, f[s].w));
            }
          }
          if (!in) continue;
          Quad z = {{0, 0}}, o;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            o.v[j] =
                finish2<decltype(kind)::value, kFloat>(sum.v[j], bias.v[j], a[u].v[j], &z.v[j]);
          store_quad(out + row * p.n + col, o);
          if (keep) store_quad(keep + row * p.n + col, z);
        }
      }
    });
  }
  if (splits > 1) cluster_sync();  // the others read this block's sums until here
}

// ------------------------------------------------------------------ large tiles
// Two blocks on paired SMs share a 256 x 256 tile: each stages 128 rows of either
// operand and holds 128 rows of sums, so that a stage brings 32 KB into an SM for 512
// clocks of its tensor core (a tile of one SM's own would bring 48 KB for 128 x 256).
// Persistent: a pair takes every (grid / 2)-th tile, and while sixteen warps of either
// block finish a tile from one half of tensor memory, the next one's products go to
// the other half. (Eight warps, two to a scheduler, did not hide each other's waits:
// for 16384 x 512 -> 2048 38 us instead of 32.)
constexpr int kPairTile = 256;
constexpr int kPairStages = 5;
constexpr int kPairSlots = 2 * kPairStages;  // of one operand
constexpr int kPairThreads = 576;
constexpr int kPairStageBytes = 2 * kOperandBytes;
constexpr int kPairWarps = 16;  // that finish tiles, 64 columns each
constexpr int kWarpCols = 4 * kPairTile / kPairWarps;
constexpr int kChunk = 32;                 // columns that a warp finishes at a time
constexpr int kChunkBytes = 32 * 64;       // of 16-bit numbers
constexpr int kStaging = 2 * kChunkBytes;  // a warp's
constexpr int kPairHead = 3 * 1024;        // rows of the bias, and barriers
constexpr size_t kPairSmem = kPairHead + kPairStages * kPairStageBytes + kPairWarps * kStaging;
static_assert(kPairSmem <= 227 * 1024, "shared memory of a block");
static_assert(kPairWarps * kChunk * 4 + (2 * kPairSlots + 5 + 2 * kPairWarps) * 8 + 24 <= kPairHead,
              "the head's parts");
static_assert(kStaging == kColumnBytes, "columns go through a warp's staging buffer");

// A slice's blocks of 64 reduction indexes.
struct Range {
  int block0, blocks;
};
__device__ __forceinline__ Range range_of(const Params &p, int slice) {
  const int all = p.pairs > 1 ? p.its / p.pairs : p.its;
  if (p.slices == 1) return {0, all};
  const int block0 = static_cast<int>(static_cast<long long>(all) * slice / p.slices);
  return {block0, static_cast<int>(static_cast<long long>(all) * (slice + 1) / p.slices) - block0};
}

// The place of tile t in the result: bands of 8 rows of tiles, column by column, so
// that the tiles under way at a time form a block as wide as it is high, whose
// operands L2 holds.
struct Place {
  int m, n;
};
__device__ __forceinline__ Place place_of(const Params &p, int t) {
  constexpr int kBand = 8;
  const int band = t / (kBand * p.n_tiles), rest = t - band * kBand * p.n_tiles;
  const int rows = min(kBand, p.m_tiles - band * kBand);
  return {(band * kBand + rest % rows) * kPairTile, rest / rows * kPairTile};
}

// 16-byte piece `c` of row `r` in a buffer of 64-byte rows with TMA's 64-byte swizzle:
// eight threads' pieces of eight rows lie in different banks.
__device__ __forceinline__ uint4 *piece64(uint8_t *buf, int r, int c) {
  return reinterpret_cast<uint4 *>(buf + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
}
// The same for rows of 128 bytes.
__device__ __forceinline__ uint4 *piece128(uint8_t *buf, int r, int c) {
  return reinterpret_cast<uint4 *>(buf + r * 128 + ((c ^ (r & 7)) << 4));
}

// A warp's 32 rows x 32 columns of floats at (row, col), a row a thread: the sums go
// through shared memory (`buf`, 4 KB), then a lane finishes four columns of every
// fourth row, as global memory is read and written.
__device__ __forceinline__ void finish_floats(const Params &p, uint8_t *buf, int lane, int slice,
                                              const float *sum, long long row, int col) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *piece128(buf, lane, e) =
        make_uint4(__float_as_uint(sum[4 * e]), __float_as_uint(sum[4 * e + 1]),
                   __float_as_uint(sum[4 * e + 2]), __float_as_uint(sum[4 * e + 3]));
  __syncwarp();
  const int ch = col + (lane & 7) * 4;
  Quad bias = {{0, 0}};
  if (p.e.bias && ch < p.n) bias = load_quad(p.e.bias + ch);
  by_kind(p.kind, [&](auto kind) {
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (row + r >= p.m || ch >= p.n) continue;
      const size_t at = static_cast<size_t>(row + r) * p.n + ch;
      const Quad v = load_quad(reinterpret_cast<const float *>(piece128(buf, r, lane & 7)));
      Quad a = {{0, 0}}, z = {{0, 0}}, y;
      if (p.e.aux) a = load_quad(static_cast<const float *>(p.e.aux) + at);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        y.v[j] = finish2<decltype(kind)::value, true>(v.v[j], bias.v[j], a.v[j], &z.v[j]);
      store_quad(static_cast<float *>(p.e.out) + slice * p.m * p.n + at, y);
      if (p.e.keep) store_quad(static_cast<float *>(p.e.keep) + at, z);
    }
  });
  __syncwarp();
}

// 32 columns of a thread's row in 16-bit numbers: aux (read from `buf` where there is
// one) and the sums make out, in its place, and z in `zbuf` where it is kept. `bias`:
// the columns', in shared memory.
template <class T>
__device__ __forceinline__ void finish_row(const Params &p, uint8_t *buf, uint8_t *zbuf, int lane,
                                           const float *sum, const float4 *bias_row) {
  by_kind(p.kind, [&](auto kind) {
    constexpr int K = decltype(kind)::value;
    constexpr bool kSlope = K == kSiluSlope || K == kGeluSlope;
    const bool has_aux = kSlope || p.e.aux;
    const bool has_bias = !kSlope && p.e.bias, keep = !kSlope && p.e.keep;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      Oct a = {{0, 0, 0, 0}}, bias = a, o, z = a;
      if (has_bias) bias = oct_of(bias_row[2 * c], bias_row[2 * c + 1]);
      if (has_aux) {
        Raw<T> r;
        r.v[0] = *piece64(buf, lane, c);
        a = oct_of(r);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.v[j] = finish2<K, false>(pk2(sum[8 * c + 2 * j], sum[8 * c + 2 * j + 1]), bias.v[j],
                                   a.v[j], &z.v[j]);
      *piece64(buf, lane, c) = raw_of<T>(o).v[0];
      if (keep) *piece64(zbuf, lane, c) = raw_of<T>(z).v[0];
    }
  });
}

template <class Out>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_pair(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
              const __grid_constant__ CUtensorMap to, const __grid_constant__ CUtensorMap tz,
              const __grid_constant__ CUtensorMap tx, const __grid_constant__ Params p) {
  constexpr bool kFloat = sizeof(Out) == 4;
  // (no room is left to align within: should the base not be, nothing is done)
  extern __shared__ __align__(1024) uint8_t smem_aligned[];
  if (smem_u32(smem_aligned) & 1023) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, static_cast<int>(VAE_EUNSUPPORTED));
    return;
  }
  float *bias_rows = reinterpret_cast<float *>(smem_aligned);
  uint8_t *smem = smem_aligned + kPairHead;
  uint8_t *staging = smem + kPairStages * kPairStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(bias_rows + kPairWarps * kChunk);
  uint64_t *empty = full + kPairSlots;
  uint64_t *acc_full = empty + kPairSlots, *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint64_t *aux_full = drain + 1;  // two of each finishing warp's
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(aux_full + 2 * kPairWarps);
  volatile uint32_t *abort = tmem_slot + 1;
  uint64_t *asked_of = reinterpret_cast<uint64_t *>(tmem_slot + 2);  // the leader's, of both
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int per = p.m_tiles * p.n_tiles, tiles = per * p.slices, stride = gridDim.x / 2;
  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int i = 0; i < kPairSlots; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 2 * kPairWarps + !!(p.inject & VAE_INJECT_WITHHOLD_ACCUMULATOR));
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * kPairWarps; ++i) mbar_init(aux_full + i, 1);
    fence_mbarrier_init();
    *abort = 0;
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.wait) grid_wait();

  if (warp == 0) {
    Ring<kPairStages> r;
    Ring<kPairSlots> slots;
    const int withheld =
        !!(p.inject & (rank == 0 ? VAE_INJECT_WITHHOLD_COPY : VAE_INJECT_WITHHOLD_PAIR_COPY));
    uint64_t asked = 0;
    bool ok = true;
    if (kFloat && p.pairs > 1) {
      for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
        const Place at = place_of(p, t % per);
        const Range its = range_of(p, t / per);
        ok = copy_parts<true>(p, &ta, &tb, smem, full, empty, its.block0, its.blocks, withheld,
                              at.m + 128 * rank, at.n + 128 * rank, rank == 0, abort, lane, &slots,
                              &asked,
                              [](uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1,
                                 int c2) {
                                tma_load_3d_pair(dst, m, mapa_rank(bar, 0), c0, c1, c2);
                              });
      }
    } else {
      for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
        const Place at = place_of(p, t % per);
        const Range its = range_of(p, t / per);
        const int m0 = at.m + 128 * rank, n0 = at.n + 128 * rank;
        const int end = its.block0 + its.blocks - withheld;
        for (int it = its.block0; it < end; ++it, ++asked, r.next()) {
          ok = mbar_wait(empty + r.s, r.round ^ 1, abort, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (lane == 0) raise_error<true>(p, abort);
            break;
          }
          const uint32_t bar = mapa_rank(full + r.s, 0);
          uint8_t *a = smem + r.s * kPairStageBytes;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full + r.s, 2 * kPairStageBytes);
            auto load = [&](uint8_t *dst, const CUtensorMap *m, int c0, int c1, int c2) {
              tma_load_3d_pair(dst, m, bar, c0, c1, c2);
            };
            load_operand(&ta, p.a_k, it * kBK, m0, 0, a, load);
            load_operand(&tb, p.b_k, it * kBK, n0, 0, a + kOperandBytes, load);
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) st_cluster(mapa_rank(asked_of + rank, 0), asked);
  } else if (warp == 1) {
    // The whole warp goes through the loop, so that descriptors stay in registers that
    // all lanes share, and one lane issues: the tensor core takes a stage 512 clocks,
    // and this loop has to be shorter.
    if (rank == 0) {
      const Operands o = operands_at(p, smem_u32(smem), smem_u32(smem) + kOperandBytes);
      const uint32_t idesc = p.idesc;
      Ring<kPairStages> r;
      int c = 0;  // accumulators taken
      bool ok = true;
      if (kFloat && p.pairs > 1) {
        const Operands same = operands_at(p, smem_u32(smem), smem_u32(smem));
        Ring<kPairSlots> slots;
        for (int t = blockIdx.x / 2; t < tiles && ok; t += stride)
          ok = multiply_parts<true, kPairSlots, kPairTile>(
              p, same, full, empty, acc_full, acc_empty, tmem, range_of(p, t / per).blocks, abort,
              lane, &slots, &c);
        ok = false;  // (the tiles are done)
      }
      for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
        const int its = range_of(p, t / per).blocks;
        for (int it = 0; it < its; ++it, r.next()) {
          const bool first = kFloat ? it % kChain == 0 : it == 0;
          const bool last = it == its - 1 || (kFloat && it % kChain == kChain - 1);
          if (first)
            ok = mbar_wait(acc_empty + (c & 1), (c >> 1 & 1) ^ 1, abort, p.wait_ns);
          ok = ok && mbar_wait(full + r.s, r.round, abort, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (lane == 0) raise_error<true>(p, abort);
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            multiply_stage<true>(o, idesc, r.s, kPairStageBytes, tmem + (c & 1) * kPairTile, first);
            umma_commit_pair(empty + r.s, 3);
            if (last) umma_commit_pair(acc_full + (c & 1), 3);
          }
          __syncwarp();
          c += last;
        }
      }
      // (elect_one names the same lane every time: it has issued all of the products)
      if (elect_one()) {
        umma_commit_pair(drain, 1);
        drain_wait(drain, 0);
      }
    }
  } else {
    const int q = warp & 3, first_col = (warp - 2) / 4 * kWarpCols;
    const uint32_t at = tmem + (static_cast<uint32_t>(q) << 21) + first_col;
    int c = 0;  // accumulators taken
    auto taken = [&](int b) -> bool {
      bool ok = mbar_wait(acc_full + (b & 1), b >> 1 & 1, abort, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) raise_error<true>(p, abort);
      tc_fence_after();
      return ok;
    };
    auto give_back = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_rank(acc_empty + (b & 1), 0));
    };
    uint8_t *buf = staging + (warp - 2) * kStaging;
    // 16-bit results: chunk g of the warp's (two a tile) uses buffer g % 2 for aux and
    // out, or the first one where the second is z's. aux is asked for a chunk ahead,
    // over the tiles' ends, where it has a buffer to go to.
    uint64_t *aux = aux_full + 2 * (warp - 2);
    const int other = p.e.keep ? 0 : 1;
    int g = 0, asked = 0;
    auto ask = [&](int k) {
      const int t = blockIdx.x / 2 + (k >> 1) * stride;
      if (t >= tiles) return;
      uint64_t *bar = aux + (k & other);
      mbar_arrive_expect_tx(bar, kChunkBytes);
      const Place at = place_of(p, t);
      tma_load_2d(buf + (k & other) * kChunkBytes, &tx, bar, at.n + first_col + (k & 1) * kChunk,
                  at.m + 128 * static_cast<int>(rank) + 32 * q);
      asked = k + 1;
    };
    float *bias_row = bias_rows + kChunk * (warp - 2);
    auto bias_at = [&](int col) -> float {
      return p.e.bias && col + lane < p.n ? __ldg(p.e.bias + col + lane) : 0.f;
    };
    if (!kFloat && p.e.aux && !p.e.keep && lane == 0) ask(0);
    bool ok = true;
    for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
      const Place place = place_of(p, t % per);
      const long long row = place.m + 128ll * rank + 32 * q;
      const int col = place.n + first_col;
      if constexpr (kFloat) {
        float acc[kWarpCols];
#pragma unroll
        for (int j = 0; j < kWarpCols; ++j) acc[j] = 0.f;
        const int slice = t / per;
        const Range its = range_of(p, slice);
        const int chunks = (its.blocks * p.pairs + kChain - 1) / kChain;
        const int it0 = its.block0 * p.pairs, it1 = it0 + its.blocks * p.pairs;
        const long long first_row = place.m + 128ll * rank;
        Columns cols;
        const int tile_col = place.n / kPairTile;
        cols.next = its.block0 + (tile_col + p.n_tiles - its.block0 % p.n_tiles) % p.n_tiles;
        for (int k = 0; k < chunks && ok; ++k, ++c) {
          add_columns<kPairWarps>(p, buf, min(it1, it0 + (k + 1) * kChain), false, first_row,
                                  warp - 2, lane, &cols);
          ok = taken(c);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < kWarpCols; j += 16) {
            float v[16];
            tmem_ld_16cols(at + (c & 1) * kPairTile + j, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j + e] += v[e];
          }
          give_back(c);
        }
        if (!ok) break;
        if (p.cols.part) {
          const Oct sum = end_columns<kPairWarps>(p, buf, first_row, warp - 2, lane, &cols);
          const long long ch = first_row + 8 * lane;
          const long long part =
              (static_cast<long long>(slice) * p.n_tiles + tile_col) * kPairWarps + warp - 2;
          if (lane < 16 && ch < p.m)
            store_raw<float, false>(p.cols.part + part * p.m + ch, 8, raw_of<float>(sum));
        }
#pragma unroll
        for (int j = 0; j < kWarpCols; j += kChunk)
          finish_floats(p, buf, lane, slice, acc + j, row, col + j);
      } else {
        // a chunk's bias is asked for a chunk ahead: from L2 it takes longer than the rest
        float bias = bias_at(col);
        ok = taken(c);
        if (!ok) break;
#pragma unroll 1
        for (int j = 0; j < 2; ++j, ++g) {
          uint8_t *mine = buf + (g & other) * kChunkBytes, *zbuf = buf + kChunkBytes;
          float v[kChunk];
          tmem_ld_32cols(at + (c & 1) * kPairTile + j * kChunk, v);
          if (j == 1) give_back(c);
          if (lane == 0) {
            if (p.e.aux || p.e.keep) {
              bulk_wait_read<0>();  // what was stored has left its buffer
              if (p.e.aux) ask(p.e.keep ? g : g + 1);
            } else {
              bulk_wait_read<1>();
            }
          }
          if (p.e.bias) {
            bias_row[lane] = bias;
            bias = bias_at(j == 0 ? col + kChunk : p.n);
          }
          __syncwarp();
          if (p.e.aux) {
            ok = mbar_wait(aux + (g & other), (p.e.keep ? g : g >> 1) & 1, abort, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
              if (lane == 0) raise_error<true>(p, abort);
              break;
            }
          }
          finish_row<Out>(p, mine, zbuf, lane, v, reinterpret_cast<const float4 *>(bias_row));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row < p.m && col + j * kChunk < p.n) {
              tma_store_2d(&to, mine, col + j * kChunk, static_cast<int>(row));
              if (p.e.keep) tma_store_2d(&tz, zbuf, col + j * kChunk, static_cast<int>(row));
            }
            bulk_commit();
          }
        }
        ++c;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!kFloat && lane == 0) {
      if (p.e.aux && *abort)  // what was asked for lands before the block leaves
        for (int k = g; k < asked; ++k)
          drain_wait(aux + (k & other), (other ? k >> 1 : k) & 1);
      bulk_wait_all();
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither block leaves while the pair's products, copies or arrivals touch it
  if (*abort) {    // (in both, raise_error's) what either asked for lands first
    if (rank == 0 && threadIdx.x == 0) {
      if (kFloat && p.pairs > 1)
        drain_pair<kPairSlots>(full, asked_of, kOperandBytes);
      else
        drain_pair<kPairStages>(full, asked_of, kPairStageBytes);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ host
// A map of `parts` matrices [rows][cols] of 16-bit numbers, in boxes of 64 by box_rows.
int encode_operand(CUtensorMap *map, const void *p, int parts, long long rows, long long cols,
                   int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                            static_cast<uint64_t>(parts)};
  const uint64_t row = static_cast<uint64_t>(cols) * 2;
  const uint64_t strides[2] = {row, parts > 1 ? row * static_cast<uint64_t>(rows) : row};
  const uint32_t box[3] = {64, static_cast<uint32_t>(box_rows), 1};
  return encode_tiled(map, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}
// A map of a result [rows][cols] of 16-bit numbers in boxes of 32 by 32.
int encode_result(CUtensorMap *map, const void *p, long long rows, long long cols) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t stride = static_cast<uint64_t>(cols) * 2;
  const uint32_t box[2] = {kChunk, 32};
  return encode_tiled(map, p, 2, dims, &stride, box, CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

// Kernels' dynamic shared memory is allowed once a device.
template <class K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> *done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done->load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done->fetch_or(1ull << dev);
  return e;
}

cudaLaunchConfig_t launch_config(cudaLaunchAttribute *attr, unsigned grid, int threads, size_t smem,
                                 int cluster, bool after, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cfg;
}

// Clusters of `splits` blocks that run at a time (76, 36 and 15 of 2, 4 and 8 on a
// GB300, whose SMs are not grouped in multiples of eight), asked once a device.
int clusters_at_once(int splits) {
  static std::atomic<int> known[64][kMaxSplits + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return std::max(1, num_sms() / splits);
  }
  int n = known[dev][splits].load(std::memory_order_relaxed);
  if (n) return n;
  static std::atomic<uint64_t> done{0};
  cudaLaunchAttribute attr[2];
  const auto cfg = launch_config(attr, splits, kTileThreads, kTileSmem, splits, false, nullptr);
  if (splits == 1 || allow_smem(gemm_tile<float>, kTileSmem, &done) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, gemm_tile<float>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = std::max(1, num_sms() / splits);
  }
  known[dev][splits].store(n, std::memory_order_relaxed);
  return n;
}

// Clocks of a stage, measured: small tiles are bound by shared memory, which takes in
// every operand for 128 rows and columns alone; floats' parts are copied once for six.
int small_stage(bool parts) { return parts ? 400 : 700; }
int pair_stage(bool parts) { return parts ? 520 : 600; }
// How many blocks share a 128 x 128 tile's reduction, and the clocks it takes: rounds of
// clusters times what a block does besides and its stages.
struct Tiling {
  int splits;
  long long clocks;
};
Tiling small_tiling(long long tiles, long long its, long long blocks) {
  Tiling best{1, 0};
  for (int s = 1; s <= kMaxSplits; s *= 2) {
    if (s > 1 && (its < 2 * s || blocks < s)) break;
    const long long at_once = clusters_at_once(s);
    const long long stages = (its + s - 1) / s, rounds = (tiles + at_once - 1) / at_once;
    const long long t = rounds * (4000 + 300 * s + small_stage(its > blocks) * stages);
    if (s == 1 || t < best.clocks) best = {s, t};
  }
  return best;
}

int launch_pair(const GemmDesc &d, Params p, cudaStream_t s) {
  CUtensorMap ta, tb;
  VAE_TRY(d.a.k_major ? encode_operand(&ta, d.a.p, d.parts, d.m, d.k, 128)
                      : encode_operand(&ta, d.a.p, d.parts, d.k, d.m, kBK));
  VAE_TRY(d.b.k_major ? encode_operand(&tb, d.b.p, d.parts, d.n, d.k, 128)
                      : encode_operand(&tb, d.b.p, d.parts, d.k, d.n, kBK));
  CUtensorMap to{}, tz{}, tx{};  // 32 x 32 pieces of 16-bit results
  if (d.dtype != VAE_F32) {
    VAE_TRY(encode_result(&to, p.e.out, d.m, d.n));
    if (p.e.keep) VAE_TRY(encode_result(&tz, p.e.keep, d.m, d.n));
    if (p.e.aux) VAE_TRY(encode_result(&tx, p.e.aux, d.m, d.n));
  }
  p.idesc = idesc_16bit(kPairTile, kPairTile, !d.f16, !d.a.k_major, !d.b.k_major);
  p.m_tiles = ceil_div(d.m, kPairTile);
  p.n_tiles = ceil_div(d.n, kPairTile);
  p.cols.step = p.n_tiles;
  const unsigned grid = 2 * std::min(p.m_tiles * p.n_tiles * p.slices, num_sms() / 2);
  return by_dtype(d.dtype, [&](auto o) -> int {
    using Out = decltype(o);
    static std::atomic<uint64_t> done{0};
    VAE_CUDA_TRY(allow_smem(gemm_pair<Out>, kPairSmem, &done));
    cudaLaunchAttribute attr[2];
    const auto cfg = launch_config(attr, grid, kPairThreads, kPairSmem, 2, p.wait, s);
    VAE_CUDA_TRY(cudaLaunchKernelEx(&cfg, gemm_pair<Out>, ta, tb, to, tz, tx, p));
    count_launches(1);
    return VAE_OK;
  });
}

// Rows that a copy of a K-major operand for a small tile takes in: a lone tile's own, in
// sixteens (the others of its 128 are whatever lies in shared memory, and make results
// outside the matrix). With 128, 116 of them zeros, 12 rows 4096 -> 4096 took 14.0 us
// instead of 9.3.
int copied_rows(const GemmDesc &d, const GemmOperand &o, long long rows) {
  if (!o.k_major || d.parts > 1 || rows >= kTile) return kTile;
  return static_cast<int>((rows + 15) / 16 * 16);
}

int launch_tile(const GemmDesc &d, Params p, cudaStream_t s) {
  CUtensorMap ta, tb;
  const int rows_a = copied_rows(d, d.a, d.m), rows_b = copied_rows(d, d.b, d.n);
  VAE_TRY(d.a.k_major ? encode_operand(&ta, d.a.p, d.parts, d.m, d.k, rows_a)
                      : encode_operand(&ta, d.a.p, d.parts, d.k, d.m, kBK));
  VAE_TRY(d.b.k_major ? encode_operand(&tb, d.b.p, d.parts, d.n, d.k, rows_b)
                      : encode_operand(&tb, d.b.p, d.parts, d.k, d.n, kBK));
  p.stage_bytes = static_cast<uint32_t>(rows_a + rows_b) * kBK * 2;
  p.idesc = idesc_16bit(kTile, kTile, !d.f16, !d.a.k_major, !d.b.k_major);
  p.m_tiles = ceil_div(d.m, kTile);
  p.n_tiles = ceil_div(d.n, kTile);
  p.cols.step = 1;
  const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
  const int splits = small_tiling(tiles, p.its, p.its / p.pairs).splits;
  if (tiles * splits * p.slices > 0x7fffffff) return VAE_EUNSUPPORTED;
  return by_dtype(d.dtype, [&](auto o) -> int {
    using Out = decltype(o);
    static std::atomic<uint64_t> done{0};
    VAE_CUDA_TRY(allow_smem(gemm_tile<Out>, kTileSmem, &done));
    cudaLaunchAttribute attr[2];
    const auto grid = static_cast<unsigned>(tiles * splits * p.slices);
    const auto cfg = launch_config(attr, grid, kTileThreads,
                                   kTileSmem, splits, p.wait, s);
    VAE_CUDA_TRY(cudaLaunchKernelEx(&cfg, gemm_tile<Out>, ta, tb, p, splits));
    count_launches(1);
    return VAE_OK;
  });
}

}  // namespace

// The plan that the clocks speak for: rounds of tiles times what one takes besides its
// stages, and its stages; adding up slices takes a launch and the reading of their sums.
GemmPlan gemm_plan(long long m, int n, long long k, int parts, bool sliced) {
  const long long blocks = (k + kBK - 1) / kBK, pairs = parts > 1 ? 6 : 1, its = blocks * pairs;
  const long long small = static_cast<long long>(ceil_div(m, kTile)) * ceil_div(n, kTile);
  const long long large = static_cast<long long>(ceil_div(m, kPairTile)) * ceil_div(n, kPairTile);
  auto merge = [&](long long slices) { return slices > 1 ? 6000 + slices * m * n / 600 : 0; };
  GemmPlan best;
  const Tiling t = small_tiling(small, its, blocks);
  long long clocks = t.clocks;
  const long long idle = clusters_at_once(t.splits) / small;  // (whole clusters)
  if (sliced && idle > 1) {
    const long long s = std::min(idle, blocks * pairs / (8 * t.splits));
    const long long c = 4000 + 300 * t.splits +
                        small_stage(parts > 1) * its / (t.splits * std::max(1ll, s)) + merge(s);
    if (s > 1 && c < clocks) {
      best.slices = best.columns = static_cast<int>(s);
      clocks = c;
    }
  }
  const long long units = num_sms() / 2;
  if (!units || large > 0x0fffffff) return best;
  for (long long s = 1; s == 1 || (sliced && s <= units / large && s * 16 <= its); ++s) {
    const long long c =
        5000 + merge(s) +
        (large * s + units - 1) / units * (1000 + pair_stage(parts > 1) * ((its + s - 1) / s));
    if (c >= clocks) continue;
    best.pairs = true;
    best.slices = static_cast<int>(s);
    best.columns = static_cast<int>(s) * ceil_div(n, kPairTile) * kPairWarps;
    clocks = c;
  }
  return best;
}

int gemm(const GemmDesc &d, cudaStream_t s) {
  Params p{};
  p.m = d.m;
  p.n = d.n;
  p.pairs = d.parts > 1 ? 6 : 1;
  const long long its = (d.k + kBK - 1) / kBK * p.pairs;
  if (its > 0x7fffffff || d.m > 0x7fffffff - kPairTile) return VAE_EUNSUPPORTED;
  p.its = static_cast<int>(its);
  p.a_k = d.a.k_major;
  p.b_k = d.b.k_major;
  p.wait = d.wait;
  p.wait_ns = wait_limit_ns();
  p.err = device_error_word();
  p.inject = injected_faults();
  if (!p.err) return VAE_ECUDA;
  p.e = d.epi;
  p.kind = kind_of(d.epi);
  p.cols = d.cols;
  p.slices = d.plan.slices;
  return d.plan.pairs ? launch_pair(d, p, s) : launch_tile(d, p, s);
}

}  // namespace vae
