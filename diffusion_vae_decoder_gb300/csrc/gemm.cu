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

#include "gn_train.cuh"
#include "linear.cuh"
#include "ptx.cuh"
#include "tokens.cuh"

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
  bool a_k, b_k;
  bool wait;
  uint32_t idesc;
  uint64_t wait_ns;
  int *err;
  GemmEpilogue e;
};

__device__ __forceinline__ void raise_error(const Params &p, volatile uint32_t *abort) {
  *abort = 1u;
  atomicCAS(p.err, 0, static_cast<int>(VAE_EDEVICE_TIMEOUT));
}
// Used only while draining after an abort.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > limit_ns) return;
}

// The parts that product q takes: hh, hm, mh, mm, hl, lh.
__device__ __forceinline__ int part_a(int q) { return (0x201100 >> (4 * q)) & 15; }
__device__ __forceinline__ int part_b(int q) { return (0x021010 >> (4 * q)) & 15; }

// v of act(z) = z sigmoid(v), and dv / dz.
__device__ __forceinline__ uint64_t gate2(uint64_t z, int act, uint64_t *slope) {
  if (act == VAE_ACT_SILU) {
    *slope = pk2(1.f, 1.f);
    return z;
  }
  // gelu: sqrt(8 / pi) (z + 0.044715 z^3)
  const float a = 1.5957691216057308f, b = 0.044715f;
  const uint64_t q = mul2(z, z);
  *slope = fma2(q, pk2(3.f * a * b, 3.f * a * b), pk2(a, a));
  return mul2(z, fma2(q, pk2(a * b, a * b), pk2(a, a)));
}
template <bool PRECISE>
__device__ __forceinline__ uint64_t act2(uint64_t z, int act) {
  if (act == VAE_ACT_NONE) return z;
  uint64_t slope;
  const uint64_t v = gate2(z, act, &slope);
  return mul2(z, PRECISE ? sigmoid2_precise(v) : sigmoid2(v));
}
// act'(z) = s + z slope s (1 - s). Beyond +-32 the derivative is 1 or 0 to far below
// float's resolution, and the products there would overflow: z is held there
// (comparisons that leave a NaN).
__device__ __forceinline__ float held(float z) { return z > 32.f ? 32.f : z < -32.f ? -32.f : z; }
template <bool PRECISE>
__device__ __forceinline__ uint64_t act_slope2(uint64_t z, int act) {
  z = pk2(held(lo2(z)), held(hi2(z)));
  uint64_t slope;
  const uint64_t v = gate2(z, act, &slope);
  const uint64_t s = PRECISE ? sigmoid2_precise(v) : sigmoid2(v);
  const uint64_t rest = fma2(s, pk2(-1.f, -1.f), pk2(1.f, 1.f));
  return fma2(mul2(mul2(z, slope), s), rest, s);
}

// Two neighbouring sums of a row -> out, and z where it is kept.
template <bool PRECISE>
__device__ __forceinline__ uint64_t finish2(const GemmEpilogue &e, uint64_t sum, uint64_t bias,
                                            uint64_t aux, uint64_t *z) {
  if (e.derivative) return e.aux ? mul2(sum, act_slope2<PRECISE>(aux, e.act)) : sum;
  *z = add2(sum, bias);
  return add2(act2<PRECISE>(*z, e.act), aux);
}

// Stage `it` of the tile at (m0, n0): `rows_a` and `rows_b` rows of the operands.
// `load(dst, map, c0, c1, c2)` issues one copy.
template <int ROWS_A, int ROWS_B, class L>
__device__ __forceinline__ void load_stage(const CUtensorMap *ta, const CUtensorMap *tb,
                                           const Params &p, int it, int m0, int n0, uint8_t *da,
                                           uint8_t *db, L &&load) {
  int k0 = it * kBK, pa = 0, pb = 0;
  if (p.pairs > 1) {
    const int q = it % p.pairs;
    k0 = it / p.pairs * kBK;
    pa = part_a(q);
    pb = part_b(q);
  }
  if (p.a_k) {
    load(da, ta, k0, m0, pa);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS_A / 64; ++i) load(da + i * kBK * 128, ta, m0 + 64 * i, k0, pa);
  }
  if (p.b_k) {
    load(db, tb, k0, n0, pb);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS_B / 64; ++i) load(db + i * kBK * 128, tb, n0 + 64 * i, k0, pb);
  }
}
// The four steps of a staged pair of operands.
template <bool PAIR>
__device__ __forceinline__ void multiply_stage(const Params &p, uint32_t sa, uint32_t sb,
                                               uint32_t acc, bool first) {
  const uint64_t da = p.a_k ? sw128_kmajor_desc(sa) : sw128_mnmajor_desc(sa, kBK * 128);
  const uint64_t db = p.b_k ? sw128_kmajor_desc(sb) : sw128_mnmajor_desc(sb, kBK * 128);
  const uint32_t step_a = (p.a_k ? 32 : 2048) >> 4, step_b = (p.b_k ? 32 : 2048) >> 4;
#pragma unroll
  for (int k = 0; k < kBK / 16; ++k)
    umma_16bit<PAIR>(acc, da + k * step_a, db + k * step_b, p.idesc, !(first && k == 0));
}

// ------------------------------------------------------------------ small tiles
// A 128 x 128 tile by a cluster of blocks that split the reduction: each adds up its
// share of the stages, puts its sums into shared memory, and finishes 128 / S rows of
// the tile from all of them, in the order of the blocks. Warp 0 copies, warp 1
// multiplies, warps 2 to 5 take the sums out.
constexpr int kTile = 128;
constexpr int kTileStages = 6;
constexpr int kTileThreads = 192;
constexpr int kTileStageBytes = 2 * kTile * kBK * 2;
constexpr int kSumLd = kTile + 4;  // floats of a row of sums: 16 bytes shift the banks
constexpr size_t kTileSmem = kTileStages * kTileStageBytes + 1024 + 256;
static_assert(kTile * kSumLd * 4 <= kTileStages * kTileStageBytes, "sums lie over the stages");

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Four numbers of type T, as two pairs.
struct Quad {
  uint64_t v[2];
};
template <class T>
__device__ __forceinline__ Quad load_quad(const T *p) {
  if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    return {{pk2(f.x, f.y), pk2(f.z, f.w)}};
  } else {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return {{unpack2(u.x, T{}), unpack2(u.y, T{})}};
  }
}
template <class T>
__device__ __forceinline__ void store_quad(T *p, const Quad &q) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4 *>(p) =
        make_float4(lo2(q.v[0]), hi2(q.v[0]), lo2(q.v[1]), hi2(q.v[1]));
  else
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(pack2(lo2(q.v[0]), hi2(q.v[0]), T{}), pack2(lo2(q.v[1]), hi2(q.v[1]), T{}));
}

template <class Out>
__global__ void __launch_bounds__(kTileThreads, 1)
    gemm_tile(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
              const Params p, int splits) {
  constexpr bool kFloat = sizeof(Out) == 4;
  constexpr uint32_t kTmem = kFloat ? 2 * kTile : kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kTileStages * kTileStageBytes);
  uint64_t *empty = full + kTileStages;
  uint64_t *acc_full = empty + kTileStages, *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / splits, rank = blockIdx.x % splits;
  const int m0 = tile / p.n_tiles * kTile, n0 = tile % p.n_tiles * kTile;
  const int it0 = static_cast<int>(static_cast<long long>(p.its) * rank / splits);
  const int its = static_cast<int>(static_cast<long long>(p.its) * (rank + 1) / splits) - it0;
  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 4);
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
    if (lane == 0) {
      int i = 0;
      for (; i < its; ++i) {
        const int s = i % kTileStages;
        if (!mbar_wait(empty + s, (i / kTileStages & 1) ^ 1, abort, p.wait_ns)) {
          raise_error(p, abort);
          break;
        }
        mbar_arrive_expect_tx(full + s, kTileStageBytes);
        uint8_t *a = smem + s * kTileStageBytes;
        load_stage<kTile, kTile>(&ta, &tb, p, it0 + i, m0, n0, a, a + kTileStageBytes / 2,
                                 [&](uint8_t *dst, const CUtensorMap *m, int c0, int c1, int c2) {
                                   tma_load_3d(dst, m, full + s, c0, c1, c2);
                                 });
      }
      if (*abort)  // what was asked for lands before the block leaves
        for (int j = max(0, i - kTileStages); j < i; ++j)
          drain_wait(full + j % kTileStages, j / kTileStages & 1, p.wait_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < its && ok; ++i) {
        const int chunk = kFloat ? i / kChain : 0, s = i % kTileStages;
        const bool first = kFloat ? i % kChain == 0 : i == 0;
        if (kFloat && first)
          ok = mbar_wait(acc_empty + (chunk & 1), (chunk >> 1 & 1) ^ 1, abort, p.wait_ns);
        ok = ok && mbar_wait(full + s, i / kTileStages & 1, abort, p.wait_ns);
        if (!ok) {
          raise_error(p, abort);
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + s * kTileStageBytes);
        multiply_stage<false>(p, sa, sa + kTileStageBytes / 2, tmem + (chunk & 1) * kTile, first);
        umma_commit(empty + s);
        if (i == its - 1 || (kFloat && i % kChain == kChain - 1)) umma_commit(acc_full + (chunk & 1));
      }
      // whatever became of the sums, no product is left when tensor memory is freed
      umma_commit(drain);
      drain_wait(drain, 0, p.wait_ns);
    }
  } else {
    const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const int chunks = kFloat ? (its + kChain - 1) / kChain : its > 0;
    float acc[kTile];
    if (kFloat || chunks == 0) {
#pragma unroll
      for (int j = 0; j < kTile; ++j) acc[j] = 0.f;
    }
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      ok = mbar_wait(acc_full + (c & 1), c >> 1 & 1, abort, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) raise_error(p, abort);
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < kTile; j += 32) {
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
    if (ok) {
      // every stage has been read: the last sums came after it
      float *sums = reinterpret_cast<float *>(smem) + (32 * (warp & 3) + lane) * kSumLd;
#pragma unroll
      for (int j = 0; j < kTile; j += 4)
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
  if (!*abort) {
    const int share = kTile / splits, r0 = rank * share;
    const int col = n0 + 4 * lane;
    const bool in = col < p.n;
    Out *out = static_cast<Out *>(p.e.out), *keep = static_cast<Out *>(p.e.keep);
    const Out *aux = static_cast<const Out *>(p.e.aux);
    Quad bias = {{0, 0}};
    if (p.e.bias && in) bias = load_quad(p.e.bias + col);
    constexpr int W = kTileThreads / 32, U = 4;
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
          sum = {{0, 0}};
          for (int s = 0; s < splits; ++s) {
            const float4 f = ld_cluster_f4(mapa_rank(mine, s));
            sum.v[0] = add2(sum.v[0], pk2(f.x, f.y));
            sum.v[1] = add2(sum.v[1], pk2(f.z, f.w));
          }
        }
        if (!in) continue;
        Quad z = {{0, 0}}, o;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          o.v[j] = finish2<kFloat>(p.e, sum.v[j], bias.v[j], a[u].v[j], &z.v[j]);
        store_quad(out + row * p.n + col, o);
        if (keep) store_quad(keep + row * p.n + col, z);
      }
    }
  }
  if (splits > 1) cluster_sync();  // the others read this block's sums until here
}

// ------------------------------------------------------------------ large tiles
// Two blocks on paired SMs share a 256 x 256 tile: each stages 128 rows of either
// operand and holds 128 rows of sums, so that a stage brings 32 KB into an SM for 512
// clocks of its tensor core (a tile of one SM's own would bring 48 KB for 128 x 256).
// Persistent: a pair takes every (grid / 2)-th tile, and while eight warps of either
// block finish a tile from one half of tensor memory, the next one's products go to
// the other half.
constexpr int kPairTile = 256;
constexpr int kPairStages = 5;
constexpr int kPairThreads = 320;
constexpr int kPairStageBytes = 2 * 128 * kBK * 2;
constexpr int kPairWarps = 8;
constexpr int kStaging = 2 * 32 * 128;  // a warp's two buffers of 32 rows of 128 bytes
constexpr size_t kPairSmem =
    kPairStages * kPairStageBytes + kPairWarps * kStaging + 1024 + 256;
static_assert(kPairSmem <= 227 * 1024, "shared memory of a block");

// 16-byte piece `c` of row `r` of a staging buffer: rows shift by a piece, so that
// neither a thread's walk along its row nor a warp's along rows meets in a bank.
__device__ __forceinline__ uint4 *piece(uint8_t *buf, int r, int c) {
  return reinterpret_cast<uint4 *>(buf + r * 128 + ((c ^ (r & 7)) << 4));
}
// Numbers in 16 bytes, as pairs of floats.
template <class T>
struct Piece {
  uint64_t v[8 / sizeof(T)];
};
template <class T>
__device__ __forceinline__ Piece<T> piece_of(uint4 u) {
  if constexpr (sizeof(T) == 4)
    return {{u.x | static_cast<uint64_t>(u.y) << 32, u.z | static_cast<uint64_t>(u.w) << 32}};
  else
    return {{unpack2(u.x, T{}), unpack2(u.y, T{}), unpack2(u.z, T{}), unpack2(u.w, T{})}};
}
template <class T>
__device__ __forceinline__ uint4 bits_of(const Piece<T> &p) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(static_cast<uint32_t>(p.v[0]), static_cast<uint32_t>(p.v[0] >> 32),
                      static_cast<uint32_t>(p.v[1]), static_cast<uint32_t>(p.v[1] >> 32));
  else
    return make_uint4(pack2(lo2(p.v[0]), hi2(p.v[0]), T{}), pack2(lo2(p.v[1]), hi2(p.v[1]), T{}),
                      pack2(lo2(p.v[2]), hi2(p.v[2]), T{}), pack2(lo2(p.v[3]), hi2(p.v[3]), T{}));
}

// A warp's 32 rows x (128 / sizeof(T)) columns of sums at (row, col), a row a thread,
// finished and stored. Global memory is read and written in whole 128-byte rows.
template <class T>
struct Emitter {
  static constexpr int kCols = 128 / sizeof(T), kPer = 16 / sizeof(T);  // of a row, of a piece
  const Params &p;
  uint8_t *buf;  // kStaging bytes: out (aux before it) and z
  int lane;

  // The piece of a row-major array that this lane carries in step i; NULL outside.
  template <class P>
  __device__ __forceinline__ P *at(P *base, long long row, int col, int i) const {
    const long long r = row + 4 * i + (lane >> 3);
    const int c = col + (lane & 7) * kPer;
    return r < p.m && c < p.n ? base + r * p.n + c : nullptr;
  }
  __device__ __forceinline__ uint4 *mine(uint8_t *b, int i) const {
    return piece(b, 4 * i + (lane >> 3), lane & 7);
  }
  __device__ __forceinline__ uint4 fetch(long long row, int col, int i) const {
    const T *a = at(static_cast<const T *>(p.e.aux), row, col, i);
    return a ? *reinterpret_cast<const uint4 *>(a) : make_uint4(0, 0, 0, 0);
  }
  // 16-bit numbers: pieces c0 .. c0 + N - 1 of the thread's row, of sums v.
  template <int N>
  __device__ __forceinline__ void finish(const float *v, int col, int c0) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i;
      Piece<T> a, o, z;
      if (p.e.aux) a = piece_of<T>(*piece(buf, lane, c));
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) {
        const int ch = col + c * kPer + 2 * j;
        uint64_t bias = 0;
        if (p.e.bias && ch < p.n) bias = __ldg(reinterpret_cast<const unsigned long long *>(p.e.bias + ch));
        z.v[j] = 0;
        o.v[j] = finish2<false>(p.e, pk2(v[i * kPer + 2 * j], v[i * kPer + 2 * j + 1]),
                                         bias, p.e.aux ? a.v[j] : 0, &z.v[j]);
      }
      *piece(buf, lane, c) = bits_of<T>(o);
      if (p.e.keep) *piece(buf + kStaging / 2, lane, c) = bits_of<T>(z);
    }
  }
  // Floats whose sums lie in the buffer.
  __device__ __forceinline__ void finish_rows(long long row, int col) const {
    const int ch = col + (lane & 7) * 4;
    Quad bias = {{0, 0}};
    if (p.e.bias && ch < p.n) bias = load_quad(p.e.bias + ch);
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      float *o = at(static_cast<float *>(p.e.out), row, col, i);
      if (!o) continue;
      const size_t off = o - static_cast<float *>(p.e.out);
      const Piece<float> sum = piece_of<float>(*mine(buf, i));
      Quad a = {{0, 0}}, z = {{0, 0}}, y;
      if (p.e.aux) a = load_quad(static_cast<const float *>(p.e.aux) + off);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        y.v[j] = finish2<true>(p.e, sum.v[j], bias.v[j], a.v[j], &z.v[j]);
      store_quad(o, y);
      if (p.e.keep) store_quad(static_cast<float *>(p.e.keep) + off, z);
    }
  }
  __device__ __forceinline__ void store(void *dst, uint8_t *from, long long row, int col) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      T *d = at(static_cast<T *>(dst), row, col, i);
      if (d) *reinterpret_cast<uint4 *>(d) = *mine(from, i);
    }
  }
  __device__ __forceinline__ void flush(long long row, int col) const {
    __syncwarp();
    store(p.e.out, buf, row, col);
    if (p.e.keep) store(p.e.keep, buf + kStaging / 2, row, col);
    __syncwarp();
  }
};

template <class Out>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_pair(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
              const Params p) {
  constexpr bool kFloat = sizeof(Out) == 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *staging = smem + kPairStages * kPairStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + kPairWarps * kStaging);
  uint64_t *empty = full + kPairStages;
  uint64_t *acc_full = empty + kPairStages, *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int tiles = p.m_tiles * p.n_tiles, stride = gridDim.x / 2;
  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 2 * kPairWarps);
    }
    mbar_init(drain, 1);
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
    if (lane == 0) {
      long long i = 0;  // stages, over all tiles
      bool ok = true;
      for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
        const int m0 = t / p.n_tiles * kPairTile + 128 * rank;
        const int n0 = t % p.n_tiles * kPairTile + 128 * rank;
        for (int it = 0; it < p.its; ++it, ++i) {
          const int s = static_cast<int>(i % kPairStages);
          ok = mbar_wait_cluster(empty + s, (i / kPairStages & 1) ^ 1, abort, p.wait_ns);
          if (!ok) {
            raise_error(p, abort);
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * kPairStageBytes);
          const uint32_t bar = mapa_rank(full + s, 0);
          uint8_t *a = smem + s * kPairStageBytes;
          load_stage<128, 128>(&ta, &tb, p, it, m0, n0, a, a + kPairStageBytes / 2,
                               [&](uint8_t *dst, const CUtensorMap *m, int c0, int c1, int c2) {
                                 tma_load_3d_pair(dst, m, bar, c0, c1, c2);
                               });
        }
      }
      // what was asked for lands before the pair leaves (both blocks' copies count on
      // the leader's barriers, and the other block waits for the leader at the end)
      if (*abort && rank == 0)
        for (long long j = i > kPairStages ? i - kPairStages : 0; j < i; ++j)
          drain_wait(full + j % kPairStages, j / kPairStages & 1, p.wait_ns);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      long long i = 0;
      int c = 0;  // accumulators taken
      bool ok = true;
      for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
        for (int it = 0; it < p.its; ++it, ++i) {
          const bool first = kFloat ? it % kChain == 0 : it == 0;
          const bool last = it == p.its - 1 || (kFloat && it % kChain == kChain - 1);
          const int s = static_cast<int>(i % kPairStages);
          if (first)
            ok = mbar_wait_cluster(acc_empty + (c & 1), (c >> 1 & 1) ^ 1, abort, p.wait_ns);
          ok = ok && mbar_wait_cluster(full + s, i / kPairStages & 1, abort, p.wait_ns);
          if (!ok) {
            raise_error(p, abort);
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * kPairStageBytes);
          multiply_stage<true>(p, sa, sa + kPairStageBytes / 2, tmem + (c & 1) * kPairTile, first);
          umma_commit_pair(empty + s, 3);
          if (last) umma_commit_pair(acc_full + (c++ & 1), 3);
        }
      }
      umma_commit_pair(drain, 1);
      drain_wait(drain, 0, p.wait_ns);
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t at = tmem + (static_cast<uint32_t>(q) << 21) + 128 * half;
    const Emitter<Out> out{p, staging + (warp - 2) * kStaging, lane};
    constexpr int kCols = Emitter<Out>::kCols;
    int c = 0;  // accumulators taken
    auto taken = [&](int b) -> bool {
      bool ok = mbar_wait_cluster(acc_full + (b & 1), b >> 1 & 1, abort, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) raise_error(p, abort);
      tc_fence_after();
      return ok;
    };
    auto give_back = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_rank(acc_empty + (b & 1), 0));
    };
    bool ok = true;
    for (int t = blockIdx.x / 2; t < tiles && ok; t += stride) {
      const long long row = static_cast<long long>(t / p.n_tiles) * kPairTile + 128 * rank + 32 * q;
      const int col = t % p.n_tiles * kPairTile + 128 * half;
      if constexpr (kFloat) {
        float acc[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = 0.f;
        const int chunks = (p.its + kChain - 1) / kChain;
        for (int k = 0; k < chunks && ok; ++k, ++c) {
          ok = taken(c);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 128; j += 16) {
            float v[16];
            tmem_ld_16cols(at + (c & 1) * kPairTile + j, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j + e] += v[e];
          }
          give_back(c);
        }
        if (!ok) break;
        // 32 columns at a time: the sums through shared memory, then a lane finishes
        // four columns of every fourth row, as global memory is read and written
#pragma unroll
        for (int j = 0; j < 128; j += kCols) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *piece(out.buf, lane, e) = make_uint4(
                __float_as_uint(acc[j + 4 * e]), __float_as_uint(acc[j + 4 * e + 1]),
                __float_as_uint(acc[j + 4 * e + 2]), __float_as_uint(acc[j + 4 * e + 3]));
          __syncwarp();
          out.finish_rows(row, col + j);
          __syncwarp();
        }
      } else {
        uint4 aux[8];
        auto fetch = [&](int j) {
          if (p.e.aux) {
#pragma unroll
            for (int i = 0; i < 8; ++i) aux[i] = out.fetch(row, col + j, i);
          }
        };
        fetch(0);  // on its way while the tile is multiplied
        ok = taken(c);
        if (!ok) break;
#pragma unroll 1
        for (int j = 0; j < 128; j += kCols) {
          if (p.e.aux) {
#pragma unroll
            for (int i = 0; i < 8; ++i) *out.mine(out.buf, i) = aux[i];
            __syncwarp();
            if (j == 0) fetch(kCols);
          }
#pragma unroll 1
          for (int e = 0; e < kCols; e += 32) {
            float v[32];
            tmem_ld_32cols(at + (c & 1) * kPairTile + j + e, v);
            if (j + e + 32 == 128) give_back(c);
            out.template finish<4>(v, col + j, e / 8);
          }
          out.flush(row, col + j);
        }
        ++c;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither block leaves while the pair's products, copies or arrivals touch it
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
  return encode_tiled(map, p, 3, dims, strides, box, true, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
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

int tile_splits(long long tiles, int its) {
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= num_sms() && its >= 4 * splits) splits *= 2;
  return splits;
}

// Whether 256 x 256 tiles on pairs of SMs finish before 128 x 128 ones: rounds of
// tiles times stages times the clocks of a stage.
bool takes_pairs(long long m, int n, int its) {
  const long long small = static_cast<long long>(ceil_div(m, kTile)) * ceil_div(n, kTile);
  const long long large = static_cast<long long>(ceil_div(m, kPairTile)) * ceil_div(n, kPairTile);
  const int s = tile_splits(small, its), sms = num_sms();
  if (sms < 2 || large > 0x3fffffff) return false;
  const long long t_small = (small * s + sms - 1) / sms * (4000 + 512ll * ((its + s - 1) / s));
  const long long t_large = 3000 + (large + sms / 2 - 1) / (sms / 2) * (1000 + 600ll * its);
  return t_large < t_small;
}

int launch_pair(const GemmDesc &d, Params p, cudaStream_t s) {
  CUtensorMap ta, tb;
  VAE_TRY(d.a.k_major ? encode_operand(&ta, d.a.p, d.parts, d.m, d.k, 128)
                      : encode_operand(&ta, d.a.p, d.parts, d.k, d.m, kBK));
  VAE_TRY(d.b.k_major ? encode_operand(&tb, d.b.p, d.parts, d.n, d.k, 128)
                      : encode_operand(&tb, d.b.p, d.parts, d.k, d.n, kBK));
  p.idesc = idesc_16bit(kPairTile, kPairTile, !d.f16, !d.a.k_major, !d.b.k_major);
  p.m_tiles = ceil_div(d.m, kPairTile);
  p.n_tiles = ceil_div(d.n, kPairTile);
  const unsigned grid = 2 * std::min(p.m_tiles * p.n_tiles, num_sms() / 2);
  return by_dtype(d.dtype, [&](auto o) -> int {
    using Out = decltype(o);
    static std::atomic<uint64_t> done{0};
    VAE_CUDA_TRY(allow_smem(gemm_pair<Out>, kPairSmem, &done));
    cudaLaunchAttribute attr[2];
    const auto cfg = launch_config(attr, grid, kPairThreads, kPairSmem, 2, p.wait, s);
    VAE_CUDA_TRY(cudaLaunchKernelEx(&cfg, gemm_pair<Out>, ta, tb, p));
    count_launches(1);
    return VAE_OK;
  });
}

int launch_tile(const GemmDesc &d, Params p, cudaStream_t s) {
  CUtensorMap ta, tb;
  VAE_TRY(d.a.k_major ? encode_operand(&ta, d.a.p, d.parts, d.m, d.k, kTile)
                      : encode_operand(&ta, d.a.p, d.parts, d.k, d.m, kBK));
  VAE_TRY(d.b.k_major ? encode_operand(&tb, d.b.p, d.parts, d.n, d.k, kTile)
                      : encode_operand(&tb, d.b.p, d.parts, d.k, d.n, kBK));
  p.idesc = idesc_16bit(kTile, kTile, !d.f16, !d.a.k_major, !d.b.k_major);
  p.m_tiles = ceil_div(d.m, kTile);
  p.n_tiles = ceil_div(d.n, kTile);
  const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
  const int splits = tile_splits(tiles, p.its);
  if (tiles * splits > 0x7fffffff) return VAE_EUNSUPPORTED;
  return by_dtype(d.dtype, [&](auto o) -> int {
    using Out = decltype(o);
    static std::atomic<uint64_t> done{0};
    VAE_CUDA_TRY(allow_smem(gemm_tile<Out>, kTileSmem, &done));
    cudaLaunchAttribute attr[2];
    const auto cfg = launch_config(attr, static_cast<unsigned>(tiles * splits), kTileThreads,
                                   kTileSmem, splits, p.wait, s);
    VAE_CUDA_TRY(cudaLaunchKernelEx(&cfg, gemm_tile<Out>, ta, tb, p, splits));
    count_launches(1);
    return VAE_OK;
  });
}

}  // namespace

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
  if (!p.err) return VAE_ECUDA;
  p.e = d.epi;
  return takes_pairs(d.m, d.n, p.its) ? launch_pair(d, p, s) : launch_tile(d, p, s);
}

}  // namespace vae
