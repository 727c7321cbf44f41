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
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= num_sms() && p.its >= 4 * splits) splits *= 2;
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
  if (its > 0x7fffffff || d.m > 0x7fffffff - kTile) return VAE_EUNSUPPORTED;
  p.its = static_cast<int>(its);
  p.a_k = d.a.k_major;
  p.b_k = d.b.k_major;
  p.wait = d.wait;
  p.wait_ns = wait_limit_ns();
  p.err = device_error_word();
  if (!p.err) return VAE_ECUDA;
  p.e = d.epi;
  return launch_tile(d, p, s);
}

}  // namespace vae
