// linear.cu -- y = act(x w^T (scaled) + bias) + residual on the tensor cores
// (cc3d_linear): bf16 or FP8 E4M3 operands, fp32 accumulation in tensor
// memory, everything after the product in the epilogue.
//
//   acc[m][n] = sum_k x[m][k] w[n][k]
//   y[m][n]   = bf16(act(acc * s_x[m] * s_w[n] + b[n]) + r[m][n])
//
// Two kernels:
//  * linear_kernel, many rows: persistent 128 x NT tiles of y (256 x NT on a
//    CTA pair), operands by TMA through a ring of 128-byte K chunks, two
//    accumulators in tensor memory so that a tile's epilogue runs under the
//    next tile's MMAs.  Bound: the tensor pipe for long K (8190 x 8192 to 2048
//    in bf16: 194 us, 1.42 PFLOP/s), the epilogue for short K (7800 x 2048 to
//    8192 in FP8: 91 us without an activation, 101 with GELU's tanh form; 7800 x
//    384 to 1152 in bf16: 10.1 us, 2.5 TB/s; 384 to 384 + residual 7.2).
//  * linear_split_kernel, few rows: bound by the weights' bytes.  The roles
//    are swapped (the 128 MMA rows are output channels, the columns are the
//    few tokens), and a cluster of CTAs splits K so that every SM streams
//    weights; the partial products meet in distributed shared memory, added
//    in rank order (the result does not depend on scheduling).  One row, 2048
//    to 12288: 11.9 us, of which the weights' 50 MB want 7.7; in FP8 8.0 of 3.9.
// (Device times of twelve calls in a graph.  In a long run of calls the power
// limit's clock makes the longest ones a fifth longer: 194 us 232, 101 us 123.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"

namespace cc3d {

namespace {

constexpr uint32_t kRowBytes = 128;  // one K chunk of a row: 64 bf16 or 128 E4M3
constexpr int kTileRows = 128;       // MMA rows per CTA
constexpr uint32_t kAStage = kTileRows * kRowBytes;
constexpr int kEpiWarps = 8;  // two per tensor-memory lane quarter
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr size_t kSmemMost = 227 * 1024;
constexpr uint64_t kDrainNs = 1000000000ull;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// act() in fp32, N pairs at a time.  One branch on the kind for all of them: a
// branch a pair kept their chains of dependent instructions from running side
// by side.
//
// What bounds this part is the unit of the exponential and the reciprocal (8
// cycles a warp each, relative error about 2^-21), so one reciprocal serves
// both of a pair: 1 / d0 = d1 / (d0 d1).
//
//  * SiLU: a / (1 + exp(-a)); GELU, tanh form: a (1 + tanh u) / 2 = a / (1 +
//    exp(-2 u)), u = sqrt(2 / pi) (a + 0.044715 a^3).  Both are max(a, 0) - |a|
//    e / (1 + e) with e = exp(-|a|) or exp(-2 |u|), taken as the square of h =
//    2^(log2(e) / 2): nothing overflows, and the values left of zero keep their
//    relative error down to bf16's least numbers, which h as a normal number
//    reaches.  |a| counts as 128 or 16 at most (e is 0 there, and +-inf give
//    their limits).
//  * GELU, erf form: max(a, 0) - |a| h, h = erfc(x) / 2, x = |a| / sqrt(2), as
//    h = t P(t) exp(-x^2) with t = 1 / (1 + x / 2).  P, of degree 8, is fitted
//    to erfcx(x) / 2t for t in (0, 1]: relative error 6e-7 in fp32.  |a| counts
//    as 64 at most (h is 0 there, and +-inf give their limits).
// NaN stays NaN and leaves the pair's other value alone.
__device__ __forceinline__ uint64_t same(float x) { return pair_of(x, x); }
// min(|a|, most)
__device__ __forceinline__ uint64_t size_of(uint64_t a, float most) {
  const float2 f = unpair(a);
  return pair_of(fminf(fabsf(f.x), most), fminf(fabsf(f.y), most));
}
// max(a, 0) - x e / (1 + e), x = |a|, e = 2^(2 w)
__device__ __forceinline__ uint64_t less_share(uint64_t a, uint64_t x, uint64_t w) {
  const float2 f = unpair(a), g = unpair(w);
  const uint64_t h = pair_of(ex2_approx(g.x), ex2_approx(g.y));
  const uint64_t e = pair_mul(h, h);
  const float2 d = unpair(pair_add(e, same(1.f)));
  const float r = rcp_approx(d.x * d.y);
  return pair_fma(pair_mul(x, e), pair_mul(same(-r), pair_of(d.y, d.x)),
                  pair_of(max_nan(f.x, 0.f), max_nan(f.y, 0.f)));
}
__device__ __forceinline__ uint64_t gelu_erf(uint64_t a) {
  const float2 f = unpair(a);
  const uint64_t x = size_of(a, 64.f);
  const float2 d = unpair(pair_fma(x, same(0.35355339f), same(1.f)));
  const float2 z = unpair(pair_mul(pair_mul(x, x), same(-0.72134752f)));
  const float r = rcp_approx(d.x * d.y);
  const uint64_t t = pair_mul(same(r), pair_of(d.y, d.x));
  uint64_t h = same(-0.021936405f);
  h = pair_fma(h, t, same(0.11050928f));
  h = pair_fma(h, t, same(-0.18864024f));
  h = pair_fma(h, t, same(0.08819317f));
  h = pair_fma(h, t, same(0.013868884f));
  h = pair_fma(h, t, same(0.09287188f));
  h = pair_fma(h, t, same(0.12302662f));
  h = pair_fma(h, t, same(0.14105959f));
  h = pair_fma(h, t, same(0.14104733f));
  h = pair_mul(pair_mul(h, t), pair_of(ex2_approx(z.x), ex2_approx(z.y)));
  return pair_fma(pair_mul(x, same(-1.f)), h, pair_of(max_nan(f.x, 0.f), max_nan(f.y, 0.f)));
}
template <int N>
__device__ __forceinline__ void activate(uint64_t (&v)[N], int act) {
  if (act == CC3D_ACT_NONE) return;
  if (act == CC3D_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t x = size_of(v[i], 128.f);
      v[i] = less_share(v[i], x, pair_mul(x, same(-0.5f * 1.4426950408889634f)));
    }
  } else if (act == CC3D_ACT_GELU_TANH) {
    constexpr float k0 = -0.79788456080286536f * 1.4426950408889634f;
    constexpr float k1 = 0.044715f * k0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t x = size_of(v[i], 16.f);
      v[i] = less_share(v[i], x, pair_mul(x, pair_fma(pair_mul(x, x), same(k1), same(k0))));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gelu_erf(v[i]);
  }
}

// Columns of y that an epilogue warp finishes at a time: rows of 64 bytes in
// its own part of shared memory, from where TMA stores them (and where it puts
// the residual's).  (A thread holds a row, so its own stores would touch 32
// lines at a time; 128-byte rows would cost the ring a stage.)
constexpr int kOutCols = 32;
constexpr uint32_t kOutBuf = 32u * kOutCols * 2u;

struct Layout {
  uint32_t stage, out, params, bars, total;  // bytes
};
// The ring of operand chunks, and for the many-row kernel the epilogue warps'
// two output buffers and column parameters (bias and scale).
__host__ __device__ inline Layout ring_layout(int b_rows, int stages, int nt = 0) {
  Layout l;
  l.stage = kAStage + static_cast<uint32_t>(b_rows) * kRowBytes;
  l.out = l.stage * static_cast<uint32_t>(stages);
  l.params = l.out + (nt ? 2u * kEpiWarps * kOutBuf : 0u);
  l.bars = l.params + (nt ? kEpiWarps * (nt / 2) * 8u : 0u);
  l.total = l.bars + 8u * (2u * stages + 5u + 2u * kEpiWarps) + 16u;
  return l;
}

// Tiles of a launch, dealt to clusters round robin in bands of kBand row
// tiles: the clusters of one wave share few rows of x and few of w in L2.
// (Divisions by multiplication: 0.2 us of every epilogue's tile otherwise.)
constexpr int kBand = 8;
struct Tile {
  int mt, nt;
  __device__ __forceinline__ Tile(const LinearArgs &p, int i) {
    const int band = p.by_band.quotient(i), r = i - band * kBand * p.n_tiles;
    const int rows = min(kBand, p.m_tiles - band * kBand);
    nt = rows == kBand ? r / kBand : p.by_last.quotient(r);
    mt = band * kBand + (r - nt * rows);
  }
};

template <bool FP8, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_y,
                  const __grid_constant__ CUtensorMap map_r, const LinearArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int b_rows = PAIR ? p.nt / 2 : p.nt;  // weight rows this CTA loads
  const Layout L = ring_layout(b_rows, p.stages, p.nt);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L.bars);
  uint64_t *empty = full + p.stages;
  uint64_t *acc_full = empty + p.stages;  // [2]
  uint64_t *acc_empty = acc_full + 2;     // [2]
  uint64_t *drain = acc_empty + 2;
  uint64_t *res_full = drain + 1;  // [epilogue warp][2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(res_full + 2 * kEpiWarps);

  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int cid = PAIR ? blockIdx.x / 2 : blockIdx.x;
  const int ncl = PAIR ? gridDim.x / 2 : gridDim.x;
  const bool leader = rank == 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kChunk = FP8 ? 128 : 64;  // K elements of a chunk
  const int nk = (p.k + kChunk - 1) / kChunk;
  constexpr int kRowsPerTile = PAIR ? 2 * kTileRows : kTileRows;
  const int n_tiles = p.m_tiles * p.n_tiles;
  const uint32_t tmem_cols = 2u * p.nt;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(&res_full[i], 1);
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
    prefetch_tmap(&map_y);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, tmem_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, tmem_cols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  bool ok = true;
  griddep_launch_dependents();

  if (warp == 0) {
    if (elect_one()) {
      // both CTAs' loads complete on the leader's barriers, which the leader
      // arms for the bytes of both
      const uint32_t lead_full = PAIR ? mapa_shared(smem_u32(full), 0u) : 0u;
      const uint32_t tx = (PAIR ? 2u : 1u) * L.stage;
      int s = 0;
      uint32_t ph = 0, used = 0, par = 0;
      griddep_wait();
      for (int t = cid; t < n_tiles && ok; t += ncl) {
        const Tile tile(p, t);
        const int row_x = tile.mt * kRowsPerTile + rank * kTileRows;
        const int row_w = tile.nt * p.nt + rank * b_rows;
        for (int kc = 0; kc < nk; ++kc) {
          if (!mbar_wait_soon(&empty[s], ph ^ 1, p.wait_limit_ns, p.status, 20)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[s], tx);
          used |= 1u << s;
          par = (par & ~(1u << s)) | (ph << s);
          const uint32_t dst = smem_base + s * L.stage;
          if constexpr (PAIR) {
            tma_load_2d_pair(dst, &map_x, lead_full + 8u * s, kc * kChunk, row_x);
            tma_load_2d_pair(dst + kAStage, &map_w, lead_full + 8u * s, kc * kChunk, row_w);
          } else {
            tma_load_2d(dst, &map_x, &full[s], kc * kChunk, row_x);
            tma_load_2d(dst + kAStage, &map_w, &full[s], kc * kChunk, row_w);
          }
          if (++s == p.stages) { s = 0; ph ^= 1; }
        }
      }
      // Every load lands before the CTA may exit.  A pair's loads complete on
      // the leader's barriers, so its follower waits until the products have
      // read them, and where they never do (the leader gave up), long enough
      // for a load that is under way.
      bool landed = true;
      for (int i = 0; i < p.stages; ++i)
        if (used >> i & 1u)
          landed &= leader ? mbar_wait_bounded(&full[i], par >> i & 1u, kDrainNs, nullptr, 0)
                           : mbar_wait_bounded(&empty[i], par >> i & 1u, p.wait_limit_ns, nullptr, 0);
      if (!leader && !landed)
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000ull;) {
        }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      griddep_wait();  // (a wait's limit does not count the kernels before)
      const uint32_t idesc = FP8 ? idesc_e4m3_f32(kRowsPerTile, p.nt)
                                 : idesc_bf16_f32(kRowsPerTile, p.nt);
      const uint64_t a0 = smem_desc_sw128(smem_base, 1024u);
      const uint64_t b0 = smem_desc_sw128(smem_base + kAStage, 1024u);
      int s = 0, it = 0;
      uint32_t ph = 0;
      for (int t = cid; t < n_tiles && ok; t += ncl, ++it) {
        const int buf = it & 1;
        const uint32_t up = static_cast<uint32_t>((it >> 1) & 1);
        if (!(PAIR ? mbar_wait_bounded_cluster(&acc_empty[buf], up ^ 1, p.wait_limit_ns, p.status,
                                               21)
                   : mbar_wait_bounded(&acc_empty[buf], up ^ 1, p.wait_limit_ns, p.status, 21))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * p.nt);
        for (int kc = 0; kc < nk; ++kc) {
          if (!mbar_wait_soon(&full[s], ph, p.wait_limit_ns, p.status, 22)) {
            ok = false;
            break;
          }
          const uint64_t a = a0 + ((s * L.stage) >> 4), b = b0 + ((s * L.stage) >> 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t acc = (kc | j) != 0;
            if constexpr (PAIR && FP8) umma_e4m3_pair(d, a + 2 * j, b + 2 * j, idesc, acc);
            else if constexpr (PAIR) umma_bf16_pair(d, a + 2 * j, b + 2 * j, idesc, acc);
            else if constexpr (FP8) umma_e4m3(d, a + 2 * j, b + 2 * j, idesc, acc);
            else umma_bf16(d, a + 2 * j, b + 2 * j, idesc, acc);
          }
          if constexpr (PAIR) umma_commit_pair(&empty[s], 3);
          else umma_commit(&empty[s]);
          if (++s == p.stages) { s = 0; ph ^= 1; }
        }
        if (!ok) break;
        if constexpr (PAIR) umma_commit_pair(&acc_full[buf], 3);
        else umma_commit(&acc_full[buf]);
      }
      // every MMA is complete before tensor memory is freed
      if constexpr (PAIR) umma_commit_pair(drain, 1);
      else umma_commit(drain);
      mbar_wait_bounded(drain, 0, kDrainNs, nullptr, 0);
    }
  } else {
    const int q = warp % 4;           // tensor-memory lanes this warp may read
    const int half = (warp - 2) / 4;  // its half of the tile's columns
    const int cols = p.nt / 2;
    uint8_t *out = smem + L.out + (warp - 2) * 2u * kOutBuf;
    float *s_bias = reinterpret_cast<float *>(smem + L.params) + (warp - 2) * 2 * cols;
    float *s_scale = s_bias + cols;
    uint64_t *res = res_full + 2 * (warp - 2);
    const uint32_t free_bar = PAIR ? mapa_shared(smem_u32(acc_empty), 0u) : 0u;
    // 16-byte piece i of this thread's row, where the 64-byte swizzle puts it
    auto piece = [&](int buf, int i) {
      return reinterpret_cast<uint4 *>(out + buf * kOutBuf + lane * 64u +
                                       ((static_cast<uint32_t>(i) ^ ((lane >> 1) & 3u)) << 4));
    };
    griddep_wait();
    int it = 0, ob = 0;      // tiles, and output buffers used so far
    uint32_t res_par = 0;    // phase parity of the two residual barriers
    auto row0_of = [&](int mt) { return mt * kRowsPerTile + rank * kTileRows + q * 32; };
    // the residual of one buffer's worth of a tile on its way (lane 0): the
    // buffer's last store has been read
    auto fetch_residual = [&](const Tile &tile, int u, int buf) {
      bulk_groups_wait_read<0>();
      mbar_arrive_expect_tx(&res[buf], kOutBuf);
      tma_load_2d(smem_u32(out) + buf * kOutBuf, &map_r, &res[buf],
                  tile.nt * p.nt + half * cols + u * kOutCols, row0_of(tile.mt));
    };
    // bias and weight scale of columns lane, lane + 32, ..., the row's scale
    float next_bias[4], next_scale[4], next_xs = 1.f;
    auto fetch_params = [&](const Tile &tile) {
      const int c0 = tile.nt * p.nt + half * cols + lane, row = row0_of(tile.mt) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        const bool used = i * 32 < cols && c < p.n;
        next_bias[i] = p.bias && used ? p.bias[c] : 0.f;
        if constexpr (FP8) next_scale[i] = used ? p.w_scales[c] : 0.f;
      }
      if constexpr (FP8)
        next_xs = row < p.m ? (p.x_scales ? p.x_scales[row] : p.x_scale) : 1.f;
    };
    Tile next(p, cid);  // (a cluster has a tile at least)
    fetch_params(next);
    if (p.residual && lane == 0) fetch_residual(next, 0, 0);
    for (int t = cid; t < n_tiles && ok; t += ncl, ++it) {
      const Tile tile = next;
      const bool more = t + ncl < n_tiles;
      const int n0 = tile.nt * p.nt + half * cols;
      // the columns' parameters where every lane reads them, and the next
      // tile's on their way
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * 32 < cols) {
          s_bias[i * 32 + lane] = next_bias[i];
          if constexpr (FP8) s_scale[i * 32 + lane] = next_scale[i];
        }
      __syncwarp();
      const float xs = next_xs;
      if (more) {
        next = Tile(p, t + ncl);
        fetch_params(next);
      }
      const int buf = it & 1;
      const uint32_t up = static_cast<uint32_t>((it >> 1) & 1);
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded(&acc_full[buf], up, p.wait_limit_ns, p.status, 23));
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(buf * p.nt + half * cols);
      uint32_t raw[32];
      tmem_ld32_nowait(taddr, raw);
      for (int u = 0; u < cols / kOutCols; ++u, ob ^= 1) {
        if (p.residual) {
          // the next buffer's worth (of this tile or the next one) on its way
          if (lane == 0) {
            if ((u + 1) * kOutCols < cols) fetch_residual(tile, u + 1, ob ^ 1);
            else if (more) fetch_residual(next, 0, ob ^ 1);
          }
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&res[ob], (res_par >> ob) & 1u,
                                                         p.wait_limit_ns, p.status, 27));
          res_par ^= 1u << ob;
          if (!ok) {
            tmem_wait_ld();  // (on their way to registers)
            break;
          }
        } else {
          if (lane == 0) bulk_groups_wait_read<1>();
          __syncwarp();
        }
        tmem_wait_ld();
        tmem_regs_after_wait<32>(raw);
        if ((u + 1) * kOutCols == cols) {
          // the accumulator is in registers: the next tile's MMAs may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) mbar_arrive_remote_relaxed(free_bar + 8u * buf);
            else mbar_arrive(&acc_empty[buf]);
          }
        }
        const float *bias = s_bias + u * kOutCols, *scale = s_scale + u * kOutCols;
        uint64_t v[kOutCols / 2];
#pragma unroll
        for (int e = 0; e < kOutCols / 2; ++e)
          v[e] = pair_of(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1]));
        const uint64_t xs2 = pair_of(xs, xs);
#pragma unroll
        for (int e = 0; e < kOutCols / 2; e += 2) {
          const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(bias + 2 * e);
          if constexpr (FP8) {
            const ulonglong2 s2 = *reinterpret_cast<const ulonglong2 *>(scale + 2 * e);
            v[e] = pair_fma(v[e], pair_mul(xs2, s2.x), b2.x);
            v[e + 1] = pair_fma(v[e + 1], pair_mul(xs2, s2.y), b2.y);
          } else {
            v[e] = pair_add(v[e], b2.x);
            v[e + 1] = pair_add(v[e + 1], b2.y);
          }
        }
        activate(v, p.act);
        if ((u + 1) * kOutCols < cols) tmem_ld32_nowait(taddr + (u + 1) * kOutCols, raw);
        if (p.residual) {
#pragma unroll
          for (int g = 0; g < kOutCols / 8; ++g) {
            const uint4 r4 = *piece(ob, g);
            const uint32_t rw[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[4 * g + e] = pair_add(v[4 * g + e],
                                      pair_of(__uint_as_float(rw[e] << 16),
                                              __uint_as_float(rw[e] & 0xffff0000u)));
          }
        }
#pragma unroll
        for (int g = 0; g < kOutCols / 8; ++g) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpair(v[4 * g + e]);
            o[e] = pack_bf16x2(f.x, f.y);
          }
          *piece(ob, g) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&map_y, smem_u32(out) + ob * kOutBuf, n0 + u * kOutCols, row0_of(tile.mt));
          bulk_group_commit();
        }
      }
    }
    if (lane == 0) {
      // nothing of this warp's is under way when the CTA ends (a residual
      // fetch neither after a wait that ran out)
      bulk_groups_wait();
      if (!ok && p.residual)
        for (int i = 0; i < 2; ++i)
          mbar_wait_bounded(&res[i], (res_par >> i) & 1u, kDrainNs, nullptr, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // (the peer may still write or signal into this CTA)
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, tmem_cols);
    else tmem_dealloc(tmem_base, tmem_cols);
  }
}

// ---- few rows -----------------------------------------------------------------------

constexpr int kSplitThreads = 192;
// Shared memory of a CTA, at least: with it two of them fill an SM, and none
// fits beside a kernel that holds all of an SM's tensor memory (those take 116
// KB or more).  Otherwise clusters of two kernels on two streams could each
// hold tensor memory that the other's second CTA waits for.
constexpr size_t kSplitSmem = 112 * 1024;

__host__ __device__ inline uint32_t split_total(int nt, int stages) {
  const Layout l = ring_layout(nt, stages);
  // the ring, later the partial sums [nt][128] fp32 in its place
  const uint32_t part = static_cast<uint32_t>(nt) * kTileRows * 4u;
  return (l.bars > part ? l.bars : part) + 8u * (2u * stages + 1u) + 16u;
}
inline size_t split_smem(int nt, int stages) {
  const size_t used = split_total(nt, stages) + 1024;
  return used > kSplitSmem ? used : kSplitSmem;
}

template <bool FP8>
__global__ void __launch_bounds__(kSplitThreads)
    linear_split_kernel(const __grid_constant__ CUtensorMap map_x,
                        const __grid_constant__ CUtensorMap map_w, const LinearArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const Layout L = ring_layout(p.nt, p.stages);
  const uint32_t part_bytes = static_cast<uint32_t>(p.nt) * kTileRows * 4u;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + (L.bars > part_bytes ? L.bars : part_bytes));
  uint64_t *empty = full + p.stages;
  uint64_t *acc_full = empty + p.stages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 1);

  const int split = p.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / split;
  const int w_tiles = (p.n + kTileRows - 1) / kTileRows;
  const int row_w = (tile % w_tiles) * kTileRows;  // output channels of the tile
  const int row_x = (tile / w_tiles) * p.nt;       // and its tokens
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kChunk = FP8 ? 128 : 64;
  const int nk = (p.k + kChunk - 1) / kChunk;
  const int k0 = static_cast<int>(static_cast<long long>(nk) * rank / split);
  const int k1 = static_cast<int>(static_cast<long long>(nk) * (rank + 1) / split);
  uint32_t tmem_cols = 32;
  while (tmem_cols < static_cast<uint32_t>(p.nt)) tmem_cols *= 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0, used = 0, par = 0;
      for (int kc = k0; kc < k1; ++kc) {
        if (!mbar_wait_soon(&empty[s], ph ^ 1, p.wait_limit_ns, p.status, 24)) break;
        mbar_arrive_expect_tx(&full[s], L.stage);
        used |= 1u << s;
        par = (par & ~(1u << s)) | (ph << s);
        const uint32_t dst = smem_base + s * L.stage;
        tma_load_2d(dst, &map_w, &full[s], kc * kChunk, row_w);
        tma_load_2d(dst + kAStage, &map_x, &full[s], kc * kChunk, row_x);
        if (++s == p.stages) { s = 0; ph ^= 1; }
      }
      for (int i = 0; i < p.stages; ++i)
        if (used >> i & 1u) mbar_wait_bounded(&full[i], par >> i & 1u, kDrainNs, nullptr, 0);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc =
          FP8 ? idesc_e4m3_f32(kTileRows, p.nt) : idesc_bf16_f32(kTileRows, p.nt);
      const uint64_t a0 = smem_desc_sw128(smem_base, 1024u);
      const uint64_t b0 = smem_desc_sw128(smem_base + kAStage, 1024u);
      int s = 0;
      uint32_t ph = 0;
      for (int kc = k0; kc < k1; ++kc) {
        if (!mbar_wait_soon(&full[s], ph, p.wait_limit_ns, p.status, 25)) break;
        const uint64_t a = a0 + ((s * L.stage) >> 4), b = b0 + ((s * L.stage) >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t acc = kc > k0 || j > 0;
          if constexpr (FP8) umma_e4m3(tmem_base, a + 2 * j, b + 2 * j, idesc, acc);
          else umma_bf16(tmem_base, a + 2 * j, b + 2 * j, idesc, acc);
        }
        umma_commit(&empty[s]);
        if (++s == p.stages) { s = 0; ph ^= 1; }
      }
      // (also after a wait that ran out: the MMAs issued so far complete)
      umma_commit(acc_full);
    }
  }
  // The partial sums, channel-fastest, take the ring's place: every load has
  // landed and every MMA has read it once acc_full completes.
  float *part = reinterpret_cast<float *>(smem);
  if (warp >= 2) {
    const int q = warp % 4;
    uint32_t got = 0;
    if (lane == 0)
      got = mbar_wait_bounded(acc_full, 0, p.wait_limit_ns + kDrainNs, p.status, 26) ? 1u : 0u;
    got = __shfl_sync(0xffffffffu, got, 0);
    tc_fence_after();
    if (got) {
      const int used_cols = min(p.nt, p.m - row_x);
      for (int j = 0; j < used_cols; j += 16) {
        __syncwarp();
        uint32_t raw[16];
        tmem_ld16_nowait(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + j, raw);
        tmem_wait_ld();
        tmem_regs_after_wait<16>(raw);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          part[(j + e) * kTileRows + q * 32 + lane] = __uint_as_float(raw[e]);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
  // rank r finishes the tokens r, r + split, ...; a thread two channels
  const int pair_c = threadIdx.x % 64;
  const int c = row_w + 2 * pair_c;
  if (c < p.n) {
    float ws0 = 1.f, ws1 = 1.f, b0 = 0.f, b1 = 0.f;
    if constexpr (FP8) {
      ws0 = p.w_scales[c];
      ws1 = p.w_scales[c + 1];
    }
    if (p.bias) {
      b0 = p.bias[c];
      b1 = p.bias[c + 1];
    }
    const int tokens = min(p.nt, p.m - row_x);
    for (int j = rank + split * (threadIdx.x / 64); j < tokens; j += split * (kSplitThreads / 64)) {
      const uint32_t at = smem_base + static_cast<uint32_t>(j * kTileRows + 2 * pair_c) * 4u;
      float v[2] = {0.f, 0.f};
      if (split == 1) {
        v[0] = part[j * kTileRows + 2 * pair_c];
        v[1] = part[j * kTileRows + 2 * pair_c + 1];
      } else {
        for (int r = 0; r < split; ++r) {
          const float2 f = ld_cluster_f32x2(mapa_shared(at, static_cast<uint32_t>(r)));
          v[0] += f.x;
          v[1] += f.y;
        }
      }
      const long long row = row_x + j;
      if constexpr (FP8) {
        const float xs = p.x_scales ? p.x_scales[row] : p.x_scale;
        v[0] *= xs * ws0;
        v[1] *= xs * ws1;
      }
      v[0] += b0;
      v[1] += b1;
      {
        uint64_t a[1] = {pair_of(v[0], v[1])};
        activate(a, p.act);
        const float2 f = unpair(a[0]);
        v[0] = f.x;
        v[1] = f.y;
      }
      if (p.residual) {
        const uint32_t rw = *reinterpret_cast<const uint32_t *>(p.residual + row * p.ldr + c);
        v[0] += __uint_as_float(rw << 16);
        v[1] += __uint_as_float(rw & 0xffff0000u);
      }
      *reinterpret_cast<uint32_t *>(p.y + row * p.ldy + c) = pack_bf16x2(v[0], v[1]);
    }
  }
  if (split > 1) cluster_sync();  // (peers may still read this CTA's partial sums)
}

// ---- choice of kernel and tile -----------------------------------------------------

using LinearKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                              const CUtensorMap, const LinearArgs);
using SplitKernel = void (*)(const CUtensorMap, const CUtensorMap, const LinearArgs);

const LinearKernel kLinear[2][2] = {{linear_kernel<false, false>, linear_kernel<false, true>},
                                    {linear_kernel<true, false>, linear_kernel<true, true>}};
const SplitKernel kSplit[2] = {linear_split_kernel<false>, linear_split_kernel<true>};

int many_stages(int pair, int nt) {
  int st = 8;
  while (ring_layout(pair ? nt / 2 : nt, st, nt).total + 1024 > kSmemMost) --st;
  return st;
}
int split_stages(int nt) {
  // two CTAs per SM
  int st = 8;
  while (st > 2 && split_total(nt, st) + 1024 > kSmemMost / 2 - 1024) --st;
  return st;
}

cudaLaunchConfig_t launch_config(unsigned grid, unsigned block, size_t smem, unsigned cluster,
                                 cudaLaunchAttribute *attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cfg;
}

// Per device, on first use: the kernels' shared-memory limit, how many CTA
// pairs of the persistent kernel and how many clusters of the split kernel
// (by N tile / 16 and split) are resident at once.
struct Prepared {
  bool done;
  int pairs[2];
  int clusters[2][9][9];
};
std::mutex g_prepare_mu;
Prepared g_prepared[64];

int resident(const void *k, unsigned block, size_t smem, unsigned cluster, int otherwise) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = launch_config(cluster, block, smem, cluster, attr, nullptr);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return otherwise;
  }
  return n;
}

cudaError_t prepare_kernels(int sm_count, const Prepared **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_prepare_mu);
  Prepared &p = g_prepared[dev];
  if (!p.done) {
    for (int f = 0; f < 2; ++f) {
      const void *ks[3] = {reinterpret_cast<const void *>(kLinear[f][0]),
                           reinterpret_cast<const void *>(kLinear[f][1]),
                           reinterpret_cast<const void *>(kSplit[f])};
      for (const void *k : ks) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemMost));
        if (e != cudaSuccess) return e;
      }
      p.pairs[f] = resident(ks[1], kThreads, kSmemMost, 2, sm_count / 2);
      for (int n = 1; n <= 8; ++n)
        for (int s = 1; s <= 8; ++s)
          p.clusters[f][n][s] =
              s == 1 ? 2 * sm_count
                     : resident(ks[2], kSplitThreads,
                                split_smem(16 * n, split_stages(16 * n)),
                                static_cast<unsigned>(s), 0);
    }
    p.done = true;
  }
  *out = &p;
  return cudaSuccess;
}

}  // namespace

// Estimated cycles, from measurements of both kernels at K = 384 to 8192 and 1
// to 16384 rows.  Many rows: rounds of tiles, each the longest of its products
// (four a chunk, N / 2 + 44 cycles), its operands (68 bytes a cycle and SM from
// L2) and its epilogue.  Few rows: the operands' bytes at 45 a cycle and SM and
// at 3500 from HBM, and the joining of the parts.
LinearChoice choose_linear(int m, int n, int k, int act, bool fp8, int sm_count, int pairs,
                           const int (*clusters)[9]) {
  const int nk = (k + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
  LinearChoice best = {};
  double best_t = 1e300;
  const int shapes[4][2] = {{1, 256}, {1, 128}, {0, 128}, {0, 64}};
  for (const auto &sh : shapes) {
    const int pair = sh[0], nt = sh[1], rows = pair ? 256 : 128;
    const double tiles = static_cast<double>((m + rows - 1) / rows) * ((n + nt - 1) / nt);
    const int slots = pair ? pairs : sm_count;
    const double rounds = std::ceil(tiles / slots);
    const double bytes = kAStage + (pair ? nt / 2 : nt) * static_cast<double>(kRowBytes);
    const double epi = 600.0 + nt * (act == CC3D_ACT_NONE ? 14.0 : 30.0);
    double per = nk * 4.0 * (nt / 2.0 + 44.0);
    per = std::fmax(per, nk * bytes / 68.0);
    per = std::fmax(per, epi);
    const double t = 5500.0 + 1000.0 * pair + epi + rounds * (per + 500.0);
    if (t < best_t) {
      best_t = t;
      best = LinearChoice{false, pair, nt, many_stages(pair, nt), 1};
    }
  }
  if (m <= 512) {
    int nt = 16;
    while (nt < m && nt < 128) nt += 16;
    for (; nt >= 64 || nt >= m; nt -= 64) {  // (the tokens' own tile, and a half of 128)
      const double tiles = static_cast<double>((n + 127) / 128) * ((m + nt - 1) / nt);
      const double hbm = (static_cast<double>(n) + m) * nk * kRowBytes / 3500.0;
      const double bytes = kAStage + nt * static_cast<double>(kRowBytes);
      for (int split = 1; split <= 8 && split <= nk; ++split) {
        const int fit = clusters[nt / 16][split];
        if (fit < 1) continue;
        const double waves = std::ceil(tiles / fit);
        const double share = tiles * split > sm_count ? 1.8 : 1.0;  // two CTAs of an SM
        const double stream = waves * std::ceil(static_cast<double>(nk) / split) * bytes * share / 45.0;
        const double t = 5400.0 + (split > 1 ? 800.0 : 0.0) + 50.0 * split + 30.0 * nt +
                         std::hypot(hbm, stream) + 900.0 * (waves - 1.0);
        if (t < best_t) {
          best_t = t;
          best = LinearChoice{true, 0, nt, split_stages(nt), split};
        }
      }
      if (nt <= 64) break;
    }
  }
  return best;
}

cudaError_t launch_linear(LinearArgs a, const void *x, long long ldx, const void *w,
                          long long ldw, bool fp8, int sm_count, cudaStream_t stream) {
  const Prepared *pre = nullptr;
  cudaError_t e = prepare_kernels(sm_count, &pre);
  if (e != cudaSuccess) return e;
  const LinearChoice c = choose_linear(a.m, a.n, a.k, a.act, fp8, sm_count, pre->pairs[fp8],
                                       pre->clusters[fp8]);
  a.nt = c.nt;
  a.stages = c.stages;
  a.split = c.split;
  const int esz = fp8 ? 1 : 2;
  const uint32_t chunk = kRowBytes / esz;
  const uint32_t x_rows = c.split_kernel ? c.nt : kTileRows;
  const uint32_t w_rows = c.split_kernel ? kTileRows : (c.pair ? c.nt / 2 : c.nt);
  CUtensorMap mx, mw;
  const uint64_t dx[2] = {static_cast<uint64_t>(a.k), static_cast<uint64_t>(a.m)};
  const uint64_t dw[2] = {static_cast<uint64_t>(a.k), static_cast<uint64_t>(a.n)};
  const uint64_t sx[1] = {static_cast<uint64_t>(ldx) * esz};
  const uint64_t sw[1] = {static_cast<uint64_t>(ldw) * esz};
  const uint32_t bx[2] = {chunk, x_rows}, bw[2] = {chunk, w_rows};
  if (!encode_rows_map(&mx, x, esz, 2, dx, sx, bx) || !encode_rows_map(&mw, w, esz, 2, dw, sw, bw))
    return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  if (c.split_kernel) {
    const unsigned tiles = static_cast<unsigned>(((a.n + 127) / 128) * ((a.m + c.nt - 1) / c.nt));
    const cudaLaunchConfig_t cfg =
        launch_config(tiles * c.split, kSplitThreads, split_smem(c.nt, c.stages),
                      static_cast<unsigned>(c.split), attr, stream);
    e = cudaLaunchKernelEx(&cfg, kSplit[fp8], mx, mw, a);
    count_launch();
    return e;
  }
  CUtensorMap my, mr;
  const uint64_t dy[2] = {static_cast<uint64_t>(a.n), static_cast<uint64_t>(a.m)};
  const uint64_t sy[1] = {static_cast<uint64_t>(a.ldy) * 2};
  const uint64_t sr[1] = {static_cast<uint64_t>(a.ldr) * 2};
  const uint32_t by[2] = {kOutCols, 32};
  if (!encode_rows_map(&my, a.y, 2, 2, dy, sy, by)) return cudaErrorInvalidValue;
  mr = my;
  if (a.residual && !encode_rows_map(&mr, a.residual, 2, 2, dy, sr, by))
    return cudaErrorInvalidValue;
  const int rows = c.pair ? 256 : 128;
  a.m_tiles = (a.m + rows - 1) / rows;
  a.n_tiles = (a.n + c.nt - 1) / c.nt;
  const long long tiles = static_cast<long long>(a.m_tiles) * a.n_tiles;
  if (tiles > INT32_MAX / 2) return cudaErrorNotSupported;
  a.by_band = FastDiv(static_cast<uint32_t>(kBand * a.n_tiles));
  a.by_last = FastDiv(static_cast<uint32_t>(a.m_tiles % kBand ? a.m_tiles % kBand : kBand));
  const long long slots = c.pair ? pre->pairs[fp8] : sm_count;
  const unsigned cluster = c.pair ? 2u : 1u;
  // (more than half an SM's shared memory: one CTA per SM, which the tensor
  // memory wants)
  const cudaLaunchConfig_t cfg = launch_config(
      static_cast<unsigned>(tiles < slots ? tiles : slots) * cluster, kThreads,
      ring_layout(c.pair ? c.nt / 2 : c.nt, c.stages, c.nt).total + 1024, cluster, attr, stream);
  e = cudaLaunchKernelEx(&cfg, kLinear[fp8][c.pair], mx, mw, my, mr, a);
  count_launch();
  return e;
}

}  // namespace cc3d
