// attention.cu -- attention in a sliding window of frames with sink frames
// (cc3d_attention) and the cache update that goes with it (cc3d_kv_append).
//
// A frame is `frame` consecutive tokens.  A query of frame i sees the keys of
// frame j when j <= i and (i - j < window or j < sinks); frames of one token
// give the token-wise sliding window, window = 1 without sinks attention
// within each frame.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i k_j - m_i)
//
// One pass over the keys with a running maximum m and sum l per query row
// (fp32).  A CTA takes 128 or 256 query rows of one kv head; the query heads
// that share it are rows of the same tile, so a key is read once for all of
// them.  S = Q K^T and O = P V run on the tensor cores with both
// accumulators in tensor memory; P replaces S in place as bf16 (values of a
// softmax carry no more than the inputs' 8 bits) and feeds the second
// product from there.  O is rescaled only when a row's maximum has grown by
// more than 2^8 since the last time: until then p may reach 256, which
// changes no rounding error (bf16 and fp32 are relative).
//
// Keys are walked in the cache's own order, tile by tile; tiles no query of
// the CTA sees are skipped, tiles all of them see are not masked.  With few
// query rows a cluster of CTAs splits the keys, and the parts meet in
// distributed shared memory, added in rank order.
//
// Bound: the tensor pipe and the exponentials (16 a cycle and SM, as many
// cycles as the two products take at d = 128) for many rows, the cache's
// bytes for one token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"

namespace cc3d {

namespace {

constexpr int kRows = 128;                        // query rows of an MMA tile
constexpr uint32_t kQChunk = kRows * 128;         // 64 channels of them
constexpr size_t kSmemMost = 227 * 1024;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr float kGrow = 8.f;                      // log2 of the growth that p may take
constexpr uint32_t kTmemCols = 512;

// Token ranges of the cache, in slot order, and the tiles that hold them.
struct Ranges {
  int lo[3], hi[3];  // tokens [lo, hi); empty where hi <= lo
  __device__ __forceinline__ bool has(int s) const {
    return (s >= lo[0] && s < hi[0]) || (s >= lo[1] && s < hi[1]) || (s >= lo[2] && s < hi[2]);
  }
  // bit i: whether token s + i is in them (i < 32)
  __device__ __forceinline__ uint32_t bits(int s) const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) m |= below(hi[i] - s) & ~below(lo[i] - s);
    return m;
  }
  static __device__ __forceinline__ uint32_t below(int n) {  // bits 0 .. n - 1
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  }
  // whether [a, b) lies inside one of them
  __device__ __forceinline__ bool covers(int a, int b) const {
    return (a >= lo[0] && b <= hi[0]) || (a >= lo[1] && b <= hi[1]) || (a >= lo[2] && b <= hi[2]);
  }
};

// The tokens of frames first .. last (none if last < first), and of the
// sinks up to frame `last_sink`, in a cache of the given shape.
__device__ __forceinline__ Ranges token_ranges(const CacheShape &c, int first, int last,
                                               int last_sink) {
  Ranges r;
  const int f = c.frame;
  const int ns = last_sink < 0 ? 0 : (last_sink >= c.sinks ? c.sinks : last_sink + 1);
  r.lo[0] = 0;
  r.hi[0] = ns * f;
  r.lo[1] = r.hi[1] = r.lo[2] = r.hi[2] = 0;
  if (c.ring == 0) {
    if (first < 0) first = 0;
    if (last >= first) {
      r.lo[2] = first * f;
      r.hi[2] = (last + 1) * f;
    }
  } else {
    if (first < c.sinks) first = c.sinks;
    const int count = last - first + 1;
    if (last >= first) {
      if (count >= c.ring) {
        r.lo[2] = c.sinks * f;
        r.hi[2] = (c.sinks + c.ring) * f;
      } else {
        const int s0 = (first - c.sinks) % c.ring, e = s0 + count;
        r.lo[2] = (c.sinks + s0) * f;
        r.hi[2] = (c.sinks + (e < c.ring ? e : c.ring)) * f;
        if (e > c.ring) {  // wrapped around
          r.lo[1] = c.sinks * f;
          r.hi[1] = (c.sinks + e - c.ring) * f;
        }
      }
    }
  }
  return r;
}

// The key tiles of KT tokens that meet the ranges, each once, ascending.
template <int KT>
struct TileList {
  int start[3], count[3], total;
  __device__ __forceinline__ explicit TileList(const Ranges &r) {
    int end = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      start[i] = count[i] = 0;
      if (r.hi[i] > r.lo[i]) {
        int a = r.lo[i] / KT;
        const int b = (r.hi[i] - 1) / KT + 1;
        if (a < end) a = end;
        if (b > a) {
          start[i] = a;
          count[i] = b - a;
          end = b;
          total += b - a;
        }
      }
    }
  }
  __device__ __forceinline__ int at(int j) const {
    if (j < count[0]) return start[0] + j;
    j -= count[0];
    if (j < count[1]) return start[1] + j;
    return start[2] + (j - count[1]);
  }
};

// What one CTA (or cluster) works on.
struct Item {
  int seq, kv_head, tok0;  // first query token
  int live;                // query tokens of the sequence (all frames of its chunk)
  int base;                // frame of query token 0 (negative: seen by nothing)
};

__device__ __forceinline__ void lengths(const CacheShape &c, int seq, int &chunk, int &all) {
  all = c.k_frames ? c.k_frames[seq] : c.total;
  if (all < 0) all = 0;
  if (c.ring == 0 && all > c.slots) all = c.slots;
  chunk = c.q_frames ? c.q_frames[seq] : c.t;
  chunk = chunk < 0 ? 0 : (chunk > c.t ? c.t : chunk);
}

template <int KT>
__host__ __device__ inline uint32_t attn_bars_off(int nq, int chunks, int stages) {
  return static_cast<uint32_t>(nq * chunks) * kQChunk + static_cast<uint32_t>(stages) * KT * 128u;
}
template <int KT>
__host__ __device__ inline uint32_t attn_smem(int nq, int chunks, int stages) {
  // barriers, and the rows' (maximum, sum) for a split
  return attn_bars_off<KT>(nq, chunks, stages) + 8u * (2u * stages + 8u) + 16u + kRows * 8u + 1024u;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Warps 0 - 3: loads, products, two idle ones (the registers of a warpgroup
// can be moved only together); then four warps per row tile.
constexpr int kFirstRowWarp = 4;
constexpr __host__ __device__ int attn_threads(int nq) { return 32 * kFirstRowWarp + 128 * nq; }
// 168 registers a thread at launch with 384 threads; the row warps' tile of
// scores wants more: 88 * 128 + 208 * 256 = 168 * 384.
constexpr int kRegsFew = 88, kRegsMany = 208;
static_assert(kRegsFew * 128 + kRegsMany * 256 <= 168 * 384, "an increase past the launch's registers waits forever");

// A row's scores of a key tile, all of them in registers on return.
__device__ __forceinline__ void tmem_ld_all128(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
        "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
        "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]),
        "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]),
        "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]),
        "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]),
        "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]),
        "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]),
        "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]),
        "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]),
        "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]),
        "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]),
        "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]),
        "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]),
        "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]),
        "=r"(r[127])
      : "r"(taddr + 0), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_all64(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
        "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
        "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]),
        "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]),
        "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr + 0), "r"(taddr + 32)
      : "memory");
}
template <int NQ, int KT>
__global__ void __launch_bounds__(attn_threads(NQ), 1)
    attn_kernel(const __grid_constant__ CUtensorMap map_q,
                const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const AttnArgs p) {
  constexpr uint32_t kSlot = KT * 128u;  // 64 channels of a key tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const CacheShape &cs = p.c;
  const int chunks = p.chunks, stages = p.stages, split = NQ == 1 ? p.split : 1;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + attn_bars_off<KT>(NQ, chunks, stages));
  uint64_t *empty = full + stages;
  uint64_t *q_full = empty + stages;
  uint64_t *s_full = q_full + 1;   // [2]
  uint64_t *p_ready = s_full + 2;  // [2]
  uint64_t *pv_done = p_ready + 2;
  uint64_t *o_full = pv_done + 1;
  uint64_t *drain = o_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  float2 *row_ml = reinterpret_cast<float2 *>(tmem_slot + 2);  // [128] (split)

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;

  // the lengths may come from an earlier kernel of the stream
  griddep_wait();
  Item it;
  {
    int i = static_cast<int>(blockIdx.x) / split;
    it.kv_head = i % cs.kv_heads;
    i /= cs.kv_heads;
    it.seq = i % cs.n;
    // the last query tiles see the most keys: first
    it.tok0 = (p.q_tiles - 1 - i / cs.n) * (NQ * p.tok_tile);
    int chunk, all;
    lengths(cs, it.seq, chunk, all);
    it.live = chunk * cs.frame;
    it.base = all - chunk;
  }
  if (it.tok0 >= it.live) return;  // (the whole cluster)
  const int tok_end = min(it.tok0 + NQ * p.tok_tile, it.live);  // of this CTA
  const int qf0 = it.base + it.tok0 / cs.frame, qf1 = it.base + (tok_end - 1) / cs.frame;
  const int reach = p.window > 0 ? p.window - 1 : INT32_MAX;  // frames back
  auto back = [&](int qf) { return qf > reach ? qf - reach : 0; };
  // keys that some query of the CTA sees, and keys that all of them see
  const Ranges any = token_ranges(cs, back(qf0), qf1, qf1);
  const Ranges every = token_ranges(cs, back(qf1), qf0, qf0);
  const TileList<KT> tiles(any);
  const int j0 = static_cast<int>(static_cast<long long>(tiles.total) * rank / split);
  const int nj = static_cast<int>(static_cast<long long>(tiles.total) * (rank + 1) / split) - j0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);  // the warps of a row tile
    }
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t ring = smem_base + static_cast<uint32_t>(NQ * chunks) * kQChunk;
  // tensor memory: S (and P in its place) of slot 0 and 1, then O of each row tile
  const uint32_t s_col[2] = {tmem, tmem + KT};
  const uint32_t o_cols = static_cast<uint32_t>(chunks) * 64u;
  const uint32_t o_col = tmem + 2 * KT;
  griddep_launch_dependents();
  bool ok = true;

  // (in the branches: code after a common point gets the smaller share)
  if (warp == 0) {
    // ------------------------------ loads ---------------------------------------
    if constexpr (NQ == 2) regs_fewer<kRegsFew>();
    if (nj > 0 && elect_one()) {
      const int rows = p.tok_tile * p.group;
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(NQ * chunks * rows) * 128u);
      for (int q = 0; q < NQ; ++q)
        for (int c = 0; c < chunks; ++c)
          tma_load_4d(smem_base + static_cast<uint32_t>(q * chunks + c) * kQChunk, &map_q, q_full,
                      c * 64, it.kv_head * p.group, it.tok0 + q * p.tok_tile, it.seq);
      int s = 0;
      uint32_t ph = 0, used = 0, par = 0;
      auto load = [&](const CUtensorMap *map, int j) {
        const int tok = tiles.at(j0 + j) * KT;
#pragma unroll 1
        for (int c = 0; c < chunks && ok; ++c) {
          if (!mbar_wait_bounded(&empty[s], ph ^ 1, p.wait_limit_ns, p.status, 30)) {
            ok = false;
            return;
          }
          mbar_arrive_expect_tx(&full[s], kSlot);
          used |= 1u << s;
          par = (par & ~(1u << s)) | (ph << s);
          tma_load_4d(ring + s * kSlot, map, &full[s], c * 64, it.kv_head, tok, it.seq);
          if (++s == stages) { s = 0; ph ^= 1; }
        }
      };
      // in the order of their first use
      load(&map_k, 0);
      for (int j = 0; j < nj && ok; ++j) {
        if (NQ == 1 && j + 1 < nj) load(&map_k, j + 1);
        if (ok) load(&map_v, j);
        if (NQ == 2 && ok && j + 1 < nj) load(&map_k, j + 1);
      }
      mbar_wait_bounded(q_full, 0, kDrainNs, nullptr, 0);
      for (int i = 0; i < stages; ++i)
        if (used >> i & 1u) mbar_wait_bounded(&full[i], par >> i & 1u, kDrainNs, nullptr, 0);
    }
  } else if (warp == 1) {
    // ------------------------------ products ------------------------------------
    if constexpr (NQ == 2) regs_fewer<kRegsFew>();
    if (nj > 0 && elect_one()) {
      const uint32_t idesc_s = idesc_bf16_f32(kRows, KT);
      // O in steps of two chunks where they pair up in the ring
      const int wide = (chunks % 2 == 0 && stages % 2 == 0) ? 2 : 1;
      const uint32_t idesc_o = idesc_bf16_f32_bt(kRows, 64 * wide);
      const uint64_t qd = smem_desc_sw128(smem_base, 1024u);
      const uint64_t kd = smem_desc_sw128(ring, 1024u);
      const uint64_t vd = smem_desc_sw128_mn(ring, kSlot, 1024u);
      int s = 0;  // ring position of the next load to be consumed
      uint32_t ph = 0;
      auto step = [&](int &slot, uint32_t &phase) {
        if (++slot == stages) { slot = 0; phase ^= 1; }
      };
      auto fail = [&]() { ok = false; };
      // S[slot] = Q[q] K^T of the key tile at ring position (ks, kp)
      auto qk = [&](int q, int slot, int ks, uint32_t kp, bool wait, bool release) {
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          if (wait && !mbar_wait_bounded(&full[ks], kp, p.wait_limit_ns, p.status, 31))
            return fail();
          const uint64_t a = qd + ((static_cast<uint32_t>(q * chunks + c) * kQChunk) >> 4);
          const uint64_t b = kd + ((ks * kSlot) >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            umma_bf16(s_col[slot], a + 2 * i, b + 2 * i, idesc_s, c > 0 || i > 0);
          if (release) umma_commit(&empty[ks]);
          step(ks, kp);
        }
        umma_commit(&s_full[slot]);
      };
      // O[q] (+)= P[slot] V of the value tile at ring position (vs, vp)
      auto pv = [&](int q, int slot, int vs, uint32_t vp, bool wait, bool release, bool first) {
#pragma unroll 1
        for (int c = 0; c < chunks; c += wide) {
          int v2 = vs;
          uint32_t p2 = vp;
          for (int u = 0; u < wide; ++u) {
            if (wait && !mbar_wait_bounded(&full[v2], p2, p.wait_limit_ns, p.status, 32))
              return fail();
            step(v2, p2);
          }
          const uint64_t b = vd + ((vs * kSlot) >> 4);
          const uint32_t d = o_col + q * o_cols + c * 64;
#pragma unroll
          for (int i = 0; i < KT / 16; ++i)
            umma_bf16_ta(d, s_col[slot] + 8 * i, b + 128 * i, idesc_o, !first || i > 0);
          if (release) {
            umma_commit(&empty[vs]);
            if (wide == 2) umma_commit(&empty[vs + 1]);
          }
          vs = v2;
          vp = p2;
        }
      };
      auto wait_p = [&](int slot, uint32_t parity) {
        if (!mbar_wait_bounded(&p_ready[slot], parity, p.wait_limit_ns, p.status, 33)) {
          ok = false;
          return;
        }
        tc_fence_after();
      };
      auto advance = [&]() {
        s += chunks;
        while (s >= stages) {
          s -= stages;
          ph ^= 1;
        }
      };
      if (!mbar_wait_bounded(q_full, 0, p.wait_limit_ns, p.status, 34)) ok = false;
      if constexpr (NQ == 1) {
        if (ok) qk(0, 0, s, ph, true, true);
        advance();
        for (int j = 0; j < nj && ok; ++j) {
          if (j + 1 < nj) {
            qk(0, (j + 1) & 1, s, ph, true, true);
            advance();
            if (!ok) break;
          }
          wait_p(j & 1, (j >> 1) & 1);
          if (!ok) break;
          pv(0, j & 1, s, ph, true, true, j == 0);
          advance();
          if (!ok) break;
          umma_commit(pv_done);
        }
      } else {
        int vs = 0;  // the last value tile's position
        uint32_t vp = 0;
        for (int j = 0; j < nj && ok; ++j) {
          const int ks = s;
          const uint32_t kp = ph;
          advance();
          qk(0, 0, ks, kp, true, false);
          if (!ok) break;
          if (j > 0) {
            wait_p(1, (j - 1) & 1);
            if (!ok) break;
            pv(1, 1, vs, vp, false, true, j == 1);
          }
          qk(1, 1, ks, kp, false, true);
          wait_p(0, j & 1);
          if (!ok) break;
          vs = s;
          vp = ph;
          advance();
          pv(0, 0, vs, vp, true, false, j == 0);
        }
        if (ok) wait_p(1, (nj - 1) & 1);
        if (ok) pv(1, 1, vs, vp, false, true, nj == 1);
      }
      if (ok) umma_commit(o_full);
      umma_commit(drain);
      mbar_wait_bounded(drain, 0, kDrainNs, nullptr, 0);
    }
  } else if (warp >= kFirstRowWarp) {
    // ------------------------------ softmax, output ------------------------------
    if constexpr (NQ == 2) regs_more<kRegsMany>();
    const int wg = (warp - kFirstRowWarp) / 4;  // this warp's row tile
    const int quarter = warp % 4;   // the tensor-memory lanes it may read
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = quarter * 32 + lane;  // its row of the tile
    const int tok = it.tok0 + wg * p.tok_tile + r / p.group;
    const int head = it.kv_head * p.group + r % p.group;
    const bool live = r < p.tok_tile * p.group && tok < it.live;
    Ranges mine;
    {
      const int qf = it.base + tok / cs.frame;
      mine = live ? token_ranges(cs, back(qf), qf, qf) : token_ranges(cs, 0, -1, -1);
    }
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;  // the maximum that p is relative to, and sum of p
    for (int j = 0; j < nj; ++j) {
      const int slot = NQ == 2 ? wg : (j & 1);
      const uint32_t par = static_cast<uint32_t>(NQ == 2 ? j : (j >> 1)) & 1u;
      if (!mbar_wait_bounded(&s_full[slot], par, p.wait_limit_ns, p.status, 35)) {
        ok = false;
        break;
      }
      __syncwarp();
      tc_fence_after();
      const int t0 = tiles.at(j0 + j) * KT;
      const bool masked = !every.covers(t0, t0 + KT);
      const uint32_t sc = s_col[slot] + lanes;
      uint32_t raw[KT];
      float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto hide = [&](uint32_t *v, int tok0) {
        const uint32_t bits = mine.bits(tok0);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!(bits >> e & 1u)) v[e] = 0xff800000u;  // -inf
      };
      if constexpr (KT == 128) tmem_ld_all128(sc, raw); else tmem_ld_all64(sc, raw);
      if (masked) {
#pragma unroll
        for (int i = 0; i < KT; i += 32) hide(raw + i, t0 + i);
      }
#pragma unroll
      for (int e = 0; e < KT; e += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          top4[u] = max3(top4[u], __uint_as_float(raw[e + 2 * u]), __uint_as_float(raw[e + 2 * u + 1]));
      const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
      const bool grow = (fmaxf(top, m) - m) * c > kGrow;  // (false for a row that saw nothing)
      if (__any_sync(0xffffffffu, grow)) {
        const float m2 = grow ? fmaxf(top, m) : m;
        const float f = grow ? exp2_fast((m - m2) * c) : 1.f;
        m = m2;
        l *= f;
        if (j > 0) {
          if (NQ == 1) {
            // (with two row tiles S of this tile was issued after P V of the last)
            if (!mbar_wait_bounded(pv_done, static_cast<uint32_t>(j - 1) & 1u, p.wait_limit_ns,
                                   p.status, 36)) {
              ok = false;
              break;
            }
            __syncwarp();
            tc_fence_after();
          }
          const uint32_t o = o_col + wg * o_cols + lanes;
#pragma unroll 1
          for (uint32_t i = 0; i < o_cols; i += 32) {
            uint32_t v[32];
            tmem_ld16_nowait(o + i, v);
            tmem_ld16_nowait(o + i + 16, v + 16);
            tmem_wait_ld();
            tmem_regs_after_wait<32>(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
            tmem_st16(o + i, v);
            tmem_st16(o + i + 16, v + 16);
          }
        }
      }
      const float mc = m == -INFINITY ? 0.f : m * c;
      const uint64_t c2 = pair_of(c, c), mc2 = pair_of(-mc, -mc);
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) {
        uint32_t *v = raw + 32 * i;
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = unpair(
              pair_fma(pair_of(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2, mc2));
          const float a = exp2_fast(x.x), b = exp2_fast(x.y);
          sum[(e / 2) & 1] = pair_add(sum[(e / 2) & 1], pair_of(a, b));
          w[e / 2] = pack_bf16x2(a, b);
        }
        // (32 scores become 16 columns, always behind the scores read)
        tmem_st16(sc + 16 * i, w);
      }
      {
        const float2 x = unpair(pair_add(sum[0], sum[1]));
        l += x.x + x.y;
      }
      tmem_wait_st();
      if (wg == 0 && masked && !any.covers(t0, t0 + KT)) {
        // Values no query of the CTA sees may be anything (a slot never
        // written, a frame beyond the end): 0 times a NaN would reach the
        // sums, so their rows are cleared before the product reads them.
        const int pos = (NQ == 2 ? 2 * j + 1 : (j + 1 < nj ? j + 2 : nj) + j) * chunks;
        for (int ch = 0; ch < chunks; ++ch) {
          const int sl = (pos + ch) % stages;
          if (!mbar_wait_bounded(&full[sl], static_cast<uint32_t>((pos + ch) / stages) & 1u,
                                 p.wait_limit_ns, p.status, 37)) {
            ok = false;
            break;
          }
          if (r < KT && !any.has(t0 + r)) {
            uint4 *row = reinterpret_cast<uint4 *>(
                smem + static_cast<uint32_t>(NQ * chunks) * kQChunk + sl * kSlot + r * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) row[e] = make_uint4(0, 0, 0, 0);
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[slot]);
    }
    if (nj > 0 && ok) {
      ok = mbar_wait_bounded(o_full, 0, p.wait_limit_ns, p.status, 38);
      __syncwarp();
      tc_fence_after();
    }
    __nv_bfloat16 *out = p.o + static_cast<long long>(it.seq) * p.o_seq +
                         static_cast<long long>(tok) * p.o_tok +
                         static_cast<long long>(head) * p.o_head;
    if (split == 1 && ok) {
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const uint32_t o = o_col + wg * o_cols + lanes;
      for (int i = 0; i < cs.d; i += 16) {
        __syncwarp();
        uint32_t v[16];
        if (nj > 0) {
          tmem_ld16_nowait(o + i, v);
          tmem_wait_ld();
          tmem_regs_after_wait<16>(v);
        }
        // (a row that saw nothing gives zeros, whatever the accumulator holds)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          v[e] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(v[e]) * inv);
        if (live) {
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            if (i + h >= cs.d) break;
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(v[h]), __uint_as_float(v[h + 1]));
            w.y = pack_bf16x2(__uint_as_float(v[h + 2]), __uint_as_float(v[h + 3]));
            w.z = pack_bf16x2(__uint_as_float(v[h + 4]), __uint_as_float(v[h + 5]));
            w.w = pack_bf16x2(__uint_as_float(v[h + 6]), __uint_as_float(v[h + 7]));
            *reinterpret_cast<uint4 *>(out + i + h) = w;
          }
        }
      }
    }
    if (split > 1) row_ml[r] = make_float2(m, l);
  } else {
    if constexpr (NQ == 2) regs_fewer<kRegsFew>();
  }
  if constexpr (NQ == 1) {
    if (split > 1) {
      __syncwarp();
      cluster_sync();
      // Every rank scales its part by its share of the whole row, leaves it
      // in its shared memory (the keys are done with), and finishes the rows
      // rank, rank + split, ...
      const int pitch = cs.d + 4;  // floats: rows start in different banks
      float *part = reinterpret_cast<float *>(smem);
      if (warp >= kFirstRowWarp) {
        const int r = (warp % 4) * 32 + lane;
        const uint32_t ml = smem_u32(row_ml) + 8u * r;
        float top = -INFINITY;
        for (int k = 0; k < split; ++k)
          top = fmaxf(top, ld_cluster_f32x2(mapa_shared(ml, k)).x);
        float all = 0.f;
        for (int k = 0; k < split; ++k) {
          const float2 v = ld_cluster_f32x2(mapa_shared(ml, k));
          if (v.x != -INFINITY) all += v.y * exp2_fast((v.x - top) * p.scale_log2);
        }
        const float2 me = row_ml[r];
        float f = 0.f;
        if (me.x != -INFINITY && (all > 0.f || all != all))
          f = exp2_fast((me.x - top) * p.scale_log2) / all;
        const uint32_t o = o_col + (static_cast<uint32_t>((warp % 4) * 32) << 16);
        if (ok && nj > 0) {
          for (int i = 0; i < cs.d; i += 8) {
            __syncwarp();
            uint32_t v[16];
            tmem_ld16_nowait(o + (i & ~15), v);
            tmem_wait_ld();
            tmem_regs_after_wait<16>(v);
            float4 w[2];
            float *wf = reinterpret_cast<float *>(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = __uint_as_float((i & 8) ? v[8 + e] : v[e]);
              wf[e] = f == 0.f ? 0.f : x * f;
            }
            float4 *dst = reinterpret_cast<float4 *>(part + r * pitch + i);
            dst[0] = w[0];
            dst[1] = w[1];
          }
        } else {
          for (int i = 0; i < cs.d; i += 4)
            *reinterpret_cast<float4 *>(part + r * pitch + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      __syncwarp();
      cluster_sync();
      const int rows = min(kRows / p.group * p.group, (tok_end - it.tok0) * p.group);
      const int per = cs.d / 4;
      const int mine = (rows - rank + split - 1) / split;  // rows this rank finishes
      for (int x = threadIdx.x; x < mine * per; x += blockDim.x) {
        const int r = rank + x / per * split, i = (x % per) * 4;
        const uint32_t at = smem_base + static_cast<uint32_t>(r * pitch + i) * 4u;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < split; ++k) {
          const uint32_t from = mapa_shared(at, k);
          const float2 a = ld_cluster_f32x2(from), b = ld_cluster_f32x2(from + 8);
          sum.x += a.x;
          sum.y += a.y;
          sum.z += b.x;
          sum.w += b.y;
        }
        uint2 w;
        w.x = pack_bf16x2(sum.x, sum.y);
        w.y = pack_bf16x2(sum.z, sum.w);
        *reinterpret_cast<uint2 *>(p.o + static_cast<long long>(it.seq) * p.o_seq +
                                   static_cast<long long>(it.tok0 + r / p.group) * p.o_tok +
                                   static_cast<long long>(it.kv_head * p.group + r % p.group) *
                                       p.o_head +
                                   i) = w;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();  // (peers may still read this CTA's part)
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the cache update ----------------------------------------------------------------

// Frame p of a sequence goes to slot p (p < sinks, or no ring), else to slot
// sinks + (p - sinks) % ring.  A chunk longer than the ring leaves only its
// last `ring` frames there: the earlier ones are not written at all, so no
// two threads write one slot.
__global__ void __launch_bounds__(256)
    kv_append_kernel(const CacheShape c, const __nv_bfloat16 *k, const Strides sk,
                     const __nv_bfloat16 *v, const Strides sv, __nv_bfloat16 *kc,
                     const Strides skc, __nv_bfloat16 *vc, const Strides svc) {
  griddep_launch_dependents();
  griddep_wait();
  const int per = c.d / 8;  // 16-byte pieces of a head
  const long long total = static_cast<long long>(c.n) * c.t * c.frame * c.kv_heads * per;
  for (long long x = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * blockDim.x) {
    long long y = x;
    const int e = static_cast<int>(y % per) * 8;
    y /= per;
    const int h = static_cast<int>(y % c.kv_heads);
    y /= c.kv_heads;
    const int tok = static_cast<int>(y % (static_cast<long long>(c.t) * c.frame));
    const int seq = static_cast<int>(y / (static_cast<long long>(c.t) * c.frame));
    int all = c.k_frames ? c.k_frames[seq] : c.total;
    int chunk = c.q_frames ? c.q_frames[seq] : c.t;
    chunk = chunk < 0 ? 0 : (chunk > c.t ? c.t : chunk);
    const int f = tok / c.frame;
    if (f >= chunk) continue;
    const int p = all - chunk + f;
    if (p < 0) continue;
    int slot = p;
    if (c.ring > 0 && p >= c.sinks) {
      if (all - p > c.ring) continue;  // a later frame of the chunk takes the slot
      slot = c.sinks + (p - c.sinks) % c.ring;
    }
    if (slot >= c.slots) continue;
    const long long dst = static_cast<long long>(slot) * c.frame + tok % c.frame;
    const uint4 a = *reinterpret_cast<const uint4 *>(k + seq * sk.seq + tok * sk.tok + h * sk.head + e);
    const uint4 b = *reinterpret_cast<const uint4 *>(v + seq * sv.seq + tok * sv.tok + h * sv.head + e);
    *reinterpret_cast<uint4 *>(kc + seq * skc.seq + dst * skc.tok + h * skc.head + e) = a;
    *reinterpret_cast<uint4 *>(vc + seq * svc.seq + dst * svc.tok + h * svc.head + e) = b;
  }
}

// ---- launches ------------------------------------------------------------------------

using AttnKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                            const AttnArgs);

cudaError_t prepare_kernels() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev]) return cudaSuccess;
  const AttnKernel ks[3] = {attn_kernel<2, 128>, attn_kernel<1, 128>, attn_kernel<1, 64>};
  for (const AttnKernel k : ks) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(k),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemMost));
    if (e != cudaSuccess) return e;
  }
  done[dev] = true;
  return cudaSuccess;
}

bool encode_heads(CUtensorMap *m, const void *base, int d, int heads, long long tokens, int n,
                  const Strides &s, int box_heads, int box_tokens) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(tokens), static_cast<uint64_t>(n)};
  // (the distance of a single entry is free: a legal one)
  const uint64_t strides[3] = {static_cast<uint64_t>(heads > 1 ? s.head : 8) * 2,
                               static_cast<uint64_t>(tokens > 1 ? s.tok : 8) * 2,
                               static_cast<uint64_t>(n > 1 ? s.seq : 8) * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens),
                           1};
  return encode_sw128_map(m, base, 2, 4, dims, strides, box);
}

}  // namespace

cudaError_t launch_attention(AttnArgs a, const void *q, const Strides &sq, const void *k,
                             const Strides &sk, const void *v, const Strides &sv, int sm_count,
                             cudaStream_t stream) {
  cudaError_t e = prepare_kernels();
  if (e != cudaSuccess) return e;
  const CacheShape &c = a.c;
  a.group = a.heads / c.kv_heads;
  a.tok_tile = kRows / a.group;
  a.chunks = (c.d + 63) / 64;
  const long long tokens = static_cast<long long>(c.t) * c.frame;
  const long long tiles = (tokens + a.tok_tile - 1) / a.tok_tile;  // of 128 rows, per head
  const long long heads = static_cast<long long>(c.n) * c.kv_heads;
  // Two row tiles a CTA (a key tile read once for both, one's softmax under
  // the other's products) when that still gives every SM a CTA; their
  // accumulators fit up to d = 128.
  const bool two = c.d <= 128 && (tiles + 1) / 2 * heads >= sm_count / 2 && tiles > 1;
  const int kt = c.d <= 128 ? 128 : 64;
  const int nq = two ? 2 : 1;
  const long long q_tiles = (tiles + nq - 1) / nq;
  a.q_tiles = static_cast<int>(q_tiles);
  a.split = 1;
  if (!two) {
    // keys split over a cluster until every SM has a part of two tiles or more
    const long long seen = a.window > 0 ? static_cast<long long>(a.window) + c.t - 1 + c.sinks
                                        : c.slots;
    const long long keys = (seen < c.slots ? seen : c.slots) * c.frame;
    const long long key_tiles = (keys + kt - 1) / kt;
    while (a.split < 8 && (a.split + 1) * q_tiles * heads <= sm_count &&
           key_tiles >= 2 * (a.split + 1))
      ++a.split;
  }
  const long long grid = q_tiles * heads * a.split;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  auto smem = [&](int st) {
    return kt == 128 ? attn_smem<128>(nq, a.chunks, st) : attn_smem<64>(nq, a.chunks, st);
  };
  a.stages = 16;
  while (a.stages > 2 && smem(a.stages) > kSmemMost) a.stages -= 2;
  CUtensorMap mq, mk, mv;
  const long long cached = static_cast<long long>(c.slots) * c.frame;
  if (!encode_heads(&mq, q, c.d, a.heads, tokens, c.n, sq, a.group, a.tok_tile) ||
      !encode_heads(&mk, k, c.d, c.kv_heads, cached, c.n, sk, 1, kt) ||
      !encode_heads(&mv, v, c.d, c.kv_heads, cached, c.n, sv, 1, kt))
    return cudaErrorInvalidValue;
  const AttnKernel kern = two ? attn_kernel<2, 128>
                              : (kt == 128 ? attn_kernel<1, 128> : attn_kernel<1, 64>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.split);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(attn_threads(nq));
  cfg.dynamicSmemBytes = smem(a.stages);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, static_cast<const AttnArgs>(a));
  count_launch();
  return e;
}

cudaError_t launch_kv_append(const CacheShape &c, const __nv_bfloat16 *k, const Strides &sk,
                             const __nv_bfloat16 *v, const Strides &sv, __nv_bfloat16 *kc,
                             const Strides &skc, __nv_bfloat16 *vc, const Strides &svc,
                             int sm_count, cudaStream_t stream) {
  const long long total = static_cast<long long>(c.n) * c.t * c.frame * c.kv_heads * (c.d / 8);
  const long long need = (total + 255) / 256, most = static_cast<long long>(sm_count) * 8;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kv_append_kernel, c, k, sk, v, sv, kc, skc, vc, svc);
  count_launch();
  return e;
}

}  // namespace cc3d
