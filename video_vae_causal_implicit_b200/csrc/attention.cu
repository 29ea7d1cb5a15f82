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
// changes no rounding error (bf16 and fp32 are relative).  l sums the weights
// before their rounding.
//
// Keys are walked in the cache's own order, tile by tile; tiles no query of
// the CTA sees are skipped, tiles all of them see are not masked.  With few
// query rows a cluster of CTAs splits the keys, and the parts meet in
// distributed shared memory, added in rank order.
//
// Bound: the tensor pipe and the exponentials (16 a cycle and SM, as many
// cycles as the two products take at d = 128) for many rows, the cache's
// bytes for one token.  Measured (device time, twelve calls in a graph, one of
// several GPUs, whose clocks under load differ by 5 %): 8190 tokens, 16 heads on
// 4 of d = 128, window 2048 and 4 sinks 129 us (930 TFLOP/s; a step of 64 keys
// takes a CTA's 256 rows about 1670 cycles, of which the products want 1130 and
// the exponentials 1024); frames of 1560 tokens, d = 384, within themselves 32
// us for five; one token of 8 sequences, 32 heads on 8, over 8208 cached 47 us
// (5.7 TB/s).
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

constexpr int kRows = 128;                        // query rows of an MMA tile
constexpr uint32_t kQChunk = kRows * 128;         // 64 channels of them
constexpr size_t kSmemMost = 227 * 1024;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr float kGrow = 8.f;                      // log2 of the growth that p may take

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
__device__ __forceinline__ Ranges token_ranges(const CacheShape &c, const FastDiv &by_ring,
                                               int first, int last, int last_sink) {
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
        const int from = first - c.sinks;
        const int s0 = from - by_ring.quotient(from) * c.ring, e = s0 + count;
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
  // the tile at position j, `tile` being the one before
  __device__ __forceinline__ int after(int tile, int j) const {
    ++tile;
    if (j == count[0]) tile = count[1] > 0 ? start[1] : start[2];
    else if (j == count[0] + count[1]) tile = start[2];
    return tile;
  }
};

__device__ __forceinline__ void lengths(const CacheShape &c, int seq, int &chunk, int &all) {
  all = c.k_frames ? c.k_frames[seq] : c.total;
  if (all < 0) all = 0;
  if (c.ring == 0 && all > c.slots) all = c.slots;
  chunk = c.q_frames ? c.q_frames[seq] : c.t;
  chunk = chunk < 0 ? 0 : (chunk > c.t ? c.t : chunk);
}

// Shapes of a kernel: NQ row tiles of 128, key tiles of KT tokens, CH chunks
// of 64 channels.  Keys and values travel in groups of GC chunks, NG a tile,
// one barrier each: whole tiles where several fit beside Q, pairs of chunks for
// wide heads (a slot is then free, and its next load on its way, as soon as
// the products of one pair have read it; single chunks, with twice the
// barriers, took a quarter longer: five frames of 1560 tokens, d = 384).  P V
// runs in steps of PC chunks (N = 64 PC).
template <int NQ, int KT, int CH, int OCC>
struct Shape {
  static constexpr int GC = CH <= 2 ? CH : 2;
  static constexpr int NG = CH / GC;
  static constexpr int PC = CH <= 2 ? CH : 2;
  static constexpr uint32_t kChunk = KT * 128u;
  static constexpr uint32_t kGroup = GC * kChunk;
  static constexpr uint32_t kQ = NQ * CH * kQChunk;
  // Shared memory: Q, the ring of groups (after them, in a split, the parts
  // of the rows in their place), barriers, the rows' (maximum, sum).
  static constexpr uint32_t rest(int stages) {
    return 8u * (2u * stages + 6u + 6u * NQ) + 32u + NQ * kRows * 8u + 1024u;
  }
  static constexpr int stages() {
    int st = 24;
    // (whole steps of P V side by side)
    while (kQ + st * kGroup + rest(st) > kSmemMost / OCC - (OCC > 1 ? 1024 : 0) ||
           st % (PC / GC) != 0)
      --st;
    return st;
  }
  static constexpr int kStages = stages();
  static constexpr uint32_t kBars = kQ + kStages * kGroup;
  // (Of two CTAs an SM 112 KB at least: none then fits beside a kernel that
  // holds all of an SM's tensor memory, which takes 116 KB or more.  Otherwise
  // clusters of two kernels on two streams could each hold tensor memory that
  // the other's second CTA waits for.)
  static constexpr uint32_t kUsed = kBars + rest(kStages);
  static constexpr uint32_t kSmem = OCC > 1 && kUsed < 112 * 1024 ? 112 * 1024 : kUsed;
  static_assert(OCC == 1 || (kSmem + 1024) * OCC <= 228 * 1024, "CTAs of an SM");
  // tensor memory: two slots of scores and the output per row tile
  static constexpr uint32_t kTmemCols = 512 / OCC;
  static_assert(2 * NQ * KT + NQ * 64 * CH <= static_cast<int>(kTmemCols), "tensor memory columns");
  // a value tile, the key tile two ahead and the value tile before fit at once
  static_assert(kStages >= 3 * NG || (NQ == 1 && kStages >= 2 * NG), "ring depth");
  // the parts of a split: rows of d + 4 floats
  static_assert(NQ * kRows * (64 * CH + 4) * 4 <= kBars, "space for the parts of the rows");
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^x of a pair for x <= 8 or so by additions and products: x = n + f, |f| <=
// 1/2, 2^f by its minimax polynomial of degree 4 (fitted by Remez exchange,
// relative error 3e-6), times 2^n by its bits.  From -126.5 down 0, and NaN
// stays NaN (its product with anything is).
__device__ __forceinline__ float2 exp2_products(float2 v) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are n
  const uint64_t x = pair_of(max_nan(v.x, -127.f), max_nan(v.y, -127.f));
  const uint64_t r = pair_add(x, pair_of(kMagic, kMagic));
  const uint64_t f = pair_fma(pair_add(r, pair_of(-kMagic, -kMagic)), pair_of(-1.f, -1.f), x);
  uint64_t y = pair_of(0.00957010221f, 0.00957010221f);
  y = pair_fma(y, f, pair_of(0.0559178591f, 0.0559178591f));
  y = pair_fma(y, f, pair_of(0.240247443f, 0.240247443f));
  y = pair_fma(y, f, pair_of(0.693121791f, 0.693121791f));
  y = pair_fma(y, f, pair_of(0.999999285f, 0.999999285f));
  const float2 n = unpair(r);
  return unpair(pair_mul(
      y, pair_of(__uint_as_float((__float_as_uint(n.x) << 23) + 0x3f800000u),
                 __uint_as_float((__float_as_uint(n.y) << 23) + 0x3f800000u))));
}

// Warps 0 - 3: loads, products (two), values behind a mask; then four warps per
// row tile.
constexpr int kFirstRowWarp = 4;
constexpr __host__ __device__ int attn_threads(int nq) { return 32 * kFirstRowWarp + 128 * nq; }
// 168 registers a thread at launch with 384 threads; the row warps' tile of
// scores wants more.
constexpr int kRegsFew = 152, kRegsMany = 176;
static_assert(kRegsFew * 128 + kRegsMany * 256 <= 168 * 384,
              "an increase past the launch's registers waits forever");

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
// The rows rank, rank + split, ... of a split's `rows`: a warp takes 8 / KS
// rows at a time (KS >= split), a lane four channels of each piece of 128, and
// every rank's part is on its way before the first is added, in rank order.
template <int KS, int PIECES>
__device__ __forceinline__ void finish_rows(const AttnArgs &p, int rank, int rows,
                                            uint32_t smem_base, int pitch, int seq, int kv_head,
                                            int tok0) {
  constexpr int kBatch = 8 / KS;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int warps = static_cast<int>(blockDim.x) / 32;
  const int tile_rows = p.tok_tile * p.group;  // used rows of a row tile
  const int step = p.split * warps;
  for (int row0 = rank + p.split * warp; row0 < rows; row0 += step * kBatch) {
    float4 v[kBatch][PIECES][KS];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = row0 + b * step;
      if (row >= rows) continue;
      const int r = row >= tile_rows ? row - tile_rows + kRows : row;  // (two row tiles at most)
      const uint32_t at = smem_base + static_cast<uint32_t>(r * pitch + 4 * lane) * 4u;
#pragma unroll
      for (int c = 0; c < PIECES; ++c)
        if (c * 128 + 4 * lane < p.c.d) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
            if (k < p.split) v[b][c][k] = ld_cluster_f32x4(mapa_shared(at + c * 512u, k));
        }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = row0 + b * step;
      if (row >= rows) continue;
      const int tk = p.by_group.quotient(row);
      __nv_bfloat16 *out = p.o + static_cast<long long>(seq) * p.o_seq +
                           static_cast<long long>(tok0 + tk) * p.o_tok +
                           static_cast<long long>(kv_head * p.group + row - tk * p.group) *
                               p.o_head;
#pragma unroll
      for (int c = 0; c < PIECES; ++c)
        if (c * 128 + 4 * lane < p.c.d) {
          float4 sum = v[b][c][0];
#pragma unroll
          for (int k = 1; k < KS; ++k)
            if (k < p.split) {
              sum.x += v[b][c][k].x;
              sum.y += v[b][c][k].y;
              sum.z += v[b][c][k].z;
              sum.w += v[b][c][k].w;
            }
          uint2 w;
          w.x = pack_bf16x2(sum.x, sum.y);
          w.y = pack_bf16x2(sum.z, sum.w);
          *reinterpret_cast<uint2 *>(out + c * 128 + 4 * lane) = w;
        }
    }
  }
}

// A bit per key of a tile.
template <int W>
struct Bits {
  uint32_t w[W];
  __device__ __forceinline__ bool any() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) m |= w[i];
    return m != 0;
  }
};

// Of the keys in `some` (bit i: key lane + 32 i of the value tile in the ring's
// groups s, s + 1, ...) those with a value that is not finite; their values
// are cleared.  (A call, as is the other part: written into the kernel they
// cost one token's step over a long cache 3 to 5 of its 47 us.)
template <int KT, int GC, int NG>
__device__ __noinline__ uint32_t take_apart(uint8_t *ring, int s, int stages, uint32_t some) {
  constexpr uint32_t kChunk = KT * 128u;
  const int lane = threadIdx.x % 32;
  auto group = [&](int g) {
    return ring + (s + g < stages ? s + g : s + g - stages) * (GC * kChunk) + lane * 128;
  };
  uint32_t odd = 0;
#pragma unroll 1
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      if (!(some >> i & 1u)) continue;
      uint32_t top = 0;  // (exponents of ones carry into bits 15 and 31)
#pragma unroll
      for (int c = 0; c < GC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // (in an order that meets every bank once)
          const uint4 x = *reinterpret_cast<const uint4 *>(group(g) + c * kChunk + i * 4096 +
                                                           (((e + lane) & 7) << 4));
          top |= (x.x & 0x7f807f80u) + 0x00800080u;
          top |= (x.y & 0x7f807f80u) + 0x00800080u;
          top |= (x.z & 0x7f807f80u) + 0x00800080u;
          top |= (x.w & 0x7f807f80u) + 0x00800080u;
        }
      if (top & 0x80008000u) odd |= 1u << i;
    }
  if (odd) {
#pragma unroll 1
    for (int g = 0; g < NG; ++g)
#pragma unroll 1
      for (int i = 0; i < KT / 32; ++i)
        if (odd >> i & 1u)
          for (int c = 0; c < GC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4 *>(group(g) + c * kChunk + i * 4096 + e * 16) =
                  make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  return odd;
}

// O[row] += P[row][s] V[s] for the keys s that are taken apart, in the rows
// that see them.  v: the tile's first value in the cache; the columns of this
// warp's rows: o of O, sc of P (two weights a column).
template <int W>
__device__ __noinline__ void add_apart(const __nv_bfloat16 *v, long long v_tok, int d, uint32_t sc,
                                       uint32_t o, int o_cols, Bits<W> keys, Bits<W> seen,
                                       bool begin) {
#pragma unroll 1
  for (int i = 0; i < o_cols; i += 32) {
    uint32_t acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0u;
    if (!begin) {
      tmem_ld32_nowait(o + i, acc);
      tmem_wait_ld();
      tmem_regs_after_wait<32>(acc);
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
#pragma unroll 1
      for (uint32_t left = keys.w[w]; left; left &= left - 1) {  // (the same in every lane)
        const int s = __ffs(left) - 1;
        uint32_t two[1] = {tmem_ld1_nowait(sc + (32 * w + s) / 2)};
        tmem_wait_ld();
        tmem_regs_after_wait<1>(two);
        const float weight = __uint_as_float(s & 1 ? two[0] & 0xffff0000u : two[0] << 16);
        const __nv_bfloat16 *at = v + (32 * w + s) * v_tok + i;
        if (seen.w[w] >> s & 1u) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            if (i + e < d) {
              const uint4 x = *reinterpret_cast<const uint4 *>(at + e);
              const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float *a = reinterpret_cast<float *>(&acc[e + 2 * k]);
                a[0] = fmaf(weight, __uint_as_float(u[k] << 16), a[0]);
                a[1] = fmaf(weight, __uint_as_float(u[k] & 0xffff0000u), a[1]);
              }
            }
        }
        __syncwarp();
      }
    }
    tmem_st32(o + i, acc);
  }
  tmem_wait_st();
}

// NQ row tiles of 128, key tiles of KT tokens.  Every row tile has two slots
// for its scores, so that the scores of the next key tile are there when the
// softmax of one ends.
//
// Measured alone, M = 128 products with both operands in shared memory (Q K^T)
// take N / 2 + 44 cycles, with A in tensor memory (P V) N / 2 + 10, and
// alternating N / 2 each: the first kind loads its A under the second's
// product.  One thread cannot issue them that fast (a product costs it some 40
// cycles, a barrier's wait 40 to 130), so two warps do: one per row tile, or
// one per kind.
template <int NQ, int KT, int CH, int OCC>
__global__ void __launch_bounds__(attn_threads(NQ), OCC)
    attn_kernel(const __grid_constant__ CUtensorMap map_q,
                const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const AttnArgs p) {
  using S = Shape<NQ, KT, CH, OCC>;
  constexpr int GC = S::GC, NG = S::NG, stages = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const CacheShape &cs = p.c;
  const int split = p.split;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *empty = full + stages;
  uint64_t *q_full = empty + stages;
  uint64_t *s_full = q_full + 1;          // [NQ][2]
  uint64_t *p_ready = s_full + 2 * NQ;    // [NQ][2]
  uint64_t *pv_done = p_ready + 2 * NQ;   // [NQ][2]
  uint64_t *o_full = pv_done + 2 * NQ;
  uint64_t *drain = o_full + 1;           // [2]
  uint64_t *v_clean = drain + 2;
  uint64_t *v_taken = v_clean + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(v_taken + 1);
  uint32_t *apart = tmem_slot + 2;                              // [4] keys of a tile
  volatile int *o_begun = reinterpret_cast<int *>(apart + 4);   // [2]
  float2 *row_ml = reinterpret_cast<float2 *>(tmem_slot + 8);   // [NQ * 128] (split)

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NQ + 1);  // (each row tile's products, and warp 3)
    }
    mbar_init(q_full, 1);
    for (int i = 0; i < 2 * NQ; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);  // the warps of a row tile
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(o_full, NQ);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_init(v_clean, 1);
    mbar_init(v_taken, 4 * NQ);
    o_begun[0] = o_begun[1] = 0;
    fence_mbar_init();
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t ring = smem_base + S::kQ;
  // tensor memory: the slots of S (and P in its place), then O, per row tile
  auto s_col = [&](int q, int slot) { return tmem + static_cast<uint32_t>((2 * q + slot) * KT); };
  constexpr uint32_t o_cols = CH * 64u;
  const uint32_t o_col = tmem + 2 * NQ * KT;
  griddep_launch_dependents();
  // Earlier kernels of the stream may still write what is read here (the
  // lengths at once, the rest where it is loaded) or read what is written.
  if (cs.k_frames || cs.q_frames) griddep_wait();

  // What this CTA (or cluster) works on: query tokens tok0 .. tok_end - 1 of
  // one sequence and kv head.
  int kv_head, seq, tok0, tok_end, base;
  {
    int i = p.by_split.quotient(static_cast<int>(blockIdx.x));
    int up = p.by_kv.quotient(i);
    kv_head = i - up * cs.kv_heads;
    i = up;
    up = p.by_n.quotient(i);
    seq = i - up * cs.n;
    // the last query tiles see the most keys: first
    const int tile = p.tile0 + p.q_tiles - 1 - up;
    int chunk, all;
    lengths(cs, seq, chunk, all);
    base = all - chunk;  // frame of query token 0 (negative: sees nothing)
    tok_end = chunk * cs.frame;
    if (p.tiles_frame > 0) {  // tiles that end with their frame
      const int f = p.by_tiles_frame.quotient(tile);
      tok0 = f * cs.frame + (tile - f * p.tiles_frame) * (NQ * p.tok_tile);
      tok_end = min(tok_end, (f + 1) * cs.frame);
    } else {
      tok0 = tile * (NQ * p.tok_tile);
    }
    tok_end = min(tok_end, tok0 + NQ * p.tok_tile);  // (<= tok0: nothing to do)
  }
  const int reach = p.window > 0 ? p.window - 1 : INT32_MAX;  // frames back
  auto back = [&](int qf) { return qf > reach ? qf - reach : 0; };
  const int qf0 = base + p.by_frame.quotient(tok0);
  const int qf1 = tok_end > tok0 ? base + p.by_frame.quotient(tok_end - 1) : -1;
  // keys that some query of the CTA sees, and keys that all of them see
  const Ranges any = token_ranges(cs, p.by_ring, back(qf0), qf1, qf1);
  const Ranges every = token_ranges(cs, p.by_ring, back(qf1), qf1 < 0 ? -1 : qf0, qf1 < 0 ? -1 : qf0);
  const TileList<KT> tiles(any);
  // (at most 2^25 tiles of at most 8 ranks)
  const int j0 = p.by_split.quotient(tiles.total * rank);
  const int nj = p.by_split.quotient(tiles.total * (rank + 1)) - j0;
  bool ok = true;
  bool sees = false;  // (row warps) whether this thread's row sees any key

  // ------------------------------ loads ---------------------------------------
  auto load_role = [&]() {
    if (nj > 0 && elect_one()) {
      griddep_wait();
      const int rows = p.tok_tile * p.group;
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(NQ * CH * rows) * 128u);
      for (int q = 0; q < NQ; ++q)
        for (int c = 0; c < CH; ++c)
          tma_load_4d(smem_base + static_cast<uint32_t>(q * CH + c) * kQChunk, &map_q, q_full,
                      c * 64, kv_head * p.group, tok0 + q * p.tok_tile, seq);
      int s = 0;
      uint32_t ph = 0, used = 0, par = 0;
      auto load = [&](const CUtensorMap *map, int j) {
        const int tok = tiles.at(j0 + j) * KT;
#pragma unroll 1
        for (int g = 0; g < NG && ok; ++g) {
          if (!mbar_wait_soon(&empty[s], ph ^ 1, p.wait_limit_ns, p.status, 30)) {
            ok = false;
            return;
          }
          mbar_arrive_expect_tx(&full[s], S::kGroup);
          used |= 1u << s;
          par = (par & ~(1u << s)) | (ph << s);
#pragma unroll
          for (int c = 0; c < GC; ++c)
            tma_load_4d(ring + s * S::kGroup + c * S::kChunk, map, &full[s], (g * GC + c) * 64,
                        kv_head, tok, seq);
          if (++s == stages) { s = 0; ph ^= 1; }
        }
      };
      // in the order of their first use: K 0, K 1, V 0, K 2, V 1, ...
      load(&map_k, 0);
#pragma unroll 1
      for (int j = 0; j < nj && ok; ++j) {
        if (j + 1 < nj) load(&map_k, j + 1);
        if (ok) load(&map_v, j);
      }
      mbar_wait_bounded(q_full, 0, kDrainNs, nullptr, 0);
      for (int i = 0; i < stages; ++i)
        if (used >> i & 1u) mbar_wait_bounded(&full[i], par >> i & 1u, kDrainNs, nullptr, 0);
    }
  };
  // ------------------------------ products ------------------------------------
  auto product_role = [&]() {
    if (nj > 0 && elect_one()) {
      griddep_wait();  // (a wait's limit does not count the kernels before)
      constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, KT);
      constexpr uint32_t idesc_o = idesc_bf16_f32_bt(kRows, 64 * S::PC);
      const uint64_t qd = smem_desc_sw128(smem_base, 1024u);
      const uint64_t kd = smem_desc_sw128(ring, 1024u);
      const uint64_t vd = smem_desc_sw128_mn(ring, S::kChunk, 1024u);
      // ring position of the first group of a tile
      struct Pos {
        int slot;
        uint32_t phase;
      };
      auto next = [&](Pos x) {
        if (++x.slot == stages) { x.slot = 0; x.phase ^= 1; }
        return x;
      };
      auto advance = [&](Pos &x, int n) {
        x.slot += n * NG;
        if (x.slot >= stages) { x.slot -= stages; x.phase ^= 1; }
      };
      auto await = [&](uint64_t *bar, uint32_t parity, int site) {
        if (ok && !mbar_wait_soon(bar, parity, p.wait_limit_ns, p.status, site)) ok = false;
        return ok;
      };
      // S[q][slot] = Q[q] K^T, a group at a time as it arrives
      auto scores = [&](int q, int slot, Pos x) {
        const uint32_t col = s_col(q, slot);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (!await(&full[x.slot], x.phase, 31)) return;
          const uint64_t b = kd + ((x.slot * S::kGroup) >> 4);
#pragma unroll
          for (int i = 0; i < 4 * GC; ++i) {
            const int c = g * GC + i / 4, k = i % 4;
            umma_bf16(col, qd + ((static_cast<uint32_t>(q * CH + c) * kQChunk) >> 4) + 2 * k,
                      b + (((i / 4) * S::kChunk) >> 4) + 2 * k, idesc_s, g > 0 || i > 0);
          }
          umma_commit(&empty[x.slot]);
          x = next(x);
        }
        umma_commit(&s_full[2 * q + slot]);
      };
      // O[q] (+)= P[q][slot] V
      auto values = [&](int q, int slot, Pos x, bool first) {
        const uint32_t col = s_col(q, slot);
#pragma unroll
        for (int c = 0; c < CH; c += S::PC) {
          const int at = x.slot;
#pragma unroll
          for (int u = 0; u < S::PC / GC; ++u) {
            if (!await(&full[x.slot], x.phase, 32)) return;
            x = next(x);
          }
          const uint64_t b = vd + ((at * S::kGroup) >> 4);
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            umma_bf16_ta(o_col + q * o_cols + c * 64, col + 8 * k, b + 128 * k, idesc_o,
                         !first || k > 0);
#pragma unroll
          for (int u = 0; u < S::PC / GC; ++u) umma_commit(&empty[at + u]);
        }
        umma_commit(&pv_done[2 * q + slot]);
      };
      await(q_full, 0, 34);
      // the ring holds K 0, K 1, V 0, K 2, V 1, ...
      Pos k{0, 0}, v{0, 0};
      advance(v, nj > 1 ? 2 : 1);
      if (NQ == 2) {
        // each row tile's products from a warp of their own
        const int q = warp - 1;
        for (int j = 0; j < 2 && j < nj && ok; ++j) {
          scores(q, j, k);
          advance(k, 1 + j);  // (past V 0)
        }
#pragma unroll 1
        for (int j = 0; j < nj && ok; ++j) {
          if (!await(&p_ready[2 * q + (j & 1)], (j >> 1) & 1, 33)) break;
          tc_fence_after();
          values(q, j & 1, v, j == 0 && !o_begun[q]);
          advance(v, j + 2 < nj ? 2 : 1);
          if (j + 2 < nj && ok) {
            scores(q, j & 1, k);
            advance(k, 2);
          }
        }
      } else if (warp == 1) {
        // the two kinds of products from a warp each
#pragma unroll 1
        for (int j = 0; j < nj && ok; ++j) {
          if (j >= 2 && !await(&pv_done[j & 1], ((j >> 1) - 1) & 1, 39)) break;
          tc_fence_after();
          scores(0, j & 1, k);
          advance(k, j == 0 ? 1 : 2);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < nj && ok; ++j) {
          if (!await(&p_ready[j & 1], (j >> 1) & 1, 33)) break;
          tc_fence_after();
          values(0, j & 1, v, j == 0 && !o_begun[0]);
          advance(v, j + 2 < nj ? 2 : 1);
        }
      }
      if (ok && (NQ == 2 || warp == 2)) umma_commit(o_full);
      umma_commit(&drain[warp - 1]);
      mbar_wait_bounded(&drain[warp - 1], 0, kDrainNs, nullptr, 0);
    }
  };
  // ------------------------------ softmax, output ------------------------------
  auto row_role = [&]() {
    griddep_wait();
    const int wg = (warp - kFirstRowWarp) / 4;  // this warp's row tile
    const int quarter = warp % 4;               // the tensor-memory lanes it may read
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = quarter * 32 + lane;  // its row of the tile
    const int tok_r = p.by_group.quotient(r);
    const int tok = tok0 + wg * p.tok_tile + tok_r;
    const int head = kv_head * p.group + r - tok_r * p.group;
    const bool live = r < p.tok_tile * p.group && tok < tok_end;
    Ranges mine;
    {
      const int qf = live ? base + p.by_frame.quotient(tok) : -1;
      mine = token_ranges(cs, p.by_ring, back(qf), qf, qf);
      sees = mine.hi[0] > mine.lo[0] || mine.hi[1] > mine.lo[1] || mine.hi[2] > mine.lo[2];
    }
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;  // the maximum that p is relative to, and sum of p
    // (every lane waits; the warp goes on as one)
    auto await = [&](uint64_t *bar, uint32_t parity, int site) {
      return __all_sync(0xffffffffu,
                        mbar_wait_soon(bar, parity, p.wait_limit_ns, p.status, site)) != 0;
    };
    // With two row tiles their exponentials take turns: the unit that
    // computes them is then busy with one tile's while the other's scores are
    // read and its weights written (left alone, both tiles' warps fall into
    // step and idle it half the time).  Every warp passes every turn, after a
    // wait that ran out too, so no turn is waited for in vain.
    auto take_turn = [&]() {
      if constexpr (NQ == 2) named_barrier_sync(1 + wg, 256);
    };
    auto pass_turn = [&](int j) {
      if constexpr (NQ == 2)
        if (wg == 0 || j + 1 < nj) named_barrier_arrive(2 - wg, 256);
    };
    if (NQ == 2 && wg == 1 && nj > 0) named_barrier_arrive(1, 256);
    int tile = nj > 0 ? tiles.at(j0) : 0, n_masked = 0;
#pragma unroll 1
    for (int j = 0; j < nj; ++j, tile = tiles.after(tile, j0 + j)) {
      const int t0 = tile * KT;
      const bool masked = !every.covers(t0, t0 + KT);
      const int slot = j & 1;
      const uint32_t sc = s_col(wg, slot) + lanes;
      uint32_t raw[KT];
      if (ok) ok = await(&s_full[2 * wg + slot], static_cast<uint32_t>(j >> 1) & 1u, 35);
      if (ok) {
        tc_fence_after();
        if constexpr (KT == 128) tmem_ld_all128(sc, raw);
        else tmem_ld_all64(sc, raw);
        if (masked) {
#pragma unroll
          for (int i = 0; i < KT; i += 32) {
            const uint32_t bits = mine.bits(t0 + i);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1u)) raw[i + e] = 0xff800000u;  // -inf
          }
        }
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
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
            // (the products of the tile before still add to O)
            ok = await(&pv_done[2 * wg + ((j - 1) & 1)], static_cast<uint32_t>((j - 1) >> 1) & 1u,
                       36);
            tc_fence_after();
            const uint32_t o = o_col + wg * o_cols + lanes;
#pragma unroll 1
            for (uint32_t i = 0; i < o_cols; i += 32) {
              uint32_t v[32];
              tmem_ld32_nowait(o + i, v);
              tmem_wait_ld();
              tmem_regs_after_wait<32>(v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
              tmem_st32(o + i, v);
            }
          }
        }
      }
      take_turn();
      if (!ok) {
        pass_turn(j);
        continue;
      }
      const float mc = m == -INFINITY ? 0.f : m * c;
      const uint64_t c2 = pair_of(c, c), mc2 = pair_of(-mc, -mc);
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int i = 0; i < KT; i += 32) {
        uint32_t *w = raw + i / 2;  // (the weights take the scores' registers)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = unpair(pair_fma(
              pair_of(__uint_as_float(raw[i + e]), __uint_as_float(raw[i + e + 1])), c2, mc2));
          // With 128 keys a tile a warp has its scheduler to itself and waits
          // for the exponential's unit: three pairs of eight take the other way
          // (one token over a long cache 3 % faster, with four of eight 3 %
          // slower than with none.  With two row tiles the warps' instructions
          // bound: 8190 tokens take the same with none or one of eight, 4 % more
          // with two).
          const bool products = KT == 128 && (0x92 >> ((e / 2) % 8) & 1);
          const float2 y =
              products ? exp2_products(x) : make_float2(exp2_fast(x.x), exp2_fast(x.y));
          sum[(e / 2) & 1] = pair_add(sum[(e / 2) & 1], pair_of(y.x, y.y));
          w[e / 2] = pack_bf16x2(y.x, y.y);
        }
      }
      {
        const float2 x = unpair(pair_add(sum[0], sum[1]));
        l += x.x + x.y;
      }
      // (stores within the turn: 2 % slower at 8190 tokens)
      pass_turn(j);
#pragma unroll
      for (int i = 0; i < KT / 2; i += 16) tmem_st16(sc + i, raw + i);
      tmem_wait_st();
      if (masked) {
        ok = await(v_clean, static_cast<uint32_t>(n_masked++) & 1u, 37);
        if (!ok) continue;
        Bits<KT / 32> keys;
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) keys.w[i] = apart[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(v_taken);
        if (r < KT && !any.has(t0 + r)) {
          // (K 0, K 1, V 0, K 2, V 1, ... in the ring)
          int at = (((j + 1 < nj ? j + 2 : nj) + j) * NG) % stages;
#pragma unroll 1
          for (int g = 0; g < NG; ++g) {
            uint4 *row = reinterpret_cast<uint4 *>(smem + S::kQ + at * S::kGroup + r * 128);
            for (int u = 0; u < GC; ++u)
#pragma unroll
              for (int e = 0; e < 8; ++e) row[u * (S::kChunk / 16) + e] = make_uint4(0, 0, 0, 0);
            if (++at == stages) at = 0;
          }
        }
        fence_proxy_async_smem();
        if (keys.any()) {
          if (j > 0) {
            ok = await(&pv_done[2 * wg + (slot ^ 1)], static_cast<uint32_t>((j - 1) >> 1) & 1u, 40);
            if (!ok) continue;
            tc_fence_after();
          }
          Bits<KT / 32> seen;
#pragma unroll
          for (int i = 0; i < KT / 32; ++i) seen.w[i] = mine.bits(t0 + 32 * i);
          add_apart(p.v + seq * p.v_seq + t0 * p.v_tok + kv_head * p.v_head, p.v_tok, cs.d, sc,
                    o_col + wg * o_cols + lanes, static_cast<int>(o_cols), keys, seen, j == 0);
          if (j == 0 && lane == 0) o_begun[wg] = 1;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[2 * wg + slot]);
    }
    if (nj > 0 && ok) {
      ok = await(o_full, 0, 38);
      tc_fence_after();
    }
    if (split == 1 && ok) {
      // 64 channels of the warp's 32 rows at a time through shared memory (Q's,
      // which every product has read), so that eight lanes store a row's 128
      // bytes.
      __nv_bfloat16 *out = p.o + static_cast<long long>(seq) * p.o_seq +
                           static_cast<long long>(tok) * p.o_tok +
                           static_cast<long long>(head) * p.o_head;
      // (a row that sees scores of -inf alone has the sum 0 and gives NaN)
      const float inv = sees ? 1.f / l : 0.f;
      const uint32_t o = o_col + wg * o_cols + lanes;
      uint8_t *stage = smem + static_cast<uint32_t>(wg * CH) * kQChunk + quarter * 4096u;
#pragma unroll 1
      for (int i = 0; i < cs.d; i += 64) {
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
          uint32_t v[32];
          if (nj > 0) {
            tmem_ld32_nowait(o + i + h, v);
            tmem_wait_ld();
            tmem_regs_after_wait<32>(v);
          }
          // (a row that saw nothing gives zeros, whatever the accumulator holds)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            v[e] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(v[e]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(v[8 * e]), __uint_as_float(v[8 * e + 1]));
            w.y = pack_bf16x2(__uint_as_float(v[8 * e + 2]), __uint_as_float(v[8 * e + 3]));
            w.z = pack_bf16x2(__uint_as_float(v[8 * e + 4]), __uint_as_float(v[8 * e + 5]));
            w.w = pack_bf16x2(__uint_as_float(v[8 * e + 6]), __uint_as_float(v[8 * e + 7]));
            *reinterpret_cast<uint4 *>(stage + lane * 128 + (((h / 8 + e) ^ (lane & 7)) << 4)) = w;
          }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int from = 4 * u + lane / 8, piece = lane % 8;  // row of the warp, 16 bytes of it
          const unsigned long long at = __shfl_sync(
              0xffffffffu, live ? reinterpret_cast<unsigned long long>(out) : 0ull, from);
          if (at != 0 && i + 8 * piece < cs.d)
            *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(at) + i + 8 * piece) =
                *reinterpret_cast<const uint4 *>(stage + from * 128 + ((piece ^ (from & 7)) << 4));
        }
        __syncwarp();
      }
    }
    if (split > 1) row_ml[wg * kRows + r] = make_float2(m, l);
  };
  // ------------------------------ values behind a mask --------------------------
  auto mask_role = [&]() {
    // A weight of 0 times an infinity or a NaN would reach the sums.  So in the
    // tiles that a mask cuts, keys' values that are not finite where only some
    // queries see them are cleared before the products read them, and the rows
    // that do see them add them apart.  Values no query of the CTA sees (they
    // may be anything: a slot never written, a frame beyond the end) are
    // cleared by the row warps once this warp says that they have landed: it
    // passes every group of the ring, so that no barrier runs ahead of it.
    griddep_wait();
    constexpr int kMine = KT / 32;  // keys of a lane: lane, lane + 32, ...
    int s = 0;
    uint32_t ph = 0, n_masked = 0;
    auto landed = [&](int n) {  // the ring's next n groups
      int at = s;
      uint32_t par = ph;
      for (int g = 0; g < n && ok; ++g) {
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&full[at], par, p.wait_limit_ns, p.status,
                                                    42)) != 0;
        if (++at == stages) { at = 0; par ^= 1; }
      }
      return ok;
    };
    auto pass = [&](int n) {
      __syncwarp();
      for (int g = 0; g < n; ++g) {
        if (lane == 0) mbar_arrive(&empty[s]);
        if (++s == stages) { s = 0; ph ^= 1; }
      }
    };
    int tile = nj > 0 ? tiles.at(j0) : 0;
    if (nj > 0 && landed(NG)) pass(NG);  // K 0, K 1, V 0, K 2, V 1, ...
#pragma unroll 1
    for (int j = 0; j < nj && ok; ++j, tile = tiles.after(tile, j0 + j)) {
      if (j + 1 < nj) {
        if (!landed(NG)) break;
        pass(NG);
      }
      if (!landed(NG)) break;
      const int t0 = tile * KT;
      if (every.covers(t0, t0 + KT)) {
        pass(NG);
        continue;
      }
      uint32_t some = 0;  // bit i: key lane + 32 i
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = t0 + 32 * i + lane;
        if (any.has(t) && !every.has(t)) some |= 1u << i;
      }
      uint32_t odd = 0;
      if (__any_sync(0xffffffffu, some))
        odd = take_apart<KT, GC, NG>(smem + S::kQ, s, stages, some);
      // (the tile before's have been read)
      if (n_masked > 0)
        ok = __all_sync(0xffffffffu, mbar_wait_soon(v_taken, (n_masked - 1) & 1u, p.wait_limit_ns,
                                                    p.status, 43)) != 0;
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const uint32_t bits = __ballot_sync(0xffffffffu, odd >> i & 1u);
        if (lane == 0) apart[i] = bits;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(v_clean);
      ++n_masked;
      pass(NG);
    }
  };
  // Registers move between the warpgroups in their branches (code after a common
  // point gets the smaller share); all warps of one execute the same instruction.
  if constexpr (NQ == 2) {
    if (warp >= kFirstRowWarp) {
      regs_more<kRegsMany>();
      row_role();
    } else {
      regs_fewer<kRegsFew>();
      if (warp == 0) load_role();
      else if (warp <= 2) product_role();
      else mask_role();
    }
  } else if (warp == 0) {
    load_role();
  } else if (warp <= 2) {
    product_role();
  } else if (warp >= kFirstRowWarp) {
    row_role();
  } else {
    mask_role();
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    // Every rank scales its part by its share of the whole row, leaves it in
    // its shared memory (the keys are done with), and finishes the rows rank,
    // rank + split, ...
    const int pitch = cs.d + 4;  // floats: rows start in different banks
    float *part = reinterpret_cast<float *>(smem);
    const int tile_rows = p.tok_tile * p.group;  // used rows of a row tile
    if (warp >= kFirstRowWarp) {
      const int wg = (warp - kFirstRowWarp) / 4;
      const int r = (warp % 4) * 32 + lane;
      const uint32_t ml = smem_u32(row_ml) + 8u * (wg * kRows + r);
      float2 of[8];  // every rank's (maximum, sum)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < split) of[k] = ld_cluster_f32x2(mapa_shared(ml, k));
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < split) top = fmaxf(top, of[k].x);
      // A rank has nothing of the row where its sum is 0.  (A maximum of -inf
      // does not say so: maxima pass over NaN, so it is that of a rank whose
      // scores are all NaN too; its sum is NaN then, and so is the row.)  Where
      // all ranks' sums are 0 the row sees nothing, or scores of -inf alone,
      // which give NaN.
      float all = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < split && of[k].y != 0.f)
          all += of[k].y * exp2_fast((of[k].x - top) * p.scale_log2);
      const float2 me = row_ml[wg * kRows + r];
      const bool part_of = me.y != 0.f || (sees && all == 0.f);
      const float f = part_of ? exp2_fast((me.x - top) * p.scale_log2) / all : 0.f;
      const uint32_t o = o_col + wg * o_cols + (static_cast<uint32_t>((warp % 4) * 32) << 16);
      const bool have = ok && nj > 0;  // (the same in every lane)
      const bool some = have && part_of;
      float *dst = part + (wg * kRows + r) * pitch;
#pragma unroll 1
      for (int i = 0; i < cs.d; i += 32) {
        __syncwarp();
        uint32_t v[32];
        if (have) {
          tmem_ld32_nowait(o + i, v);
          tmem_wait_ld();
          tmem_regs_after_wait<32>(v);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          v[e] = some ? __float_as_uint(__uint_as_float(v[e]) * f) : 0u;
        if (r < tile_rows) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            if (i + e < cs.d)
              *reinterpret_cast<uint4 *>(dst + i + e) =
                  make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
    __syncwarp();
    cluster_sync();
    griddep_wait();
    const int rows = max(0, tok_end - tok0) * p.group;  // of all row tiles
    if (split <= 2) finish_rows<2, (CH + 1) / 2>(p, rank, rows, smem_base, pitch, seq, kv_head, tok0);
    else if (split <= 4) finish_rows<4, (CH + 1) / 2>(p, rank, rows, smem_base, pitch, seq, kv_head, tok0);
    else finish_rows<8, (CH + 1) / 2>(p, rank, rows, smem_base, pitch, seq, kv_head, tok0);
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();  // (peers may still read this CTA's part)
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
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
    const int all = max(0, c.k_frames ? c.k_frames[seq] : c.total);
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

// The kernels: head sizes (d_above, d_most] in whole chunks of 64 channels,
// zero-padded; `step`: cycles of a key tile, measured in the loop.
struct Variant {
  AttnKernel kernel;
  int nq, kt, occ, d_above, d_most, threads;
  uint32_t smem;
  double step;
};
constexpr int kVariants = kAttnKernels;
template <int NQ, int KT, int CH, int OCC>
Variant variant(int d_above, double step) {
  return Variant{attn_kernel<NQ, KT, CH, OCC>, NQ, KT, OCC, d_above, 64 * CH,
                 attn_threads(NQ), Shape<NQ, KT, CH, OCC>::kSmem, step};
}
const Variant (&variants())[kVariants] {
  static const Variant v[kVariants] = {
      variant<2, 64, 1, 1>(0, 1700.0),  variant<2, 64, 2, 1>(64, 1780.0),
      variant<1, 64, 1, 2>(0, 1750.0),  variant<1, 64, 2, 2>(64, 1850.0),
      variant<1, 128, 1, 1>(0, 2000.0), variant<1, 128, 2, 1>(64, 2100.0),
      variant<1, 64, 4, 1>(128, 1800.0), variant<1, 64, 6, 1>(256, 2400.0)};
  return v;
}

cudaLaunchConfig_t launch_config(const Variant &v, unsigned grid, int split,
                                 cudaLaunchAttribute *attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
  if (split > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(split);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(v.threads);
  cfg.dynamicSmemBytes = v.smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cfg;
}

// Per device: the kernels' shared-memory limit, and how many clusters of 1 to
// 8 CTAs of each kernel are resident at once.
struct Prepared {
  bool done;
  int fit[kVariants][9];
};
std::mutex g_prepare_mu;
Prepared g_prepared[64];

cudaError_t prepare_kernels(int sm_count, const Prepared **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_prepare_mu);
  Prepared &p = g_prepared[dev];
  if (!p.done) {
    for (int i = 0; i < kVariants; ++i) {
      const Variant &v = variants()[i];
      e = cudaFuncSetAttribute(reinterpret_cast<const void *>(v.kernel),
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(v.smem));
      if (e != cudaSuccess) return e;
      p.fit[i][1] = sm_count * v.occ;
      for (int split = 2; split <= 8; ++split) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg =
            launch_config(v, static_cast<unsigned>(split), split, attr, nullptr);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void *>(v.kernel), &cfg) !=
            cudaSuccess) {
          (void)cudaGetLastError();
          n = 0;
        }
        p.fit[i][split] = n;
      }
    }
    p.done = true;
  }
  *out = &p;
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
  return encode_rows_map(m, base, 2, 4, dims, strides, box);
}

}  // namespace

int choose_attention(const CacheShape &c, int heads, int window, int sm_count,
                     const int (*fits)[9], AttnLaunch *out) {
  const long long tok_tile = kRows / (heads / c.kv_heads);
  const long long tokens = static_cast<long long>(c.t) * c.frame;
  const long long groups = static_cast<long long>(c.n) * c.kv_heads;
  // frames that a query sees
  const long long seen = window > 0 ? static_cast<long long>(window) + c.sinks : c.slots;
  // Row tiles of a CTA, its query tokens, and the tiles of a chunk.  Tiles
  // that cross frames see the keys of all of their frames; tiles that end
  // with their frame leave rows unused: whichever reads fewer keys.
  auto tile_count = [&](int nq, int *per_frame) {
    const long long rows = static_cast<long long>(nq) * tok_tile;
    const long long across = (tokens + rows - 1) / rows;
    const long long within = (c.frame + rows - 1) / rows;
    const double cost_across = static_cast<double>(across) * (seen + (rows - 1.0) / c.frame);
    const double cost_within = static_cast<double>(c.t) * within * seen;
    if (c.t > 1 && cost_within < cost_across) {
      *per_frame = static_cast<int>(within);
      return c.t * within;
    }
    *per_frame = 0;
    return across;
  };
  // frames there are (an empty sequence still wants its zeros written)
  const long long have = c.k_frames || c.ring > 0 ? c.slots : c.total > 0 ? c.total : 1;
  // A launch: two row tiles a CTA (d <= 128: a key tile is read once for both,
  // and one's softmax runs under the other's products), one, or one and two
  // CTAs an SM; keys split over 1 to 8 CTAs of a cluster.
  struct Launch {
    const Variant *kernel;
    int split, per_frame;
    long long tiles;
    double time;
  };
  // key tiles of a query tile (its first frame's window and what its later
  // frames add)
  auto key_tiles = [&](const Variant &v, int per_frame) {
    const long long span =
        per_frame > 0 ? 1 : (static_cast<long long>(v.nq) * tok_tile - 1) / c.frame + 1;
    const long long frames = seen + (span < c.t ? span : c.t) - 1;
    const long long keys = (frames < have ? frames : have) * c.frame;
    return static_cast<double>((keys + v.kt - 1) / v.kt);
  };
  // Cycles that a key tile's steps, a CTA's start and end, and the joining of
  // the parts were measured to take (d = 64 to 384, 1 to 8190 queries, 500 to
  // 20000 keys), of `waves` whole waves of what fits at once.
  auto time_of = [&](const Variant &v, double steps, int split, double waves, double step) {
    const double join = split > 1 ? 3000.0 + 30.0 * v.nq * c.d : 0.0;
    return waves * (std::ceil(steps / split) * step + 7000.0 + 20.0 * c.d + join);
  };
  // The fastest single launch for all query tokens, or those from the first
  // `skip` on (skip > 0 with t = 1 only).
  auto fastest = [&](long long skip) {
    Launch best = {nullptr, 1, 0, 0, 1e300};
    for (const Variant &v : variants()) {
      if (c.d > v.d_most || c.d <= v.d_above) continue;
      const long long rows = static_cast<long long>(v.nq) * tok_tile;
      if (skip % rows != 0) continue;
      int per_frame = 0;
      const long long tiles = tile_count(v.nq, &per_frame) - skip / rows;
      if (tiles * groups > INT32_MAX / 8) continue;
      const double steps = key_tiles(v, per_frame);
      for (int split = 1; split <= 8 && split <= steps; ++split) {
        const int fit = fits[&v - variants()][split];
        if (fit < 1) continue;
        // (a few waves are whole ones; the last of many overlaps the others')
        const double parts = static_cast<double>(tiles * groups) / fit;
        const double waves = parts < 4.0 ? std::ceil(parts) : parts + 0.5;
        // (alone on its SM a CTA of a pair steps faster)
        const double step =
            v.occ == 2 && tiles * groups * split <= sm_count ? 0.85 * v.step : v.step;
        const double t = time_of(v, steps, split, waves, step);
        if (t < best.time) best = {&v, split, per_frame, tiles, t};
      }
    }
    return best;
  };
  Launch parts[2] = {fastest(0), {}};
  if (!parts[0].kernel) return 0;
  int n_parts = 1;
  // The queries of one frame, of which all see the same keys, may also go in
  // two launches: whole waves of full tiles, and what is left with more CTAs a
  // tile.  (A frame of 1560 tokens, 12 heads of 128, over 7 frames: 84 pairs of
  // row tiles are more than half of the SMs, and 12 of them nearly empty: 134
  // us in one launch, 120 in two; 24 heads 259 and 207; a frame of 6240, 4
  // heads, over 5 frames 410 and 360.)  Looked for where a call is long enough
  // to hide the search.
  if (c.t == 1 && parts[0].time > 80000.0) {
    // (a second launch costs some 4000 cycles; a gain of 3 % or less is within
    // the estimate's error)
    double least = 0.97 * parts[0].time - 4000.0;
    for (const Variant &v : variants()) {
      if (c.d > v.d_most || c.d <= v.d_above) continue;
      const long long rows = static_cast<long long>(v.nq) * tok_tile;
      const double steps = key_tiles(v, 0);
      for (int split = 1; split <= 8 && split <= steps; ++split) {
        const int fit = fits[&v - variants()][split];
        for (int waves = 1; waves <= 3; ++waves) {
          long long tiles = static_cast<long long>(waves) * fit / groups;
          if (tiles > tokens / rows) tiles = tokens / rows;
          if (tiles < 1 || tiles * rows >= tokens || tiles * groups > INT32_MAX / 8) continue;
          const double first = time_of(v, steps, split, waves, v.step);
          if (first >= least) break;
          const Launch rest = fastest(tiles * rows);
          if (rest.kernel && first + rest.time < least) {
            least = first + rest.time;
            parts[0] = {&v, split, 0, tiles, first};
            parts[1] = rest;
            n_parts = 2;
          }
        }
      }
    }
  }
  for (int i = 0; i < n_parts; ++i)
    out[i] = AttnLaunch{static_cast<int>(parts[i].kernel - variants()), parts[i].split,
                        parts[i].per_frame, parts[i].tiles};
  return n_parts;
}

cudaError_t launch_attention(AttnArgs a, const void *q, const Strides &sq, const void *k,
                             const Strides &sk, const void *v, const Strides &sv, int sm_count,
                             cudaStream_t stream) {
  const Prepared *prepared = nullptr;
  cudaError_t e = prepare_kernels(sm_count, &prepared);
  if (e != cudaSuccess) return e;
  const CacheShape &c = a.c;
  a.group = a.heads / c.kv_heads;
  a.tok_tile = kRows / a.group;
  const long long tokens = static_cast<long long>(c.t) * c.frame;
  const long long groups = static_cast<long long>(c.n) * c.kv_heads;
  AttnLaunch parts[2];
  const int n_parts = choose_attention(c, a.heads, a.window, sm_count, prepared->fit, parts);
  if (n_parts == 0) return cudaErrorNotSupported;  // (too many tiles for a grid)
  a.by_frame = FastDiv(static_cast<uint32_t>(c.frame));
  a.by_group = FastDiv(static_cast<uint32_t>(a.group));
  a.by_kv = FastDiv(static_cast<uint32_t>(c.kv_heads));
  a.by_n = FastDiv(static_cast<uint32_t>(c.n));
  a.by_ring = FastDiv(static_cast<uint32_t>(c.ring > 0 ? c.ring : 1));
  CUtensorMap mq;
  const long long cached = static_cast<long long>(c.slots) * c.frame;
  if (!encode_heads(&mq, q, c.d, a.heads, tokens, c.n, sq, a.group, a.tok_tile))
    return cudaErrorInvalidValue;
  long long first_row = 0;  // query tokens of the launch before
  for (int i = 0; i < n_parts; ++i) {
    const Variant &v0 = variants()[parts[i].kernel];
    const long long rows = static_cast<long long>(v0.nq) * a.tok_tile;
    a.q_tiles = static_cast<int>(parts[i].tiles);
    a.tile0 = static_cast<int>(first_row / rows);
    first_row = parts[i].tiles * rows;
    a.split = parts[i].split;
    a.tiles_frame = parts[i].per_frame;
    a.by_split = FastDiv(static_cast<uint32_t>(a.split));
    a.by_tiles_frame = FastDiv(static_cast<uint32_t>(a.tiles_frame > 0 ? a.tiles_frame : 1));
    const long long grid = parts[i].tiles * groups * a.split;
    if (grid > INT32_MAX) return cudaErrorNotSupported;
    CUtensorMap mk, mv;
    if (!encode_heads(&mk, k, c.d, c.kv_heads, cached, c.n, sk, 1, v0.kt) ||
        !encode_heads(&mv, v, c.d, c.kv_heads, cached, c.n, sv, 1, v0.kt))
      return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        launch_config(v0, static_cast<unsigned>(grid), a.split, attr, stream);
    e = cudaLaunchKernelEx(&cfg, v0.kernel, mq, mk, mv, static_cast<const AttnArgs>(a));
    if (e != cudaSuccess) return e;
    count_launch();
  }
  return cudaSuccess;
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
