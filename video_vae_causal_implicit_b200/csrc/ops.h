// ops.h -- the transformer operators' launchers and the small host helpers
// their entry points share (not part of the public interface).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "cc3d.h"

namespace cc3d {

inline bool aligned_to(const void *p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0;
}
inline bool ranges_meet(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
inline cc3d_status status_of(cudaError_t e) {
  return e == cudaSuccess ? CC3D_OK
         : e == cudaErrorMemoryAllocation ? CC3D_ERR_OOM
         : e == cudaErrorNotSupported     ? CC3D_ERR_UNSUPPORTED
                                          : CC3D_ERR_CUDA;
}

// Facts of the current device, looked up once per device: its SM count, and
// whether it is an sm_100 part.
struct DeviceInfo {
  int sm_count;
  bool sm100;
};
bool device_info(DeviceInfo *out);

// A tiled tensor map with `rank` dimensions of bf16 (esz 2) or byte (esz 1)
// elements, boxes of 128- or 64-byte rows with the swizzle of that length, and
// zero fill out of bounds.  strides: bytes of dimensions 1 .. rank - 1.
bool encode_rows_map(CUtensorMap *m, const void *base, int esz, int rank, const uint64_t *dims,
                      const uint64_t *strides, const uint32_t *box);

struct AddNormArgs {
  const __nv_bfloat16 *x, *residual;  // [rows][c]; residual nullable
  const float *gamma, *beta;          // [c]; beta nullable
  __nv_bfloat16 *h, *y;               // [rows][c], nullable
  uint8_t *q;                         // [rows][c] E4M3, nullable
  float *scales;                      // [rows], nullable: one scale per row
  float q_scale;                      // the given scale where `scales` is null
  float eps;
  long long rows;
  int c, silu;
};
// (ordinary loads for everything a call reads: a read-only load may not
// see what an earlier, overlapped kernel of the stream wrote)
cudaError_t launch_add_rms_norm(const AddNormArgs &a, int sm_count, cudaStream_t stream);

// x / d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery,
// "Division by invariant integers using multiplication"): with l = ceil(log2
// d) and mul = floor(2^32 (2^l - d) / d) + 1 the quotient is (x + (x mul >> 32)) >> l.
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), mul(1), shift(0) {
    while ((1ull << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int quotient(int x) const {
    return static_cast<int>((static_cast<uint32_t>(x) + __umulhi(static_cast<uint32_t>(x), mul)) >>
                            shift);
  }
#endif
};

struct LinearArgs {
  const float *x_scales, *w_scales;  // FP8: [m] (nullable) and [n]
  const float *bias;                 // [n], nullable
  const __nv_bfloat16 *residual;     // [m][ldr], nullable
  __nv_bfloat16 *y;                  // [m][ldy]
  long long ldy, ldr;
  float x_scale;                     // FP8: where x_scales is null
  int m, n, k, act;
  int *status;
  unsigned long long wait_limit_ns;
  // set by launch_linear: the tile and ring, and the walk over the tiles
  int nt, stages, split, m_tiles, n_tiles;
  FastDiv by_band, by_last;
};
// x [m][ldx] and w [n][ldw]: bf16, or E4M3 bytes (fp8).
cudaError_t launch_linear(LinearArgs a, const void *x, long long ldx, const void *w,
                          long long ldw, bool fp8, int sm_count, cudaStream_t stream);

// What a call launches: the many-row kernel with tiles of nt columns (on CTA
// pairs or not), or the few-row kernel with nt tokens and K split over `split`
// CTAs.  pairs: CTA pairs of the former, clusters[nt / 16][split]: clusters of
// the latter that are resident at once.
struct LinearChoice {
  bool split_kernel;
  int pair, nt, stages, split;
};
LinearChoice choose_linear(int m, int n, int k, int act, bool fp8, int sm_count, int pairs,
                           const int (*clusters)[9]);

// Which frame of a sequence a cache slot holds: slot s < sinks frame s; the
// later slots frame s (ring 0), or cyclically the last `ring` frames.
struct CacheShape {
  int n, kv_heads, d, frame, slots, sinks, ring;
  int t;                           // frames of the call's chunk
  int total;                       // frames of every sequence, the chunk included, ...
  const int *q_frames, *k_frames;  // ... or per sequence: chunk frames, all frames (nullable)
};

struct AttnArgs {
  CacheShape c;
  int heads, window;       // window: frames, 0 = unlimited
  float scale_log2;        // softmax scale * log2(e)
  __nv_bfloat16 *o;
  const __nv_bfloat16 *v;  // (read apart from the tiles where a value is not finite)
  long long o_seq, o_tok, o_head, v_seq, v_tok, v_head;
  int *status;
  unsigned long long wait_limit_ns;
  int group, tok_tile;     // query heads per kv head; tokens per 128 rows
  // set by launch_attention; tile0: the launch's first query tile; tiles_frame: query tiles of a frame, 0 where tiles
  // cross frames
  int split, q_tiles, tile0, tiles_frame;
  FastDiv by_frame, by_group, by_kv, by_n, by_split, by_ring, by_tiles_frame;
};
struct Strides {
  long long seq, tok, head;  // in elements
};
cudaError_t launch_attention(AttnArgs a, const void *q, const Strides &sq, const void *k,
                             const Strides &sk, const void *v, const Strides &sv, int sm_count,
                             cudaStream_t stream);
// What a call launches: the kernel (by its place in the list of them), the CTAs
// that share a query tile's keys, query tiles of a frame (0: tiles cross
// frames) and of the launch.  Returns the number of launches (1 or 2; 0: too
// many tiles for a grid).  fits[kernel][split]: clusters of that many CTAs that
// are resident at once.
constexpr int kAttnKernels = 8;
struct AttnLaunch {
  int kernel, split, per_frame;
  long long tiles;
};
int choose_attention(const CacheShape &c, int heads, int window, int sm_count,
                     const int (*fits)[9], AttnLaunch *out);
cudaError_t launch_kv_append(const CacheShape &c, const __nv_bfloat16 *k, const Strides &sk,
                             const __nv_bfloat16 *v, const Strides &sv, __nv_bfloat16 *kc,
                             const Strides &skc, __nv_bfloat16 *vc, const Strides &svc,
                             int sm_count, cudaStream_t stream);

}  // namespace cc3d
