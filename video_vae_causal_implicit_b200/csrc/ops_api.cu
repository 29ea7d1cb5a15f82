// ops_api.cu -- entry points of the transformer operators (declared in
// include/cc3d.h): argument checks, tensor maps and launches.  Every check
// runs on the host before anything is launched.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "cc3d.h"
#include "internal.h"
#include "ops.h"

namespace cc3d {

bool device_info(DeviceInfo *out) {
  static std::mutex mu;
  static DeviceInfo known[64];
  static bool have[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lk(mu);
  if (!have[dev]) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return false;
    known[dev].sm100 = major == 10 && minor == 0;
    known[dev].sm_count = sms;
    have[dev] = true;
  }
  *out = known[dev];
  return true;
}

bool encode_rows_map(CUtensorMap *m, const void *base, int esz, int rank, const uint64_t *dims,
                      const uint64_t *strides, const uint32_t *box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn || rank < 2 || rank > 5) return false;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i > 0) s[i - 1] = strides[i - 1];
  }
  return fn(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, s, b, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            box[0] * static_cast<uint32_t>(esz) == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// Elements from the first to the last of a [n][tok][head][d] view, plus one.
long long span(int n, long long toks, int heads, int d, const Strides &s) {
  return (n - 1) * s.seq + (toks - 1) * s.tok + (heads - 1) * s.head + d;
}

// Strides that 16-byte pieces and a tensor map allow (only of dimensions with
// more than one entry; the others are not used).
bool strides_ok(int n, long long toks, int heads, const Strides &s) {
  const long long ext[3] = {n, toks, heads}, st[3] = {s.seq, s.tok, s.head};
  for (int i = 0; i < 3; ++i)
    if (ext[i] > 1 && (st[i] < 8 || st[i] % 8 != 0 || st[i] > (1ll << 38))) return false;
  return true;
}

// Whether no two entries of the view share an element: ordered by stride,
// each dimension steps over all of the smaller ones.  `apart` > 0: of two such
// views, that many elements from each other.
bool disjoint_entries(int n, long long toks, int heads, int d, const Strides &s,
                      long long apart = 0) {
  long long ext[4] = {n, toks, heads, apart > 0 ? 2 : 1}, st[4] = {s.seq, s.tok, s.head, apart};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3 - i; ++j)
      if (st[j] > st[j + 1]) {
        long long t = st[j];
        st[j] = st[j + 1];
        st[j + 1] = t;
        t = ext[j];
        ext[j] = ext[j + 1];
        ext[j + 1] = t;
      }
  long long covered = d;
  for (int i = 0; i < 4; ++i) {
    if (ext[i] == 1) continue;
    if (st[i] < covered) return false;
    covered = (ext[i] - 1) * st[i] + covered;
  }
  return true;
}

constexpr long long kMostTokens = (1ll << 31) - 1024;

// The checks that the cache's shape needs, shared by both calls.
cc3d_status check_cache(int n, int kv_heads, int d, int frame, int t, int slots, int sinks,
                        int ring, int total, const int *q_frames, const int *k_frames) {
  if (n < 0 || kv_heads < 1 || d < 1 || frame < 1 || t < 0 || slots < 1 || sinks < 0 || ring < 0)
    return CC3D_ERR_INVALID_ARG;
  if (ring > 0 && static_cast<long long>(sinks) + ring != slots) return CC3D_ERR_INVALID_ARG;
  if (!k_frames && (total < 0 || (ring == 0 && total > slots))) return CC3D_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > 384 || n > 65535 || kv_heads > 65535) return CC3D_ERR_UNSUPPORTED;
  if (static_cast<long long>(slots) * frame > kMostTokens ||
      static_cast<long long>(t) * frame > kMostTokens)
    return CC3D_ERR_UNSUPPORTED;
  if (!aligned_to(q_frames, 4) || !aligned_to(k_frames, 4)) return CC3D_ERR_ALIGNMENT;
  return CC3D_OK;
}

}  // namespace

}  // namespace cc3d

using namespace cc3d;

extern "C" {

cc3d_status cc3d_add_rms_norm(const cc3d_add_norm_call *p, void *stream) {
  if (!p) return CC3D_ERR_INVALID_ARG;
  const void *x = p->x, *residual = p->residual;
  const float *gamma = p->gamma, *beta = p->beta;
  void *h = p->h, *y = p->y, *q = p->q;
  float *scales = p->scales;
  const long long rows = p->rows;
  const int c = p->c;
  const float eps = p->eps, scale = p->scale;
  if (rows < 0 || c < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return CC3D_ERR_INVALID_ARG;
  if (rows == 0) return CC3D_OK;  // (such a call may come with null tensors)
  if (!x || !gamma || (!y && !q && !h)) return CC3D_ERR_INVALID_ARG;
  // 8 bits need exactly one kind of scale
  if (q ? (scales != nullptr) == (scale > 0.f && std::isfinite(scale)) : scales != nullptr)
    return CC3D_ERR_INVALID_ARG;
  if (q && !scales && (!(scale >= 1e-36f) || !std::isfinite(scale))) return CC3D_ERR_INVALID_ARG;
  if (c % 8 != 0 || c > 16384) return CC3D_ERR_UNSUPPORTED;
  if (rows > LLONG_MAX / 65536) return CC3D_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(residual, 16) || !aligned_to(h, 16) ||
      !aligned_to(y, 16) || !aligned_to(q, 8) || !aligned_to(gamma, 16) ||
      !aligned_to(beta, 16) || !aligned_to(scales, 4))
    return CC3D_ERR_ALIGNMENT;
  const size_t vals = static_cast<size_t>(rows) * c, full = vals * 2;
  const size_t sb = static_cast<size_t>(rows) * 4, pb = static_cast<size_t>(c) * 4;
  // h may be x or the residual itself (the stream updated in place), and so
  // may y: an element is read and written by one thread.  Nothing else meets.
  const void *in[2] = {x, residual};
  for (const void *i : in) {
    if ((h != i && ranges_meet(h, full, i, full)) || (y != i && ranges_meet(y, full, i, full)) ||
        ranges_meet(q, vals, i, full) || ranges_meet(scales, sb, i, full))
      return CC3D_ERR_ALIAS;
  }
  if (ranges_meet(h, full, y, full) || ranges_meet(h, full, q, vals) ||
      ranges_meet(y, full, q, vals) || ranges_meet(scales, sb, h, full) ||
      ranges_meet(scales, sb, y, full) || ranges_meet(scales, sb, q, vals))
    return CC3D_ERR_ALIAS;
  const float *par[2] = {gamma, beta};
  for (const float *g : par)
    if (ranges_meet(g, pb, h, full) || ranges_meet(g, pb, y, full) ||
        ranges_meet(g, pb, q, vals) || ranges_meet(g, pb, scales, sb))
      return CC3D_ERR_ALIAS;
  DeviceInfo dev;
  if (!device_info(&dev) || !dev.sm100) return CC3D_ERR_UNSUPPORTED;
  AddNormArgs a;
  a.x = static_cast<const __nv_bfloat16 *>(x);
  a.residual = static_cast<const __nv_bfloat16 *>(residual);
  a.gamma = gamma;
  a.beta = beta;
  a.h = static_cast<__nv_bfloat16 *>(h);
  a.y = static_cast<__nv_bfloat16 *>(y);
  a.q = static_cast<uint8_t *>(q);
  a.scales = scales;
  a.q_scale = scale;
  a.eps = eps;
  a.rows = rows;
  a.c = c;
  a.silu = p->silu != 0;
  return status_of(launch_add_rms_norm(a, dev.sm_count, static_cast<cudaStream_t>(stream)));
}

cc3d_status cc3d_linear(const cc3d_linear_call *p, void *stream) {
  if (!p) return CC3D_ERR_INVALID_ARG;
  const void *x = p->x, *weight = p->weight, *residual = p->residual;
  const float *bias = p->bias, *x_scales = p->x_scales, *w_scales = p->w_scales;
  void *y = p->y;
  const long long ldx = p->ldx, ldw = p->ldw, ldr = p->ldr, ldy = p->ldy, m = p->m;
  const int n = p->n, k = p->k;
  const cc3d_dtype dtype = p->dtype;
  const cc3d_act act = p->act;
  const float x_scale = p->x_scale;
  // (a call without rows may come with null tensors)
  if ((m != 0 && (!x || !weight || !y)) || m < 0 || n < 1 || k < 1 || ldx < k || ldw < k || ldy < n ||
      (residual && ldr < n) || act < CC3D_ACT_NONE || act > CC3D_ACT_GELU_TANH)
    return CC3D_ERR_INVALID_ARG;
  if (dtype != CC3D_BF16 && dtype != CC3D_FP8_E4M3) return CC3D_ERR_UNSUPPORTED;
  const bool fp8 = dtype == CC3D_FP8_E4M3;
  // (the scale that is not in use has to be 0, not only of no use)
  const bool one_scale = x_scale > 0.f && std::isfinite(x_scale);
  if (fp8 ? (!w_scales || (x_scales ? x_scale != 0.f : !one_scale))
          : (w_scales || x_scales || x_scale != 0.f))
    return CC3D_ERR_INVALID_ARG;
  const int step = fp8 ? 16 : 8;  // operand elements of 16 bytes
  constexpr long long kMost = 1ll << 30;
  if (k % step != 0 || ldx % step != 0 || ldw % step != 0 || n % 8 != 0 || ldy % 8 != 0 ||
      (residual && ldr % 8 != 0) || m > kMost || n > kMost || k > kMost || ldx > kMost ||
      ldw > kMost || ldy > kMost || (residual && ldr > kMost))
    return CC3D_ERR_UNSUPPORTED;
  if (!aligned_to(x, 16) || !aligned_to(weight, 16) || !aligned_to(y, 16) ||
      !aligned_to(residual, 16) || !aligned_to(bias, 16) || !aligned_to(w_scales, 16) ||
      !aligned_to(x_scales, 4))
    return CC3D_ERR_ALIGNMENT;
  if (m == 0) return CC3D_OK;
  const size_t esz = fp8 ? 1 : 2, rows = static_cast<size_t>(m), nn = static_cast<size_t>(n);
  const size_t xb = ((rows - 1) * ldx + k) * esz, wb = ((nn - 1) * ldw + k) * esz;
  const size_t yb = ((rows - 1) * ldy + nn) * 2, rb = residual ? ((rows - 1) * ldr + nn) * 2 : 0;
  // y may be the residual itself (the stream updated in place)
  const bool in_place = residual == y && ldr == ldy;
  if (ranges_meet(y, yb, x, xb) || ranges_meet(y, yb, weight, wb) ||
      ranges_meet(y, yb, bias, nn * 4) || ranges_meet(y, yb, w_scales, nn * 4) ||
      ranges_meet(y, yb, x_scales, rows * 4) || (!in_place && ranges_meet(y, yb, residual, rb)))
    return CC3D_ERR_ALIAS;
  DeviceInfo dev;
  if (!device_info(&dev) || !dev.sm100) return CC3D_ERR_UNSUPPORTED;
  LinearArgs a = {};
  a.x_scales = x_scales;
  a.w_scales = w_scales;
  a.bias = bias;
  a.residual = static_cast<const __nv_bfloat16 *>(residual);
  a.y = static_cast<__nv_bfloat16 *>(y);
  a.ldy = ldy;
  a.ldr = ldr;
  a.x_scale = x_scale;
  a.m = static_cast<int>(m);
  a.n = n;
  a.k = k;
  a.act = act;
  a.status = device_status_word();
  if (!a.status) return CC3D_ERR_CUDA;
  a.wait_limit_ns = wait_limit_ns();
  return status_of(launch_linear(a, x, ldx, weight, ldw, fp8, dev.sm_count,
                                 static_cast<cudaStream_t>(stream)));
}

cc3d_status cc3d_attention(const cc3d_attn_call *p, void *stream) {
  if (!p) return CC3D_ERR_INVALID_ARG;
  const cc3d_status s = check_cache(p->n, p->kv_heads, p->d, p->frame, p->t, p->slots, p->sinks,
                                    p->ring, p->total, p->q_frames, p->k_frames);
  if (s != CC3D_OK) return s;
  if (p->heads < 1 || p->heads % p->kv_heads != 0 || p->window < 0 || !(p->scale >= 0.f) ||
      !std::isfinite(p->scale))
    return CC3D_ERR_INVALID_ARG;
  // a ring has to hold every frame that a query of the chunk sees
  if (p->ring > 0 && (p->window == 0 || static_cast<long long>(p->window) - 1 + p->t > p->ring))
    return CC3D_ERR_INVALID_ARG;
  if (p->heads / p->kv_heads > 128) return CC3D_ERR_UNSUPPORTED;
  if (p->n == 0 || p->t == 0) return CC3D_OK;  // (such a call may come with null tensors)
  if (!p->q || !p->k || !p->v || !p->o) return CC3D_ERR_INVALID_ARG;
  const long long qt = static_cast<long long>(p->t) * p->frame;
  const long long kt = static_cast<long long>(p->slots) * p->frame;
  const Strides sq{p->q_seq, p->q_tok, p->q_head}, sk{p->k_seq, p->k_tok, p->k_head},
      sv{p->v_seq, p->v_tok, p->v_head}, so{p->o_seq, p->o_tok, p->o_head};
  if (!strides_ok(p->n, qt, p->heads, sq) || !strides_ok(p->n, kt, p->kv_heads, sk) ||
      !strides_ok(p->n, kt, p->kv_heads, sv) || !strides_ok(p->n, qt, p->heads, so))
    return CC3D_ERR_UNSUPPORTED;
  if (!aligned_to(p->q, 16) || !aligned_to(p->k, 16) || !aligned_to(p->v, 16) ||
      !aligned_to(p->o, 16))
    return CC3D_ERR_ALIGNMENT;
  if (!disjoint_entries(p->n, qt, p->heads, p->d, so)) return CC3D_ERR_ALIAS;
  const size_t ob = static_cast<size_t>(span(p->n, qt, p->heads, p->d, so)) * 2;
  if (ranges_meet(p->o, ob, p->q, static_cast<size_t>(span(p->n, qt, p->heads, p->d, sq)) * 2) ||
      ranges_meet(p->o, ob, p->k, static_cast<size_t>(span(p->n, kt, p->kv_heads, p->d, sk)) * 2) ||
      ranges_meet(p->o, ob, p->v, static_cast<size_t>(span(p->n, kt, p->kv_heads, p->d, sv)) * 2) ||
      ranges_meet(p->o, ob, p->q_frames, static_cast<size_t>(p->n) * 4) ||
      ranges_meet(p->o, ob, p->k_frames, static_cast<size_t>(p->n) * 4))
    return CC3D_ERR_ALIAS;
  DeviceInfo dev;
  if (!device_info(&dev) || !dev.sm100) return CC3D_ERR_UNSUPPORTED;
  AttnArgs a = {};
  a.c = CacheShape{p->n, p->kv_heads, p->d, p->frame, p->slots, p->sinks, p->ring, p->t, p->total,
                   p->q_frames, p->k_frames};
  a.heads = p->heads;
  a.window = p->window;
  const float scale = p->scale > 0.f ? p->scale : 1.f / sqrtf(static_cast<float>(p->d));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.o = static_cast<__nv_bfloat16 *>(p->o);
  a.v = static_cast<const __nv_bfloat16 *>(p->v);
  a.v_seq = p->v_seq;
  a.v_tok = p->v_tok;
  a.v_head = p->v_head;
  a.o_seq = p->o_seq;
  a.o_tok = p->o_tok;
  a.o_head = p->o_head;
  a.status = device_status_word();
  if (!a.status) return CC3D_ERR_CUDA;
  a.wait_limit_ns = wait_limit_ns();
  return status_of(launch_attention(a, p->q, sq, p->k, sk, p->v, sv, dev.sm_count,
                                    static_cast<cudaStream_t>(stream)));
}

cc3d_status cc3d_kv_append(const cc3d_kv_call *p, void *stream) {
  if (!p) return CC3D_ERR_INVALID_ARG;
  const cc3d_status s = check_cache(p->n, p->kv_heads, p->d, p->frame, p->t, p->slots, p->sinks,
                                    p->ring, p->total, p->q_frames, p->k_frames);
  if (s != CC3D_OK) return s;
  if (p->n == 0 || p->t == 0) return CC3D_OK;
  if (!p->k || !p->v || !p->k_cache || !p->v_cache) return CC3D_ERR_INVALID_ARG;
  const long long nt = static_cast<long long>(p->t) * p->frame;
  const long long ct = static_cast<long long>(p->slots) * p->frame;
  const Strides sk{p->k_seq, p->k_tok, p->k_head}, sv{p->v_seq, p->v_tok, p->v_head},
      skc{p->kc_seq, p->kc_tok, p->kc_head}, svc{p->vc_seq, p->vc_tok, p->vc_head};
  if (!strides_ok(p->n, nt, p->kv_heads, sk) || !strides_ok(p->n, nt, p->kv_heads, sv) ||
      !strides_ok(p->n, ct, p->kv_heads, skc) || !strides_ok(p->n, ct, p->kv_heads, svc))
    return CC3D_ERR_UNSUPPORTED;
  if (!aligned_to(p->k, 16) || !aligned_to(p->v, 16) || !aligned_to(p->k_cache, 16) ||
      !aligned_to(p->v_cache, 16))
    return CC3D_ERR_ALIGNMENT;
  if (!disjoint_entries(p->n, ct, p->kv_heads, p->d, skc) ||
      !disjoint_entries(p->n, ct, p->kv_heads, p->d, svc))
    return CC3D_ERR_ALIAS;
  void *const out[2] = {p->k_cache, p->v_cache};
  const size_t ob[2] = {static_cast<size_t>(span(p->n, ct, p->kv_heads, p->d, skc)) * 2,
                        static_cast<size_t>(span(p->n, ct, p->kv_heads, p->d, svc)) * 2};
  // the two caches may be interleaved: the same strides, and entries that do
  // not meet
  if (ranges_meet(out[0], ob[0], out[1], ob[1])) {
    const bool same = (p->n == 1 || skc.seq == svc.seq) && (ct == 1 || skc.tok == svc.tok) &&
                      (p->kv_heads == 1 || skc.head == svc.head);
    const long long bytes = static_cast<const char *>(out[0]) - static_cast<const char *>(out[1]);
    if (!same || bytes == 0 ||
        !disjoint_entries(p->n, ct, p->kv_heads, p->d, skc, (bytes < 0 ? -bytes : bytes) / 2))
      return CC3D_ERR_ALIAS;
  }
  for (int i = 0; i < 2; ++i)
    if (ranges_meet(out[i], ob[i], p->k,
                    static_cast<size_t>(span(p->n, nt, p->kv_heads, p->d, sk)) * 2) ||
        ranges_meet(out[i], ob[i], p->v,
                    static_cast<size_t>(span(p->n, nt, p->kv_heads, p->d, sv)) * 2) ||
        ranges_meet(out[i], ob[i], p->q_frames, static_cast<size_t>(p->n) * 4) ||
        ranges_meet(out[i], ob[i], p->k_frames, static_cast<size_t>(p->n) * 4))
      return CC3D_ERR_ALIAS;
  DeviceInfo dev;
  if (!device_info(&dev) || !dev.sm100) return CC3D_ERR_UNSUPPORTED;
  const CacheShape c{p->n, p->kv_heads, p->d, p->frame, p->slots, p->sinks, p->ring, p->t,
                     p->total, p->q_frames, p->k_frames};
  return status_of(launch_kv_append(
      c, static_cast<const __nv_bfloat16 *>(p->k), sk, static_cast<const __nv_bfloat16 *>(p->v), sv,
      static_cast<__nv_bfloat16 *>(p->k_cache), skc, static_cast<__nv_bfloat16 *>(p->v_cache), svc,
      dev.sm_count, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
