// Flash-decode of a batch whose sequences share a prefix (q4g_flash_decode_shared).
#include <math.h>

#include "../../include/q4g.h"
#include "q4g_common.cuh"
#include "q4g_internal.h"

using namespace q4g;

namespace {

struct SharedParams {
  const __half* q;
  const void* k[2];       // K rows: [0] the prefix, [1] the sequences' own
  const void* v[2];
  const float* ks[2];     // int8 rows: scales
  const float* vs[2];
  int64_t prefix, own_cap;
  const int32_t* own_len;
  int32_t batch, n_q, n_kv, n_split;  // prefix splits; one more entry holds the own rows
  float* ml;              // [batch * n_q][n_split + 1][2]
  float* acc;             // [batch * n_q][n_split + 1][hd]
  __half* out;
};

template <int HD, bool I8>
Q4G_DEV void load_row(const void* base, const float* scales, int64_t row, int lane, float (&x)[HD / 32]) {
  constexpr int E = HD / 32;
  if constexpr (I8) {
    const float s = scales[row];
    const int8_t* p = reinterpret_cast<const int8_t*>(base) + row * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = (float)p[e] * s;
  } else {
    const __half* p = reinterpret_cast<const __half*>(base) + row * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __half2float(p[e]);
  }
}

// One warp per (query row, part of its keys).
template <int HD, bool I8>
__global__ void shared_kernel(const SharedParams p) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x;
  const int qr = blockIdx.x, part = blockIdx.y, b = qr / p.n_q, h = (qr % p.n_q) / (p.n_q / p.n_kv);
  const int own = part == p.n_split;
  int64_t k0 = 0, k1 = 0, row0 = 0;
  if (own) {
    if (p.own_cap > 0) k1 = min((int64_t)max(p.own_len[b], 0), p.own_cap);
    row0 = b * p.own_cap;
  } else {
    k0 = p.prefix * part / p.n_split;
    k1 = p.prefix * (part + 1) / p.n_split;
  }
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __half2float(p.q[(int64_t)qr * HD + lane * E + e]), acc[e] = 0.f;
  for (int64_t k = k0; k < k1; ++k) {
    const int64_t row = (row0 + k) * p.n_kv + h;
    float x[E], s = 0.f;
    load_row<HD, I8>(p.k[own], p.ks[own], row, lane, x);
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * x[e];
    s = warp_sum(s);
    const float mn = fmaxf(m, s), w = mn == -INFINITY ? 0.f : expf(m - mn), pr = mn == -INFINITY ? 0.f : expf(s - mn);
    load_row<HD, I8>(p.v[own], p.vs[own], row, lane, x);
    l = l * w + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * w + pr * x[e];
    m = mn;
  }
  const int64_t at = (int64_t)qr * (p.n_split + 1) + part;
  if (lane == 0) p.ml[2 * at] = m, p.ml[2 * at + 1] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) p.acc[at * HD + lane * E + e] = acc[e];
}

template <int HD>
__global__ void shared_combine_kernel(const SharedParams p) {
  const int64_t qr = blockIdx.x;
  const int n = p.n_split + 1;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int i = 0; i < n; ++i) m = fmaxf(m, p.ml[2 * (qr * n + i)]);
  for (int i = 0; i < n && m != -INFINITY; ++i) {
    const float w = expf(p.ml[2 * (qr * n + i)] - m);
    l += w * p.ml[2 * (qr * n + i) + 1];
    o += w * p.acc[(qr * n + i) * HD + threadIdx.x];
  }
  p.out[qr * HD + threadIdx.x] = __float2half_rn(l > 0.f ? o / l : 0.f);
}

q4g_status bad(q4g_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kSplits = 32;

q4g_status run_shared(const uint16_t* q, int32_t batch, int32_t n_q, int32_t n_kv, int32_t hd, const void* kp,
                      const float* kps, const void* vp, const float* vps, int64_t prefix, const void* ko,
                      const float* kos, const void* vo, const float* vos, int64_t own_cap, const int32_t* own_len,
                      uint16_t* out, void* ws, size_t ws_bytes, bool i8, cudaStream_t st) {
  if (hd != 256 && hd != 512) return bad(Q4G_EINVAL, "head_dim must be 256 or 512");
  if (n_q < 1 || n_kv < 1 || n_q % n_kv || n_q > 1024) return bad(Q4G_EINVAL, "n_q must be a positive multiple of n_kv, at most 1024");
  if (batch < 1 || batch > 256) return bad(Q4G_ERANGE, "batch outside [1, 256]");
  if (prefix < 0 || prefix > ((int64_t)1 << 30)) return bad(Q4G_ERANGE, "prefix_len outside [0, 2^30]");
  if (own_cap < 0 || own_cap > (1 << 24) || own_cap * batch > ((int64_t)1 << 30))
    return bad(Q4G_ERANGE, "own_capacity outside [0, 2^24] or batch * own_capacity above 2^30");
  if (!q || !out || !ws) return bad(Q4G_EINVAL, "NULL pointer");
  if (prefix > 0 && (!kp || !vp || (i8 && (!kps || !vps)))) return bad(Q4G_EINVAL, "prefix rows NULL");
  if (own_cap > 0 && (!ko || !vo || !own_len || (i8 && (!kos || !vos)))) return bad(Q4G_EINVAL, "own rows NULL");
  const void* p16[] = {q, prefix ? kp : nullptr, prefix ? vp : nullptr, own_cap ? ko : nullptr,
                       own_cap ? vo : nullptr, out, ws};
  const void* p4[] = {i8 && prefix ? kps : nullptr, i8 && prefix ? vps : nullptr, i8 && own_cap ? kos : nullptr,
                      i8 && own_cap ? vos : nullptr, own_cap ? own_len : nullptr};
  for (const void* p : p16)
    if (!aligned(p, 16)) return bad(Q4G_EINVAL, "misaligned pointer");
  for (const void* p : p4)
    if (!aligned(p, 4)) return bad(Q4G_EINVAL, "misaligned pointer");
  if (!aligned(ws, 256)) return bad(Q4G_EINVAL, "workspace misaligned");
  for (const void* p : p16)
    if (p && !on_current_device(p)) return bad(Q4G_EINVAL, "a pointer is not memory of the current device");
  for (const void* p : p4)
    if (p && !on_current_device(p)) return bad(Q4G_EINVAL, "a pointer is not memory of the current device");
  if (ws_bytes < q4g_flash_decode_shared_workspace_bytes(batch, n_q, n_kv, hd))
    return bad(Q4G_EINVAL, "workspace too small");
  SharedParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.k[0] = kp, p.k[1] = ko, p.v[0] = vp, p.v[1] = vo;
  p.ks[0] = kps, p.ks[1] = kos, p.vs[0] = vps, p.vs[1] = vos;
  p.prefix = prefix;
  p.own_cap = own_cap;
  p.own_len = own_len;
  p.batch = batch, p.n_q = n_q, p.n_kv = n_kv, p.n_split = kSplits;
  p.ml = reinterpret_cast<float*>(ws);
  p.acc = p.ml + (((size_t)batch * n_q * (kSplits + 1) * 2 + 63) & ~(size_t)63);
  p.out = reinterpret_cast<__half*>(out);
  const dim3 grid(batch * n_q, kSplits + 1);
  if (hd == 512) {
    if (i8) shared_kernel<512, true><<<grid, 32, 0, st>>>(p);
    else shared_kernel<512, false><<<grid, 32, 0, st>>>(p);
    shared_combine_kernel<512><<<batch * n_q, 512, 0, st>>>(p);
  } else {
    if (i8) shared_kernel<256, true><<<grid, 32, 0, st>>>(p);
    else shared_kernel<256, false><<<grid, 32, 0, st>>>(p);
    shared_combine_kernel<256><<<batch * n_q, 256, 0, st>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? Q4G_OK : bad(Q4G_ECUDA, cudaGetErrorString(e));
}

}  // namespace

extern "C" size_t q4g_flash_decode_shared_workspace_bytes(int32_t batch, int32_t n_q, int32_t n_kv,
                                                          int32_t head_dim) {
  if (batch < 1 || n_q < 1 || n_kv < 1 || head_dim < 1) return 256;
  const size_t rows = (size_t)batch * n_q * (kSplits + 1);
  return sizeof(float) * (((rows * 2 + 63) & ~(size_t)63) + rows * head_dim);
}

extern "C" q4g_status q4g_flash_decode_shared(const uint16_t* q, int32_t batch, int32_t n_q, int32_t n_kv,
                                              int32_t head_dim, const uint16_t* k_prefix, const uint16_t* v_prefix,
                                              int64_t prefix_len, const uint16_t* k_own, const uint16_t* v_own,
                                              int64_t own_capacity, const int32_t* own_len, uint16_t* out,
                                              void* workspace, size_t workspace_bytes, q4g_stream_t stream) {
  return run_shared(q, batch, n_q, n_kv, head_dim, k_prefix, nullptr, v_prefix, nullptr, prefix_len, k_own, nullptr,
                    v_own, nullptr, own_capacity, own_len, out, workspace, workspace_bytes, false,
                    (cudaStream_t)stream);
}

extern "C" q4g_status q4g_flash_decode_shared_i8(
    const uint16_t* q, int32_t batch, int32_t n_q, int32_t n_kv, int32_t head_dim, const int8_t* k_prefix_codes,
    const float* k_prefix_scales, const int8_t* v_prefix_codes, const float* v_prefix_scales, int64_t prefix_len,
    const int8_t* k_own_codes, const float* k_own_scales, const int8_t* v_own_codes, const float* v_own_scales,
    int64_t own_capacity, const int32_t* own_len, uint16_t* out, void* workspace, size_t workspace_bytes,
    q4g_stream_t stream) {
  return run_shared(q, batch, n_q, n_kv, head_dim, k_prefix_codes, k_prefix_scales, v_prefix_codes, v_prefix_scales,
                    prefix_len, k_own_codes, k_own_scales, v_own_codes, v_own_scales, own_capacity, own_len, out,
                    workspace, workspace_bytes, true, (cudaStream_t)stream);
}
