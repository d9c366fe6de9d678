// int8 K/V rows written into a cache as they are produced, and read back
// (q4g_kv_write_*_i8, q4g_kv_read_*_i8): per row of head_dim fp16 values one fp32
// scale = amax / 127 and codes rint(x / scale), the format the decode step writes
// (kv_quantize_row_warp) and the _i8 attention kernels read.
//
// Bound by HBM: 2 + 1 bytes per element and 4 per row, nothing read twice. A warp
// holds a whole row in registers (8 or 16 values per lane, 16-byte loads), so the
// amax needs no second pass; the row goes out as one 8- or 16-byte store per lane.
#include "../../include/q4g.h"
#include "q4g_common.cuh"
#include "q4g_internal.h"

using namespace q4g;

namespace {

constexpr int kKvThreads = 256;

struct KvCopyParams {
  __half *k, *v;         // fp16 rows: read by a write, written by a read
  int8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  const int64_t* slots;  // or NULL: slot = slot0 + t, wrapped at `wrap`
  int64_t slot0, wrap;   // slot0 in [0, wrap)
  int64_t row_stride;    // fp16 elements between rows t and t + 1
  int64_t slot_stride, head_stride;  // cache rows between slots and between KV heads
  int32_t n, n_kv;       // rows and KV heads, n * n_kv <= 2^30
};

// The cache row of (t, h), or -1 if its slot lies outside the cache.
Q4G_DEV int64_t cache_row(const KvCopyParams& p, int t, int h) {
  int64_t s;
  if (p.slots) {
    s = __ldg(reinterpret_cast<const long long*>(p.slots) + t);
    if (s < 0 || s >= p.wrap) return -1;
  } else {
    s = p.slot0 + t;
    if (s >= p.wrap) s -= p.wrap;
  }
  return s * p.slot_stride + h * p.head_stride;
}

// Codes of E values of one row at scale s: rint of the IEEE quotient v / s. One
// division per lane gives the correctly rounded reciprocal y; q = v y and the
// residual step q + (v - q s) y then give the correctly rounded quotient (P. Markstein,
// IBM J. Res. Dev. 34, 1990; no underflow: 2^-24 <= |v| <= 2^16 here), two FMAs in
// place of a division of about ten instructions per value, which would cost more
// issue slots than the row's bytes cost HBM time. |v| / s rounds to 127 at most.
// Adding 1.5 * 2^23 rounds to the nearest integer, ties to even, in the low bits.
template <int E>
Q4G_DEV void quantize(float (&v)[E], float s, bool finite, uint32_t (&w)[E / 4]) {
  constexpr float kMagic = 12582912.0f;
  const bool huge = s > 3.0e38f;  // an infinite value in the row: every code 0
  if (!finite || huge) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = huge || !(fabsf(v[e]) < 1e6f) ? 0.f : v[e];
  }
  const float d = s > 0.f && !huge ? s : 1.0f;
  const float y = __fdiv_rn(1.0f, d);
  uint32_t b[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float q = __fmul_rn(v[e], y);
    b[e] = __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-q, d, v[e]), y, q), kMagic));
  }
#pragma unroll
  for (int k = 0; k < E / 4; ++k) {
    const uint32_t lo = __byte_perm(b[4 * k], b[4 * k + 1], 0x0040);
    const uint32_t hi = __byte_perm(b[4 * k + 2], b[4 * k + 3], 0x0040);
    w[k] = __byte_perm(lo, hi, 0x5410);
  }
}

template <int E>
Q4G_DEV void load_row(const __half* p, uint4 (&r)[E / 8]) {
#pragma unroll
  for (int k = 0; k < E / 8; ++k) r[k] = ld_stream_u4(p + 8 * k);
}

template <int HD>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvCopyParams p) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const bool is_v = blockIdx.y != 0;
  __half* const rows = is_v ? p.v : p.k;
  int8_t* const codes = is_v ? p.v_codes : p.k_codes;
  float* const scales = is_v ? p.v_scales : p.k_scales;
  const int total = p.n * p.n_kv;
  const int step = gridDim.x * (kKvThreads / 32);
  for (int64_t i = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const int t = (int)i / p.n_kv, h = (int)i - t * p.n_kv;
    const int64_t row = cache_row(p, t, h);
    if (row < 0) continue;
    uint4 raw[E / 8];
    load_row<E>(rows + t * p.row_stride + h * HD + lane * E, raw);
    float v[E], amax = 0.f, odd = 0.f;
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      const uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
        v[8 * k + 2 * j] = f.x;
        v[8 * k + 2 * j + 1] = f.y;
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        odd = fmaf(f.x, 0.f, fmaf(f.y, 0.f, odd));  // a NaN or an infinity makes it NaN
      }
    }
    const float s = __fdiv_rn(warp_max(amax), 127.0f);
    uint32_t w[E / 4];
    quantize<E>(v, s, odd == 0.f, w);
    int8_t* out = codes + row * HD + lane * E;
    if constexpr (E == 16) {
      *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    }
    if (lane == 0) scales[row] = s;
  }
}

template <int HD>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvCopyParams p) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const bool is_v = blockIdx.y != 0;
  __half* const rows = is_v ? p.v : p.k;
  int8_t* const codes = is_v ? p.v_codes : p.k_codes;
  float* const scales = is_v ? p.v_scales : p.k_scales;
  const int total = p.n * p.n_kv;
  const int step = gridDim.x * (kKvThreads / 32);
  for (int64_t i = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const int t = (int)i / p.n_kv, h = (int)i - t * p.n_kv;
    const int64_t row = cache_row(p, t, h);
    uint32_t w[E / 4];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < E / 4; ++k) w[k] = 0u;
    if (row >= 0) {
      const int8_t* in = codes + row * HD + lane * E;
      s = __ldg(scales + row);
      if constexpr (E == 16) {
        const uint4 u = ld_stream_u4(in);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(in));
        w[0] = u.x, w[1] = u.y;
      }
    }
    __half* out = rows + t * p.row_stride + h * HD + lane * E;
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = w[2 * k + (j >> 1)] >> (16 * (j & 1));
        const __half2 h2 = __floats2half2_rn((float)(int8_t)(c & 0xff) * s, (float)(int8_t)((c >> 8) & 0xff) * s);
        o[j] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      *reinterpret_cast<uint4*>(out + 8 * k) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

q4g_status bad(q4g_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Sizes that the four entry points check alike.
q4g_status check_sizes(int64_t n_rows, int64_t row_stride, int32_t n_kv, int32_t hd, int64_t capacity) {
  if (hd != 256 && hd != 512) return bad(Q4G_EINVAL, "head_dim must be 256 or 512");
  if (n_kv < 1) return bad(Q4G_EINVAL, "n_kv must be positive");
  if (n_rows < 0 || n_rows > ((int64_t)1 << 30) || n_rows * n_kv > ((int64_t)1 << 30))
    return bad(Q4G_ERANGE, "need 0 <= n_rows * n_kv <= 2^30");
  if (capacity < 1 || capacity > ((int64_t)1 << 30)) return bad(Q4G_ERANGE, "capacity or ring outside [1, 2^30]");
  if (row_stride < (int64_t)n_kv * hd || row_stride % 8 || row_stride > ((int64_t)1 << 32))
    return bad(Q4G_EINVAL, "row_stride must be a multiple of 8, at least n_kv * head_dim, at most 2^32");
  return Q4G_OK;
}

q4g_status check_linear(const int64_t* slots, int64_t slot0, int64_t n_rows, int64_t capacity) {
  if (slots && slot0 != 0) return bad(Q4G_EINVAL, "slot0 must be 0 with slots");
  if (!slots && (slot0 < 0 || n_rows > capacity || slot0 > capacity - n_rows))
    return bad(Q4G_ERANGE, "rows outside [0, capacity)");
  return Q4G_OK;
}

q4g_status check_ring(int64_t pos0, int64_t n_rows) {
  if (pos0 < 0 || pos0 > INT64_MAX - n_rows) return bad(Q4G_ERANGE, "need pos0 >= 0 and pos0 + n_rows < 2^63");
  return Q4G_OK;
}

q4g_status check_pointers(const void* k, const void* v, const void* kc, const void* ks, const void* vc,
                          const void* vs, const int64_t* slots) {
  const void* ptrs[] = {k, v, kc, vc, ks, vs, slots};
  const size_t align[] = {16, 16, 16, 16, 4, 4, 8};
  for (int i = 0; i < 6; ++i)
    if (!ptrs[i]) return bad(Q4G_EINVAL, "NULL pointer");
  for (int i = 0; i < 7; ++i)
    if (!aligned(ptrs[i], align[i])) return bad(Q4G_EINVAL, "misaligned pointer");
  for (const void* p : ptrs)
    if (p && !on_current_device(p)) return bad(Q4G_EINVAL, "a pointer is not memory of the current device");
  return Q4G_OK;
}

template <typename K>
q4g_status launch(K kernel, const KvCopyParams& p, cudaStream_t st) {
  const int warps = kKvThreads / 32;
  const int64_t need = ((int64_t)p.n * p.n_kv + warps - 1) / warps;
  const int64_t cap = 4ll * device_sm_count();
  const dim3 grid((unsigned)(need < cap ? need : cap), 2);
  kernel<<<grid, kKvThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? Q4G_OK : bad(Q4G_ECUDA, cudaGetErrorString(e));
}

KvCopyParams cache_params(int8_t* kc, float* ks, int8_t* vc, float* vs, int64_t n, int32_t n_kv, int64_t row_stride) {
  KvCopyParams p{};
  p.k_codes = kc, p.v_codes = vc;
  p.k_scales = ks, p.v_scales = vs;
  p.n = (int32_t)n;
  p.n_kv = n_kv;
  p.row_stride = row_stride;
  return p;
}

void linear_slots(KvCopyParams& p, const int64_t* slots, int64_t slot0, int64_t capacity) {
  p.slots = slots;
  p.slot0 = slot0;
  p.wrap = capacity;
  p.slot_stride = p.n_kv;
  p.head_stride = 1;
}

void ring_slots(KvCopyParams& p, int64_t pos0, int64_t ring) {
  p.slot0 = pos0 % ring;
  p.wrap = ring;
  p.slot_stride = 1;
  p.head_stride = ring;
}

q4g_status run_write(KvCopyParams& p, const uint16_t* k, const uint16_t* v, int32_t hd, cudaStream_t st) {
  p.k = reinterpret_cast<__half*>(const_cast<uint16_t*>(k));
  p.v = reinterpret_cast<__half*>(const_cast<uint16_t*>(v));
  return hd == 512 ? launch(kv_write_kernel<512>, p, st) : launch(kv_write_kernel<256>, p, st);
}

q4g_status run_read(KvCopyParams& p, uint16_t* k, uint16_t* v, int32_t hd, cudaStream_t st) {
  p.k = reinterpret_cast<__half*>(k);
  p.v = reinterpret_cast<__half*>(v);
  return hd == 512 ? launch(kv_read_kernel<512>, p, st) : launch(kv_read_kernel<256>, p, st);
}

}  // namespace

extern "C" q4g_status q4g_kv_write_linear_i8(const uint16_t* k, const uint16_t* v, int64_t n_rows,
                                             int64_t row_stride, int32_t n_kv, int32_t head_dim,
                                             const int64_t* slots, int64_t slot0, int64_t capacity, int8_t* k_codes,
                                             float* k_scales, int8_t* v_codes, float* v_scales,
                                             q4g_stream_t stream) {
  q4g_status s = check_sizes(n_rows, row_stride, n_kv, head_dim, capacity);
  if (s || (s = check_linear(slots, slot0, n_rows, capacity)) || n_rows == 0) return s;
  if ((s = check_pointers(k, v, k_codes, k_scales, v_codes, v_scales, slots))) return s;
  KvCopyParams p = cache_params(k_codes, k_scales, v_codes, v_scales, n_rows, n_kv, row_stride);
  linear_slots(p, slots, slot0, capacity);
  return run_write(p, k, v, head_dim, (cudaStream_t)stream);
}

extern "C" q4g_status q4g_kv_write_ring_i8(const uint16_t* k, const uint16_t* v, int64_t n_rows, int64_t row_stride,
                                           int32_t n_kv, int32_t head_dim, int64_t pos0, int64_t ring,
                                           int8_t* k_codes, float* k_scales, int8_t* v_codes, float* v_scales,
                                           q4g_stream_t stream) {
  q4g_status s = check_sizes(n_rows, row_stride, n_kv, head_dim, ring);
  if (s || (s = check_ring(pos0, n_rows)) || n_rows == 0) return s;
  if ((s = check_pointers(k, v, k_codes, k_scales, v_codes, v_scales, nullptr))) return s;
  // of more rows than slots only the last `ring` stay: the older ones are not written
  const int64_t skip = n_rows > ring ? n_rows - ring : 0;
  KvCopyParams p = cache_params(k_codes, k_scales, v_codes, v_scales, n_rows - skip, n_kv, row_stride);
  ring_slots(p, pos0 + skip, ring);
  return run_write(p, k + skip * row_stride, v + skip * row_stride, head_dim, (cudaStream_t)stream);
}

extern "C" q4g_status q4g_kv_read_linear_i8(const int8_t* k_codes, const float* k_scales, const int8_t* v_codes,
                                            const float* v_scales, int32_t n_kv, int32_t head_dim,
                                            const int64_t* slots, int64_t slot0, int64_t capacity, int64_t n_rows,
                                            uint16_t* k, uint16_t* v, int64_t row_stride, q4g_stream_t stream) {
  q4g_status s = check_sizes(n_rows, row_stride, n_kv, head_dim, capacity);
  if (s || (s = check_linear(slots, slot0, n_rows, capacity)) || n_rows == 0) return s;
  if ((s = check_pointers(k, v, k_codes, k_scales, v_codes, v_scales, slots))) return s;
  KvCopyParams p = cache_params(const_cast<int8_t*>(k_codes), const_cast<float*>(k_scales),
                                const_cast<int8_t*>(v_codes), const_cast<float*>(v_scales), n_rows, n_kv, row_stride);
  linear_slots(p, slots, slot0, capacity);
  return run_read(p, k, v, head_dim, (cudaStream_t)stream);
}

extern "C" q4g_status q4g_kv_read_ring_i8(const int8_t* k_codes, const float* k_scales, const int8_t* v_codes,
                                          const float* v_scales, int32_t n_kv, int32_t head_dim, int64_t pos0,
                                          int64_t ring, int64_t n_rows, uint16_t* k, uint16_t* v,
                                          int64_t row_stride, q4g_stream_t stream) {
  q4g_status s = check_sizes(n_rows, row_stride, n_kv, head_dim, ring);
  if (s || (s = check_ring(pos0, n_rows))) return s;
  if (n_rows > ring) return bad(Q4G_ERANGE, "a ring holds no more than `ring` rows");
  if (n_rows == 0) return Q4G_OK;
  if ((s = check_pointers(k, v, k_codes, k_scales, v_codes, v_scales, nullptr))) return s;
  KvCopyParams p = cache_params(const_cast<int8_t*>(k_codes), const_cast<float*>(k_scales),
                                const_cast<int8_t*>(v_codes), const_cast<float*>(v_scales), n_rows, n_kv, row_stride);
  ring_slots(p, pos0, ring);
  return run_read(p, k, v, head_dim, (cudaStream_t)stream);
}
