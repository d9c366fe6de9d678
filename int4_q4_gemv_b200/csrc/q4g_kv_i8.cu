// int8 K/V rows written into a cache as they are produced, and read back
// (q4g_kv_write_*_i8, q4g_kv_read_*_i8): per row of head_dim fp16 values one fp32
// scale = amax / 127 and codes rint(x / scale), the format the decode step writes
// (kv_quantize_row_warp) and the _i8 attention kernels read.
//
// Bound by HBM: 2 + 1 bytes per element and 4 per row, nothing read twice. A lane holds
// 16 values of a row, 32 lanes (hd 512) or 16 (hd 256, two rows a warp) the row, so the
// amax needs no second pass. 32,768 rows of K and V of hd 512, one KV head, written and
// read back (2 x 101 MB): 35.2 us, 5.7 TB/s, reads and writes mixed; 1,531 rows of 8 heads
// of 256 (2 x 19 MB): 9.1 us; 5,003 rows of 2 heads of 256 read in any order (15 MB): 3.8 us.
// (8 values a lane at hd 256 ran at 3.6 TB/s: what a row costs beside its bytes came twice
// as often.)
#include "../../include/q4g.h"
#include "q4g_common.cuh"
#include "q4g_internal.h"

using namespace q4g;

namespace {

constexpr int kKvThreads = 256;
// CTAs per SM at most, for K and V each. A write keeps 32 bytes a thread in flight and runs
// best as about three waves of CTAs that loop; a read is a wait for 16 bytes a thread and
// wants many short CTAs. Every CTA gets the same number of turns. 131,072 rows of hd 512,
// write and read: 135 us, against 142 with 12 for both and the last turns uneven (32,768
// rows: 35.2 against 38.3).
constexpr int kWriteCtas = 8, kReadCtas = 32;

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
    s = p.slots[t];
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
Q4G_DEV void quantize(float (&v)[E], float s, bool no_nan, uint32_t (&w)[E / 4]) {
  constexpr float kMagic = 12582912.0f;
  const bool huge = s > 3.0e38f;  // an infinite value in the row: every code 0
  if (!no_nan || huge) {
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

// Element offset of (t, h) among the fp16 rows; head counts may pass 2^31 / hd.
template <int HD>
Q4G_DEV int64_t row_offset(const KvCopyParams& p, int t, int h) {
  return t * p.row_stride + (int64_t)h * HD;
}

constexpr int E = 16;  // values of a row per lane
template <int HD>
constexpr int kRowLanes = HD / E;
template <int HD>
constexpr int kRowsAtOnce = kKvThreads / kRowLanes<HD>;  // rows of a CTA at a time

// A lane's values are 8 of the row's first half and 8 of its second, so that the lanes of a
// 16-byte load or store (8 bytes of codes) are neighbours.
template <int HD>
Q4G_DEV void load_row(const __half* p, uint4 (&r)[2]) {
  r[0] = ld_stream_u4_ordered(p);
  r[1] = ld_stream_u4_ordered(p + HD / 2);
}

// Both kernels load the next row before they work on this one.
template <int HD>
__global__ void __launch_bounds__(kKvThreads, 5) kv_write_kernel(const KvCopyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kRowLanes<HD>;
  const bool is_v = blockIdx.y != 0;
  const __half* const rows = (is_v ? p.v : p.k) + lane * 8;
  int8_t* const codes = (is_v ? p.v_codes : p.k_codes) + lane * 8;
  float* const scales = is_v ? p.v_scales : p.k_scales;
  const int total = p.n * p.n_kv, step = gridDim.x * kRowsAtOnce<HD>;
  int i = blockIdx.x * kRowsAtOnce<HD> + threadIdx.x / kRowLanes<HD>;
  // the lanes of a warp stay together: a row past the end is no row
  uint4 next[2] = {};
  int64_t next_row = -1;
  auto load = [&]() {
    next_row = -1;
    if (i >= total) return;
    const int t = i / p.n_kv, h = i - t * p.n_kv;
    load_row<HD>(rows + row_offset<HD>(p, t, h), next);
    next_row = cache_row(p, t, h);
  };
  load();
  for (int turns = (total + step - 1) / step; turns > 0; --turns) {
    const uint4 raw[2] = {next[0], next[1]};
    const int64_t row = next_row;
    i = i < total - step ? i + step : total;
    load();
    const uint32_t u[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    float v[E];
    __half2 most = __floats2half2_rn(0.f, 0.f), any = most;  // `any` keeps a NaN, `most` does not
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __half2 x = *reinterpret_cast<const __half2*>(&u[k]);
      const float2 f = __half22float2(x);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
      most = __hmax2(most, __habs2(x));
      any = __hmax2_nan(any, __habs2(x));
    }
    float amax = fmaxf(__low2float(most), __high2float(most));
#pragma unroll
    for (int o = kRowLanes<HD> / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = __fdiv_rn(amax, 127.0f);
    uint32_t w[E / 4];
    quantize<E>(v, s, !(__hisnan(__low2half(any)) || __hisnan(__high2half(any))), w);
    if (row >= 0) {
      *reinterpret_cast<uint2*>(codes + row * HD) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(codes + row * HD + HD / 2) = make_uint2(w[2], w[3]);
      if (lane == 0) scales[row] = s;
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvCopyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kRowLanes<HD>;
  const bool is_v = blockIdx.y != 0;
  __half* const rows = (is_v ? p.v : p.k) + lane * 8;
  const int8_t* const codes = (is_v ? p.v_codes : p.k_codes) + lane * 8;
  const float* const scales = is_v ? p.v_scales : p.k_scales;
  const int total = p.n * p.n_kv, step = gridDim.x * kRowsAtOnce<HD>;
  int i = blockIdx.x * kRowsAtOnce<HD> + threadIdx.x / kRowLanes<HD>;
  uint2 next[2] = {};
  float next_s = 0.f;
  __half* next_out = nullptr;
  auto load = [&]() {
    if (i >= total) return;
    const int t = i / p.n_kv, h = i - t * p.n_kv;
    next_out = rows + row_offset<HD>(p, t, h);
    const int64_t row = cache_row(p, t, h);
    next[0] = next[1] = make_uint2(0u, 0u);  // a slot outside the cache: zeros
    next_s = 0.f;
    if (row >= 0) {
      next[0] = *reinterpret_cast<const uint2*>(codes + row * HD);
      next[1] = *reinterpret_cast<const uint2*>(codes + row * HD + HD / 2);
      next_s = scales[row];
    }
  };
  load();
  while (i < total) {
    const uint32_t w[4] = {next[0].x, next[0].y, next[1].x, next[1].y};
    const float s = next_s;
    __half* const out = next_out;
    i = i < total - step ? i + step : total;
    load();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = w[2 * k + (j >> 1)] >> (16 * (j & 1));
        const __half2 h2 = __floats2half2_rn((float)(int8_t)(c & 0xff) * s, (float)(int8_t)((c >> 8) & 0xff) * s);
        o[j] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      *reinterpret_cast<uint4*>(out + k * (HD / 2)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

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
q4g_status launch(K kernel, int rows_at_once, int ctas, const KvCopyParams& p, cudaStream_t st) {
  const int64_t need = ((int64_t)p.n * p.n_kv + rows_at_once - 1) / rows_at_once;
  const int64_t cap = (int64_t)ctas * device_sm_count();  // for K and V each
  const int64_t turns = (need + cap - 1) / cap;
  const dim3 grid((unsigned)((need + turns - 1) / turns), 2);
  const cudaError_t e = launch_pdl(kernel, grid, kKvThreads, 0, st, true, 1, p);
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
  return hd == 512 ? launch(kv_write_kernel<512>, kRowsAtOnce<512>, kWriteCtas, p, st)
                   : launch(kv_write_kernel<256>, kRowsAtOnce<256>, kWriteCtas, p, st);
}

q4g_status run_read(KvCopyParams& p, uint16_t* k, uint16_t* v, int32_t hd, cudaStream_t st) {
  p.k = reinterpret_cast<__half*>(k);
  p.v = reinterpret_cast<__half*>(v);
  return hd == 512 ? launch(kv_read_kernel<512>, kRowsAtOnce<512>, kReadCtas, p, st)
                   : launch(kv_read_kernel<256>, kRowsAtOnce<256>, kReadCtas, p, st);
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
