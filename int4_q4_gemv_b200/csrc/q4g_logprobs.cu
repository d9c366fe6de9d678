// Log probabilities of given tokens, entropy and the likeliest alternatives of rows
// of logits (q4g_token_logprobs). With m the row's largest logit, T the temperature
// and d_i = (x_i - m) / T:
//   S = sum exp(d_i), logprob = d_t - ln S, entropy = ln S - sum(exp(d_i) d_i) / S.
//
// Bound by HBM: 4 bytes per logit, read once. Every thread keeps its own running
// (m, S, E = sum exp(d) d) and rescales them when its maximum moves; E counts from
// the maximum, so the entropy is a sum of terms of one sign and cancels nothing.
// The alternatives come out of the same pass: logits at or above a threshold enter
// a candidate buffer in shared memory, and the threshold is always a value that at
// least n_top logits of the row reach (first from the lane maxima of a warp, then
// the n_top-th best candidate), so nothing that belongs to the answer is left out.
// A row is split over the CTAs of one thread-block cluster when there are few rows;
// they join through distributed shared memory, in rank order, without scratch memory
// or atomics between CTAs: the sums do not depend on timing, nor does the answer on
// the order in which candidates enter the buffer (it is sorted by value and index).
#include <math.h>

#include "../../include/q4g.h"
#include "q4g_common.cuh"
#include "q4g_internal.h"

using namespace q4g;

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kVecs = 4;                            // 16-byte loads per thread and tile
constexpr int kTile = kLpThreads * kVecs * 4;       // logits per tile
constexpr int kKeep = 128;                          // candidates that may wait for the next tile
constexpr int kBuf = kTile + kKeep;
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster <= kLpWarps, "one warp merges one CTA's list");

typedef unsigned long long u64;

// Sort key: larger is better. High word: the logit's bits made monotonic (-0 as +0);
// low word: the index, inverted, so the lowest index wins ties. 0: no candidate.
Q4G_DEV u64 make_key(float x, int idx) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((u64)o << 32) | (uint32_t)~idx;
}
Q4G_DEV float key_value(u64 k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
Q4G_DEV int key_index(u64 k) { return (int)~(uint32_t)k; }

Q4G_DEV u64 shfl_xor_u64(u64 v, int o) {
  const uint32_t lo = __shfl_xor_sync(0xffffffffu, (uint32_t)v, o);
  const uint32_t hi = __shfl_xor_sync(0xffffffffu, (uint32_t)(v >> 32), o);
  return ((u64)hi << 32) | lo;
}
Q4G_DEV uint32_t shfl_xor_key(uint32_t v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
Q4G_DEV u64 shfl_xor_key(u64 v, int o) { return shfl_xor_u64(v, o); }

template <typename K>
Q4G_DEV K cmp_swap(K v, int o, bool up) {  // the smaller value to the lane that `up` names
  const K w = shfl_xor_key(v, o);
  return ((v < w) == up) ? v : w;
}
// A bitonic sequence over the lanes into falling order.
template <typename K>
Q4G_DEV K bitonic_merge_desc(K v, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = cmp_swap(v, o, (lane & o) != 0);
  return v;
}
// One value per lane into falling order.
template <typename K>
Q4G_DEV K sort_desc(K v, int lane) {
#pragma unroll
  for (int k = 2; k <= 16; k <<= 1)
#pragma unroll
    for (int o = k >> 1; o > 0; o >>= 1) v = cmp_swap(v, o, ((lane & o) != 0) == ((lane & k) == 0));
  return bitonic_merge_desc(v, lane);
}
// The 32 best of two lists in falling order, in falling order.
Q4G_DEV u64 merge_lists(u64 a, u64 b, int lane) {
  const int src = 31 - lane;
  const uint32_t lo = __shfl_sync(0xffffffffu, (uint32_t)b, src);
  const uint32_t hi = __shfl_sync(0xffffffffu, (uint32_t)(b >> 32), src);
  const u64 r = ((u64)hi << 32) | lo;
  return bitonic_merge_desc(a > r ? a : r, lane);
}

Q4G_DEV float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Running statistics in base 2: m, l = sum 2^(c (x - m)), e = sum 2^(c (x - m)) c (x - m),
// with c = log2(e) / T. m starts at the lowest finite value, so a row of -inf keeps l = 0.
struct Stat {
  float m, l, e;
};
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = -1e28f;  // far below any exponent that counts; times 0 it stays 0

Q4G_DEV Stat stat_join(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf((a.m - m) * c, kFar), db = fmaxf((b.m - m) * c, kFar);
  const float wa = ex2(da), wb = ex2(db);
  return {m, a.l * wa + b.l * wb, (a.e + da * a.l) * wa + (b.e + db * b.l) * wb};
}

struct LpShared {
  u64 lists[kLpWarps][32];  // per-warp lists while merging; [0] is the CTA's list
  u64 best;                 // the n_top-th best key so far (0: none)
  Stat warp_stat[kLpWarps];
  Stat stat;
  uint32_t warp_thr[kLpWarps];
  int count;                // candidates in the buffer
};

Q4G_DEV u64 ld_peer_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// The 32 best of the candidate buffer and of the list already held (lists[0], as
// candidates of their own when `held`), into lists[0]. All threads call it.
Q4G_DEV void compact(LpShared& sh, const u64* buf, int count, bool held, int n_top) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 best = warp == 0 && held ? sh.lists[0][lane] : 0ull;
  for (int b = warp * 32; b < count; b += kLpThreads) {
    const u64 k = b + lane < count ? buf[b + lane] : 0ull;
    best = merge_lists(best, sort_desc(k, lane), lane);
  }
  sh.lists[warp][lane] = best;
  __syncthreads();
#pragma unroll
  for (int s = 1; s < kLpWarps; s <<= 1) {
    if (warp % (2 * s) == 0) {
      best = merge_lists(best, sh.lists[warp + s][lane], lane);
      sh.lists[warp][lane] = best;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    sh.best = sh.lists[0][n_top - 1];
    sh.count = 0;
  }
  __syncthreads();
}

// A cluster of gridDim.x CTAs per row, gridDim.y rows. TOP: alternatives are wanted.
template <bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const LogprobParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  LpShared& sh = *reinterpret_cast<LpShared*>(smem_raw);
  u64* const buf = reinterpret_cast<u64*>(smem_raw + ((sizeof(LpShared) + 15) & ~15ul));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;
  const float* x = p.logits + (int64_t)row * p.row_stride;
  // the row in 16-byte pieces: piece v holds the logits 4 v - skew .. 4 v - skew + 3
  const int skew = (int)(((uintptr_t)x >> 2) & 3);
  const int n_vec = (int)(((int64_t)p.vocab + skew + 3) >> 2);
  const int per = (n_vec + ranks - 1) / ranks;
  const int v_end = min(n_vec, (rank + 1) * per);
  const float c = 1.4426950408889634f / p.temperature;
  const float x_target = rank == 0 && tid == 0 && p.targets && p.targets[row] >= 0 && p.targets[row] < p.vocab
                             ? x[p.targets[row]]
                             : __uint_as_float(0x7fc00000u);
  if (TOP) {
    if (tid == 0) sh.best = 0ull, sh.count = 0;
    __syncthreads();
  }

  Stat st = {kLowest, 0.f, 0.f};
  bool held = false;
  for (int v0 = rank * per; v0 < v_end; v0 += kLpThreads * kVecs) {
    float f[4 * kVecs];
    int first[kVecs];  // index of each piece's first logit
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int v = v0 + k * kLpThreads + tid;
      first[k] = 4 * v - skew;
      if (v < v_end && first[k] >= 0 && first[k] + 3 < p.vocab) {
        const uint4 u = ld_stream_u4(x + first[k]);
        f[4 * k] = __uint_as_float(u.x), f[4 * k + 1] = __uint_as_float(u.y);
        f[4 * k + 2] = __uint_as_float(u.z), f[4 * k + 3] = __uint_as_float(u.w);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = first[k] + j;
          f[4 * k + j] = v < v_end && i >= 0 && i < p.vocab ? __ldg(x + i) : -INFINITY;
        }
      }
    }
    float mx = f[0];
#pragma unroll
    for (int k = 1; k < 4 * kVecs; ++k) mx = fmaxf(mx, f[k]);
    {
      const float m = fmaxf(st.m, mx);
      const float d0 = fmaxf((st.m - m) * c, kFar), w = ex2(d0);
      st.e = (st.e + d0 * st.l) * w;
      st.l *= w;
      st.m = m;
    }
#pragma unroll
    for (int k = 0; k < 4 * kVecs; ++k) {
      const float d = (f[k] - st.m) * c;
      const float w = ex2(d);
      st.l += w;
      st.e = fmaf(w, fmaxf(d, kFar), st.e);
    }
    if (TOP) {
      // the lowest logit that may still belong to the answer
      uint32_t thr;
      u64 best = 0ull;
      if (!held) {
        // a warp's n_top-th largest lane maximum is reached by n_top logits; the
        // highest of the warps' counts
        const uint32_t mine = (uint32_t)(make_key(mx, 0) >> 32);
        const uint32_t s = __shfl_sync(0xffffffffu, sort_desc(mine, lane), p.n_top - 1);
        if (lane == 0) sh.warp_thr[warp] = s;
        __syncthreads();
        thr = 0u;
#pragma unroll
        for (int k = 0; k < kLpWarps; ++k) thr = max(thr, sh.warp_thr[k]);
      } else {
        best = sh.best;
        thr = (uint32_t)(best >> 32);
      }
      if ((uint32_t)(make_key(mx, 0) >> 32) >= thr) {
#pragma unroll
        for (int k = 0; k < 4 * kVecs; ++k) {
          const int i = first[k >> 2] + (k & 3);
          const int v = v0 + (k >> 2) * kLpThreads + tid;
          const u64 key = make_key(f[k], i);
          if (v < v_end && i >= 0 && i < p.vocab && (uint32_t)(key >> 32) >= thr && key > best) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kBuf) buf[at] = key;
          }
        }
      }
      __syncthreads();
      const int count = sh.count;
      __syncthreads();
      if (!held || count > kKeep) {
        compact(sh, buf, min(count, kBuf), held, p.n_top);
        held = true;
      }
    }
  }
  if (TOP) {
    const int count = sh.count;
    __syncthreads();
    if (count > 0 || !held) compact(sh, buf, min(count, kBuf), held, p.n_top);
  }

  // the CTA's statistics: lanes, then warps, in a fixed order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.l, o),
              __shfl_xor_sync(0xffffffffu, st.e, o)};
    st = stat_join(st, b, c);
  }
  if (lane == 0) sh.warp_stat[warp] = st;
  __syncthreads();
  if (tid == 0) {
    st = sh.warp_stat[0];
    for (int k = 1; k < kLpWarps; ++k) st = stat_join(st, sh.warp_stat[k], c);
    sh.stat = st;
  }
  if (ranks > 1) {
    cluster_sync();  // every rank's list and statistics are written
    if (rank == 0) {
      if (TOP) {
        u64 best = warp < ranks ? ld_peer_u64(peer_addr(&sh.lists[0][lane], warp)) : 0ull;
        __syncthreads();  // lists[0] of this CTA is read before lists[] is reused
        sh.lists[warp][lane] = best;
        __syncthreads();
#pragma unroll
        for (int s = 1; s < kLpWarps; s <<= 1) {
          if (warp % (2 * s) == 0) {
            best = merge_lists(best, sh.lists[warp + s][lane], lane);
            sh.lists[warp][lane] = best;
          }
          __syncthreads();
        }
      }
      if (tid == 0) {
        for (int r = 1; r < ranks; ++r) {
          const Stat b = {ld_peer_f32(peer_addr(&sh.stat.m, r)), ld_peer_f32(peer_addr(&sh.stat.l, r)),
                          ld_peer_f32(peer_addr(&sh.stat.e, r))};
          st = stat_join(st, b, c);
        }
        sh.stat = st;
      }
    }
    cluster_sync();  // no rank leaves while rank 0 reads its shared memory
    if (rank != 0) return;
  }
  __syncthreads();
  if (warp != 0) return;
  const Stat all = sh.stat;
  const float ln = all.l == 0.f ? 0.f : logf(all.l);  // l = 0: every logit is -inf
  if (lane == 0) {
    if (p.logprob) p.logprob[row] = (x_target - all.m) / p.temperature - ln;
    const float h = all.l == 0.f ? 0.f : ln - all.e / all.l * 0.6931471805599453f;
    if (p.entropy) p.entropy[row] = h < 0.f ? 0.f : h;  // a NaN stays one
  }
  if (TOP && lane < p.n_top) {
    const u64 k = sh.lists[0][lane];
    const int64_t at = (int64_t)row * p.n_top + lane;
    // a NaN among the logits may leave fewer than n_top candidates: stay inside the row
    if (p.top_ids) p.top_ids[at] = k ? key_index(k) : 0;
    if (p.top_logprobs)
      p.top_logprobs[at] = (k ? key_value(k) - all.m : __uint_as_float(0x7fc00000u)) / p.temperature - ln;
  }
}

q4g_status bad(q4g_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <bool TOP>
cudaError_t launch_t(const LogprobParams& p, int ranks, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kLpThreads);
  cfg.gridDim = dim3(ranks, p.rows);
  cfg.dynamicSmemBytes = ((sizeof(LpShared) + 15) & ~15ul) + (TOP ? sizeof(u64) * kBuf : 0);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<TOP>, p);
}

}  // namespace

cudaError_t q4g::launch_logprobs(const LogprobParams& p, cudaStream_t st) {
  // CTAs per row: enough for about six CTAs on every SM, but at least a tile for each
  const int64_t tiles = ((int64_t)p.vocab + kTile - 1) / kTile;
  int ranks = 1;
  while (ranks < kMaxCluster && (int64_t)p.rows * ranks < 6ll * device_sm_count() && 2 * ranks <= tiles) ranks *= 2;
  // the grid's y extent ends at 65535: longer calls go in pieces
  for (int r0 = 0; r0 < p.rows; r0 += 65535) {
    LogprobParams q = p;
    q.rows = p.rows - r0 < 65535 ? p.rows - r0 : 65535;
    q.logits += (int64_t)r0 * p.row_stride;
    if (q.targets) q.targets += r0;
    if (q.logprob) q.logprob += r0;
    if (q.entropy) q.entropy += r0;
    if (q.top_ids) q.top_ids += (int64_t)r0 * p.n_top;
    if (q.top_logprobs) q.top_logprobs += (int64_t)r0 * p.n_top;
    const cudaError_t e = p.n_top ? launch_t<true>(q, ranks, st) : launch_t<false>(q, ranks, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int q4g::make_logprobs(const float* logits, int64_t rows, int64_t vocab, int64_t row_stride, float temperature,
                       const int32_t* targets, float* logprob, float* entropy, int32_t n_top, int32_t* top_ids,
                       float* top_logprobs, LogprobParams* out) {
  if (rows < 0 || rows > (1 << 20)) return bad(Q4G_ERANGE, "rows outside [0, 2^20]");
  if (vocab < 1 || vocab > (1 << 30)) return bad(Q4G_ERANGE, "vocab outside [1, 2^30]");
  if (row_stride < vocab || row_stride > ((int64_t)1 << 40))
    return bad(Q4G_EINVAL, "row_stride must be at least vocab, at most 2^40");
  // a subnormal temperature would make log2(e) / temperature infinite
  if (!isnormal(temperature) || temperature < 0.f)
    return bad(Q4G_EINVAL, "temperature must be positive, finite and not subnormal");
  if (n_top < 0 || n_top > Q4G_LOGPROBS_MAX_TOP || n_top > vocab)
    return bad(Q4G_ERANGE, "n_top outside [0, min(32, vocab)]");
  if ((targets == nullptr) != (logprob == nullptr)) return bad(Q4G_EINVAL, "targets and logprob go together");
  if (n_top > 0 && !top_ids && !top_logprobs) return bad(Q4G_EINVAL, "n_top > 0 without top_ids and top_logprobs");
  if (rows > 0) {
    if (!logits) return bad(Q4G_EINVAL, "NULL pointer");
    const void* ptrs[] = {logits, targets, logprob, entropy, n_top ? top_ids : nullptr,
                          n_top ? top_logprobs : nullptr};
    for (const void* p : ptrs) {
      if (!p) continue;
      if (!aligned(p, 4)) return bad(Q4G_EINVAL, "misaligned pointer");
      if (!on_current_device(p)) return bad(Q4G_EINVAL, "a pointer is not memory of the current device");
    }
  }
  *out = {logits, row_stride, (int32_t)rows, (int32_t)vocab, temperature, targets, logprob, entropy, n_top,
          n_top ? top_ids : nullptr, n_top ? top_logprobs : nullptr};
  return Q4G_OK;
}

extern "C" q4g_status q4g_token_logprobs(const float* logits, int64_t rows, int64_t vocab, int64_t row_stride,
                                         float temperature, const int32_t* targets, float* logprob,
                                         float* entropy, int32_t n_top, int32_t* top_ids, float* top_logprobs,
                                         q4g_stream_t stream) {
  LogprobParams p;
  const int s = make_logprobs(logits, rows, vocab, row_stride, temperature, targets, logprob, entropy, n_top, top_ids,
                              top_logprobs, &p);
  if (s) return (q4g_status)s;
  if (!targets && !entropy && n_top == 0) return bad(Q4G_EINVAL, "no output wanted");
  if (rows == 0) return Q4G_OK;
  const cudaError_t e = launch_logprobs(p, (cudaStream_t)stream);
  return e == cudaSuccess ? Q4G_OK : bad(Q4G_ECUDA, cudaGetErrorString(e));
}
