// Log probabilities of given tokens, entropy and the likeliest alternatives of rows
// of logits (q4g_token_logprobs). With m the row's largest logit, T the temperature
// and d_i = (x_i - m) / T:
//   S = sum exp(d_i), logprob = d_t - ln S, entropy = ln S - sum(exp(d_i) d_i) / S.
//
// Bound by HBM: 4 bytes per logit, read once. Every thread keeps its own running
// (m, S, E = sum exp(d) d) and rescales them when its maximum moves; E counts from
// the maximum, so the entropy is a sum of terms of one sign and cancels nothing.
// The alternatives cost the pass little: it leaves the largest logit of every share (a
// thread's logits in an eighth of a CTA's tiles), and the n_top best logits of a CTA's part
// lie in the shares whose largest is at least the n_top-th largest of those (n_top logits
// reach it). Only these n_top of some 2000 shares are read again, and what reaches that
// value is sorted. On 256 rows of 262,144 logits (268 MB, 41.0 us at the measured copy
// rate) 42 to 44 us without alternatives, 50 to 52 us with 20; tried instead: shares of
// whole threads (42 MB read again) 60 us, lists kept up to date while reading 98 (a CTA's)
// and 106 us (a warp's), bulk copies into a ring in shared memory 55 without alternatives.
// Where the n_top-th largest is no threshold the row is read again in full, through the warps'
// lists: 256 rows of equal logits take 472 us, with 5 finite logits and n_top 20 655 us (one
// row 109 and 151, against 9.7).
// A row is split over the CTAs of one thread-block cluster when there are few rows; they
// join through distributed shared memory, in rank order, without scratch memory or atomics
// between CTAs. The sums depend on no timing; candidates arrive in any order, and sorting
// them by value and index gives the same list each time.
#include <math.h>

#include "../../include/q4g.h"
#include "q4g_common.cuh"
#include "q4g_internal.h"

using namespace q4g;

namespace {

constexpr int kVecs = 4;           // 16-byte loads per thread and tile
constexpr int kMaxCluster = 8;     // no more than a CTA's warps: one merges one CTA's list
constexpr int kSmall = 256, kLarge = 1024;  // threads per CTA
constexpr int tile_of(int threads) { return threads * kVecs * 4; }  // logits per tile
constexpr int shares_of(int threads) { return 2048 / threads; }    // of a thread, at most

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
Q4G_DEV uint32_t shfl_key(uint32_t v, int src) { return __shfl_sync(0xffffffffu, v, src); }
Q4G_DEV u64 shfl_key(u64 v, int src) {
  return ((u64)shfl_key((uint32_t)(v >> 32), src) << 32) | shfl_key((uint32_t)v, src);
}
// The 32 best of two lists in falling order, in falling order.
template <typename K>
Q4G_DEV K merge_lists(K a, K b, int lane) {
  const K r = shfl_key(b, 31 - lane);
  return bitonic_merge_desc(a > r ? a : r, lane);
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

template <int THREADS>
struct LpShared {
  u64 lists[THREADS / 32][32];  // the warps' lists while merging; [0] is then the CTA's
  u64 wait[THREADS / 32][64];   // candidates: the CTA's in a row, or each warp's until they are 32
  Stat warp_stat[THREADS / 32];
  Stat stat;
  uint32_t maxima[THREADS / 32][32];  // as lists, of the shares' largest logits (keys' high words)
  float largest[shares_of(THREADS)][THREADS];
  uint16_t hits[shares_of(THREADS) * THREADS];  // shares to read again: number * THREADS + thread
  int n_hits, n_found;
};

Q4G_DEV u64 ld_peer_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// The first N warps' lists, each in falling order, into one: the 32 best, in lists[0]. All
// threads call it; it ends with a barrier.
template <int N, int WARPS, typename K>
Q4G_DEV void merge_warps(K (&lists)[WARPS][32], K best) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < N) lists[warp][lane] = best;
  __syncthreads();
#pragma unroll
  for (int s = 1; s < N; s <<= 1) {
    if (warp < N && warp % (2 * s) == 0) {
      best = merge_lists(best, lists[warp + s][lane], lane);
      lists[warp][lane] = best;
    }
    __syncthreads();
  }
}

// A warp's running list: `best` in falling order over the lanes, `n` candidates waiting.
struct Top {
  u64 best = 0ull, last = 0ull;  // last: the n_top-th, the same in all lanes
  int n = 0;
};
// The first 32 waiting candidates (or all n < 32) into the list.
Q4G_DEV void take_in(Top& t, u64* wait, int lane, int n_top) {
  __syncwarp();
  const u64 k = lane < t.n ? wait[lane] : 0ull, rest = 32 + lane < t.n ? wait[32 + lane] : 0ull;
  t.best = merge_lists(t.best, sort_desc(k, lane), lane);
  __syncwarp();
  t.n = t.n > 32 ? t.n - 32 : 0;
  if (lane < t.n) wait[lane] = rest;
  __syncwarp();
  t.last = shfl_key(t.best, n_top - 1);
}

// Four logits from index 4 v - skew on, -inf for what lies outside [0, vocab).
Q4G_DEV float4 load_piece(const float* x, int v, int v_end, int skew, int vocab) {
  const int first = 4 * v - skew;
  if (v < v_end && first >= 0 && first + 3 < vocab) {
    const uint4 u = ld_stream_u4_ordered(x + first);
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  auto one = [&](int i) { return v < v_end && i >= 0 && i < vocab ? x[i] : -INFINITY; };
  return make_float4(one(first), one(first + 1), one(first + 2), one(first + 3));
}

template <int THREADS>
Q4G_DEV void load_tile(const float* x, int v0, int v_end, int skew, int vocab, float (&f)[4 * kVecs]) {
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const float4 u = load_piece(x, v0 + k * THREADS + threadIdx.x, v_end, skew, vocab);
    f[4 * k] = u.x, f[4 * k + 1] = u.y, f[4 * k + 2] = u.z, f[4 * k + 3] = u.w;
  }
}

// Every piece of the shares in sh.hits, a warp a share and a lane a piece: take(key, whether
// the index is inside the row and the logit reaches thr) in converged warps. `per`: pieces
// of a thread in a share.
template <int THREADS, typename F>
Q4G_DEV void read_again(const LpShared<THREADS>& sh, const float* x, int v_begin, int v_end, int per, int skew,
                        int vocab, float thr, F take) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_hits = sh.n_hits;
  for (int h = warp; h < n_hits; h += THREADS / 32) {
    const int share = sh.hits[h] / THREADS, v_hit = v_begin + share * per * THREADS + sh.hits[h] % THREADS;
    for (int q0 = 0; q0 < per; q0 += 64) {
      float4 f[2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
        f[b] = load_piece(x, q0 + 32 * b + lane < per ? v_hit + (q0 + 32 * b + lane) * THREADS : v_end, v_end, skew,
                          vocab);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int v = v_hit + (q0 + 32 * b + lane) * THREADS;
        const float e[4] = {f[b].x, f[b].y, f[b].z, f[b].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (__any_sync(0xffffffffu, e[j] >= thr)) {
            const int i = 4 * v - skew + j;
            take(make_key(e[j], i), e[j] >= thr && q0 + 32 * b + lane < per && v < v_end && i >= 0 && i < vocab);
          }
        }
      }
    }
  }
}

// The CTA's 32 best logits (n_top of them for certain) into sh.lists[0], from the shares'
// largest in sh.largest (each thread's own are written). Ends with a barrier.
template <int THREADS>
Q4G_DEV void find_top(LpShared<THREADS>& sh, const float* x, int v_begin, int v_end, int shares, int per, int skew,
                      int vocab, int n_top) {
  constexpr int kWarps = THREADS / 32, kPool = kWarps * 64;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sh.n_hits = sh.n_found = 0;
  uint32_t best = 0u;
  for (int c = 0; c < shares; ++c) {
    const uint32_t k = sort_desc((uint32_t)(make_key(sh.largest[c][tid], 0) >> 32), lane);
    best = c == 0 ? k : merge_lists(best, k, lane);
  }
  merge_warps<kWarps>(sh.maxima, best);
  const uint32_t lowest = sh.maxima[0][n_top - 1];
  for (int c = 0; c < shares; ++c)
    if ((uint32_t)(make_key(sh.largest[c][tid], 0) >> 32) >= lowest)
      sh.hits[atomicAdd(&sh.n_hits, 1)] = (uint16_t)(c * THREADS + tid);
  __syncthreads();
  // all that reaches the threshold in one row, as far as there is room: usually a few more
  // than n_top, which one warp sorts
  const float thr = key_value((u64)lowest << 32);
  u64* const pool = &sh.wait[0][0];
  read_again<THREADS>(sh, x, v_begin, v_end, per, skew, vocab, thr, [&](u64 k, bool in) {
    const uint32_t all = __ballot_sync(0xffffffffu, in);
    int at = 0;
    if (lane == 0) at = atomicAdd(&sh.n_found, __popc(all));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(all & ((1u << lane) - 1));
    if (in && at < kPool) pool[at] = k;
  });
  __syncthreads();
  const int found = sh.n_found;
  Top top;
  if (found <= kPool) {
    const int n = found <= 96 ? 1 : kWarps;  // warps at work
    if (warp < n)
      for (int b = warp * 32; b < found; b += 32 * n)
        top.best = merge_lists(top.best, sort_desc(b + lane < found ? pool[b + lane] : 0ull, lane), lane);
    if (n == 1) {
      if (warp == 0) sh.lists[0][lane] = top.best;
      __syncthreads();
      return;
    }
  } else {  // many equal logits, or all the large ones with few threads: list by list
    __syncthreads();  // the pool is each warp's own from here on
    read_again<THREADS>(sh, x, v_begin, v_end, per, skew, vocab, thr, [&](u64 k, bool reaches) {
      const bool in = reaches && k > top.last;
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      if (in) sh.wait[warp][top.n + __popc(all & ((1u << lane) - 1))] = k;
      top.n += __popc(all);
      if (top.n >= 32) take_in(top, sh.wait[warp], lane, n_top);
    });
    if (top.n > 0) take_in(top, sh.wait[warp], lane, n_top);
  }
  merge_warps<kWarps>(sh.lists, top.best);
}

// A cluster of gridDim.x CTAs per row, gridDim.y rows. TOP: alternatives are wanted.
template <bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kSmall ? 4 : 1) logprob_kernel(const LogprobParams p) {
  constexpr int kWarps = THREADS / 32;
  __shared__ LpShared<THREADS> sh;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;
  const float* x = p.logits + (int64_t)row * p.row_stride;
  // the row in 16-byte pieces: piece v holds the logits 4 v - skew .. 4 v - skew + 3
  const int skew = (int)(((uintptr_t)x >> 2) & 3);
  const int n_vec = (int)(((int64_t)p.vocab + skew + 3) >> 2);
  const int per = (n_vec + ranks - 1) / ranks;
  const int v_end = min(n_vec, (rank + 1) * per);
  const float c = 1.4426950408889634f / p.temperature;
  float next[4 * kVecs];  // the tile after the one at work: its loads are in flight meanwhile
  load_tile<THREADS>(x, rank * per, v_end, skew, p.vocab, next);
  const float x_target = rank == 0 && tid == 0 && p.targets && p.targets[row] >= 0 && p.targets[row] < p.vocab
                             ? x[p.targets[row]]
                             : __uint_as_float(0x7fc00000u);

  Stat st = {kLowest, 0.f, 0.f};
  float largest = -INFINITY;  // of the share at work
  const int tiles = max((v_end - rank * per + THREADS * kVecs - 1) / (THREADS * kVecs), 1);
  // at least 8 tiles: more shares cost more sorting than they save reading (64 rows of
  // 262,144 logits, 8 tiles a CTA: 18.4 us as one share, 23.8 us as eight)
  const int share_tiles = max((tiles + shares_of(THREADS) - 1) / shares_of(THREADS), 8);
  int share = 0, left = share_tiles;
  for (int v0 = rank * per; v0 < v_end; v0 += THREADS * kVecs) {
    float f[4 * kVecs];
#pragma unroll
    for (int k = 0; k < 4 * kVecs; ++k) f[k] = next[k];
    if (v0 + THREADS * kVecs < v_end) load_tile<THREADS>(x, v0 + THREADS * kVecs, v_end, skew, p.vocab, next);
    float mx = f[0];
#pragma unroll
    for (int k = 1; k < 4 * kVecs; ++k) mx = fmaxf(mx, f[k]);
    if (TOP) {
      largest = fmaxf(largest, mx);
      if (--left == 0) {
        sh.largest[share++][tid] = largest;
        left = share_tiles;
        largest = -INFINITY;
      }
    }
    if (mx > st.m) {
      const float d0 = fmaxf((st.m - mx) * c, kFar), w = ex2(d0);
      st.e = (st.e + d0 * st.l) * w;
      st.l *= w;
      st.m = mx;
    }
#pragma unroll
    for (int k = 0; k < 4 * kVecs; ++k) {
      const float d = (f[k] - st.m) * c;
      const float w = ex2(d);
      st.l += w;
      st.e = fmaf(w, fmaxf(d, kFar), st.e);
    }
  }
  // not earlier: the next kernel's CTAs would gather on the SMs that finish first
  pdl_launch_dependents();
  if (TOP) {
    if (left < share_tiles || share == 0) sh.largest[share++][tid] = largest;
    find_top(sh, x, rank * per, v_end, share, min(share_tiles, tiles) * kVecs, skew, p.vocab, p.n_top);
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
  if (warp == 0) {
    st = lane < kWarps ? sh.warp_stat[lane] : Stat{kLowest, 0.f, 0.f};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      Stat b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.l, o),
                __shfl_xor_sync(0xffffffffu, st.e, o)};
      st = stat_join(st, b, c);
    }
    if (lane == 0) sh.stat = st;
  }
  if (ranks > 1) {
    cluster_sync();  // every rank's list and statistics are written
    if (rank == 0) {
      u64 best = 0ull;
      if (TOP && warp < ranks) best = ld_peer_u64(peer_addr(&sh.lists[0][lane], warp));
      if (warp == 0) {  // a lane per rank
        Stat b = {kLowest, 0.f, 0.f};
        if (lane < ranks)
          b = {ld_peer_f32(peer_addr(&sh.stat.m, lane)), ld_peer_f32(peer_addr(&sh.stat.l, lane)),
               ld_peer_f32(peer_addr(&sh.stat.e, lane))};
#pragma unroll
        for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
          const Stat a = {__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.l, o),
                          __shfl_xor_sync(0xffffffffu, b.e, o)};
          b = stat_join(b, a, c);
        }
        __syncwarp();
        if (lane == 0) sh.stat = b;
      }
      if (TOP) {
        __syncthreads();  // lists[0] of this CTA is read before lists[] is reused
        merge_warps<kMaxCluster>(sh.lists, best);
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
    // NaNs among the logits may leave fewer than n_top candidates: stay inside the row
    if (p.top_ids) p.top_ids[at] = k ? key_index(k) : 0;
    if (p.top_logprobs)
      p.top_logprobs[at] = (k ? key_value(k) - all.m : __uint_as_float(0x7fc00000u)) / p.temperature - ln;
  }
}

template <int THREADS>
cudaError_t launch_rows(const LogprobParams& p, int ranks, cudaStream_t st) {
  const dim3 grid(ranks, p.rows);
  // many rows fill the GPU: CTAs that arrive while the kernel before ends gather on the SMs
  // that it leaves first (256 rows of 262,144 logits: 44.6 us against 42.1)
  constexpr bool pdl = THREADS == kLarge;
  return p.n_top ? launch_pdl(logprob_kernel<true, THREADS>, grid, THREADS, 0, st, pdl, ranks, p)
                 : launch_pdl(logprob_kernel<false, THREADS>, grid, THREADS, 0, st, pdl, ranks, p);
}

}  // namespace

cudaError_t q4g::launch_logprobs(const LogprobParams& p, cudaStream_t st) {
  // Few rows: clusters of CTAs of 1024 threads, an SM each, so that a row's loads are all
  // in flight within a few tiles (three quarters of the SMs: more clusters do not fit on the
  // GPU at once, 16 rows as 16 clusters of 8 took 22 us, as clusters of 4 they take 12). Many:
  // CTAs of 256 threads, four on every SM at most, the number that fits: one wave, 42 us for
  // 256 rows of 262,144 logits against 47 with up to six. The edges of that rule, rows of 32,003:
  // 296 rows with two CTAs each 8.6 us, 297 with one 8.9 (with 8 alternatives 13.0 and 12.3);
  // 592 rows, one wave, 12.0, 600 rows 14.2 (15.4 and 19.7).
  const int sms = device_sm_count();
  const bool large = (int64_t)p.rows * kMaxCluster <= sms && p.vocab > 2 * tile_of(kSmall);
  const int64_t tiles = ((int64_t)p.vocab + tile_of(large ? kLarge : kSmall) - 1) / tile_of(large ? kLarge : kSmall);
  const int64_t most = large ? sms * 3 / 4 : 4 * sms;
  int ranks = 1;
  while (ranks < kMaxCluster && 2 * p.rows * (int64_t)ranks <= most && 2 * ranks <= tiles) ranks *= 2;
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
    const cudaError_t e = large ? launch_rows<kLarge>(q, ranks, st) : launch_rows<kSmall>(q, ranks, st);
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
