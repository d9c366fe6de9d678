// Flash-decode of a batch whose sequences share a prefix (q4g_flash_decode_shared).
//
// Per KV head the queries of all sequences form one matrix Q [rows][hd], so a prefix
// row is read once for up to 64 query rows. The products run on the tensor cores
// transposed, the keys as the wide dimension:
//   S^T [128 keys][n rows] = K Q^T        (K tile as it lies in memory, k = hd)
//   O^T [hd][n rows]      += V^T P^T      (V tile as it lies in memory, k = keys)
// with n = 16..64 query rows. Single-token rows are few, and M = 128 is then full of
// keys or value dimensions instead of padding; O^T of hd 512 takes 256 tensor-memory
// columns and leaves room for two S^T; and a key's int8 scales belong to one thread
// (a lane of tensor memory is a key): the K scale multiplies its scores, the V scale
// its probabilities, the codes enter the products as exact fp16 integers.
//
// Softmax: a column (query row) has a reference exponent that the probabilities are
// taken against, 2^(s log2 e - ref + 7); it is raised, and the sums and O^T rescaled,
// only when a tile's maximum passes it by 8, so weights stay below 2^15 and rescaling
// is rare. Probabilities (times the V scale) are rounded to fp16 for the second
// product, 2^-11 relative as the fp16 output itself; sums and O^T are fp32. With int8
// rows the reference covers the weight p * scale, not p, so no scale overflows fp16.
//
// Work: the (unit, 128-key tile) pairs of the whole call in one line, cut into equal
// contiguous pieces, one per CTA (one CTA per SM). A unit is a row group of a KV head
// over the prefix, or a sequence's heads over its own rows; a piece of a unit leaves
// one partial (reference, sum, O) and a second kernel joins each row's partials. A
// unit u and a CTA c meet at most once and both only grow along the line, so u + c
// numbers the partials without any table, on both sides.
//
// Bound by HBM up to about 190 rows per key read (a 128-key tile of hd 512 is 256 KB,
// about 11,000 cycles of an SM's share of HBM, against 3,000 cycles of products for 64
// rows); by the tensor cores' shared-memory operands above that.
#include <cuda.h>
#include <math.h>

#include <mutex>

#include "../../include/q4g.h"
#include "q4g_common.cuh"
#include "q4g_internal.h"
#include "q4g_tc.cuh"

using namespace q4g;

namespace {

constexpr int kTileKeys = 128;
constexpr int kGroupRows = 64;   // query rows of one unit, at most
constexpr int kMaxBatch = 256;
constexpr int kSoftmaxThreads = 256;
constexpr int kSoftmaxWarps = 8;
constexpr int kConvertWarps = 8;  // in two groups that take turns at the ring's items
constexpr float kHeadroom = 8.f;  // a tile may pass the reference by 2^8
constexpr float kOffset = 7.f;    // probabilities are scaled by 2^7: 2^15 at most
constexpr float kLog2e = 1.4426950408889634f;

struct SharedParams {
  const __half* q;
  const float* ks[2];  // int8 rows: K and V scales, [0] the prefix's, [1] the sequences' own
  const float* vs[2];
  int64_t prefix;
  int32_t own_cap;
  const int32_t* own_len;
  int32_t batch, n_q, n_kv, G;  // G = n_q / n_kv
  int32_t groups, own_groups;   // row groups of a KV head: over the prefix, over own rows
  int32_t rows, own_rows;       // query rows that a partial of either kind holds
  int32_t ctas;
  // partials: (reference, sum) per row, then O per row; the prefix units' slots, then the own units'
  float *ml, *acc, *own_ml, *own_acc;
  __half* out;
  int32_t* err;
  uint64_t wait_ns;
};

struct alignas(64) SharedMaps {
  CUtensorMap k, v, own_k, own_v;
};

// ------------------------------------------------------------- the work line ----
// A unit takes its tiles and kUnitCost places before them: starting one (its queries,
// the first tile's latency, the partial) costs about as long as kUnitCost tiles.
constexpr int kUnitCost = 1;
Q4G_DEV int64_t places(int64_t tiles) { return tiles > 0 ? tiles + kUnitCost : 0; }

struct Line {
  int64_t prefix, total;      // places of one prefix unit; of the whole call
  const int32_t* own_places;  // [batch + 1] places of one KV head's own rows, summed up
  int32_t ctas;               // pieces of the line: no more than places, so that none is empty
};

struct Segment {
  int own, b, h, row0, n_rows;
  int64_t key0, key_end;  // keys [key0, key_end) of the unit's rows
  int32_t tiles;
  int64_t slot;
};

// Divisions of 64 bits take some hundred instructions: only calls beyond 2^32 pay them.
Q4G_DEV int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
Q4G_DEV int64_t line_begin(const Line& w, int c) { return quotient(w.total * min(c, w.ctas), max(w.ctas, 1)); }
Q4G_DEV int line_cta(const Line& w, int64_t t) { return (int)quotient((t + 1) * w.ctas - 1, w.total); }

Q4G_DEV int own_len_of(const SharedParams& p, int b) {
  return p.own_cap > 0 ? min(max(p.own_len[b], 0), p.own_cap) : 0;
}

// The part of the places [t, end) that lies in the unit of place t; moves t behind it.
// tiles = 0: nothing but places before the unit's first tile.
Q4G_DEV Segment next_segment(const SharedParams& p, const Line& w, int64_t& t, int64_t end, int cta) {
  Segment s;
  const int64_t in_prefix = (int64_t)p.n_kv * p.groups * w.prefix;
  int64_t j, len, n;
  if (t < in_prefix) {
    const int64_t u = quotient(t, w.prefix);
    j = t - u * w.prefix;
    n = w.prefix;
    len = p.prefix;
    s.own = 0, s.b = 0;
    s.h = (int)quotient(u, p.groups);
    s.row0 = (int)(u - (int64_t)s.h * p.groups) * kGroupRows;
    s.n_rows = min(kGroupRows, p.batch * p.G - s.row0);
    s.slot = u + cta;
  } else {
    const int per = p.n_kv * p.own_groups;
    const int64_t x = t - in_prefix;
    int lo = 0, hi = p.batch - 1;  // the last sequence that starts at or before x: it is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)w.own_places[mid] * per <= x) lo = mid;
      else hi = mid - 1;
    }
    s.b = lo;
    n = w.own_places[lo + 1] - w.own_places[lo];
    const int64_t y = x - (int64_t)w.own_places[lo] * per;
    const int u = (int)quotient(y, n);
    j = y - (int64_t)u * n;
    len = own_len_of(p, lo);
    s.own = 1;
    s.h = u / p.own_groups;
    s.row0 = (u % p.own_groups) * kGroupRows;
    s.n_rows = min(kGroupRows, p.G - s.row0);
    s.slot = (int64_t)lo * per + u + cta;
  }
  const int64_t e = min(n, j + end - t);
  t += e - j;
  const int64_t first = max(j - kUnitCost, (int64_t)0);
  s.tiles = (int32_t)max(e - kUnitCost - first, (int64_t)0);
  s.key0 = first * kTileKeys;
  s.key_end = min(len, s.key0 + (int64_t)s.tiles * kTileKeys);
  return s;
}

// own_places[0..batch], by one warp.
Q4G_DEV void sum_own_places(const SharedParams& p, int32_t* own_places, int lane) {
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    int v = b < p.batch ? (int)places((own_len_of(p, b) + kTileKeys - 1) / kTileKeys) : 0;
    const int mine = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (b < p.batch) own_places[b] = base + v - mine;
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) own_places[p.batch] = base;
}

Q4G_DEV Line make_line(const SharedParams& p, const int32_t* own_places) {
  Line w;
  w.prefix = places((p.prefix + kTileKeys - 1) / kTileKeys);
  w.own_places = own_places;
  w.total = (int64_t)p.n_kv * p.groups * w.prefix + (int64_t)own_places[p.batch] * p.n_kv * p.own_groups;
  w.ctas = (int)min((int64_t)p.ctas, w.total);
  return w;
}

// ------------------------------------------------------------- shared memory ----
// A ring stage holds 128 keys x 128 columns of K or V in fp16, as two swizzled slabs of
// 64 columns. int8 rows arrive in a second ring of 16 KB stages and are widened into it.
template <int HD, bool I8>
struct Plan {
  static constexpr int kStages = I8 ? 3 : (HD == 512 ? 4 : 5);
  static constexpr int kCodeStages = I8 ? (HD == 512 ? 2 : 4) : 0;
  static constexpr int kThreads = 32 * (4 + kSoftmaxWarps + (I8 ? kConvertWarps : 0));
  static constexpr int kSlab = kTileKeys * 128;            // bytes of a 64-column slab
  static constexpr int kStage = 2 * kSlab;
  static constexpr int kCodeStage = kTileKeys * 128;
  static constexpr int kQSlab = kGroupRows * 128;
  static constexpr int kQ = 0;
  static constexpr int kP = kQ + HD / 64 * kQSlab;
  static constexpr int kPBytes = kTileKeys * 128;            // P^T of a tile; two of them
  static constexpr int kRing = kP + 2 * kPBytes;
  static constexpr int kCodes = kRing + kStages * kStage;
  static constexpr int kState = kCodes + kCodeStages * kCodeStage;
};

struct State {
  float wmax[4][kGroupRows];  // per key quarter: a tile's column maxima; at the end column sums
  float ref[kGroupRows];
  float factor[kGroupRows];
  int32_t own_places[kMaxBatch + 1];
  uint32_t tmem;
  uint64_t full[5], empty[5], code_full[5], code_empty[5];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], q_ready, drain;
  volatile int abort;
};

template <int HD, bool I8>
constexpr size_t smem_bytes() {
  return Plan<HD, I8>::kState + sizeof(State);
}
static_assert(smem_bytes<512, false>() <= 232448 && smem_bytes<512, true>() <= 232448 &&
                  smem_bytes<256, false>() <= 232448 && smem_bytes<256, true>() <= 232448,
              "227 KB of shared memory");

// Bounded wait; a wait that gives up, here or elsewhere in the CTA, ends every role.
// (mbar_try_wait sleeps; spinning instead took issue slots from the products: +10%.)
Q4G_DEV bool wait(State& sh, const SharedParams& p, uint64_t* bar, uint32_t phase) {
  if (mbar_try_wait(bar, phase)) return true;
  const uint64_t t0 = global_ns();
  for (int it = 0; it < kSpinLimit; ++it) {
    if (mbar_try_wait(bar, phase)) return true;
    if (sh.abort) return false;
    if (global_ns() - t0 > p.wait_ns) break;
  }
  sh.abort = 1;
  atomicOr(p.err, 1);
  return false;
}
// The same for a warp: all lanes agree.
Q4G_DEV bool wait_warp(State& sh, const SharedParams& p, uint64_t* bar, uint32_t phase) {
  return __all_sync(0xffffffffu, wait(sh, p, bar, phase));
}

Q4G_DEV void softmax_sync() { asm volatile("barrier.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); }
Q4G_DEV bool softmax_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.red.or.pred b, 1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kSoftmaxThreads)
      : "memory");
  return r != 0;
}
Q4G_DEV float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
Q4G_DEV float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Lane i's result is the sum of v[i] over the warp's lanes: halves change places with
// the lane 16, 8, ... away, 31 shuffles in place of 160.
Q4G_DEV float lane_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

// -------------------------------------------------------------------- roles ----
// Ring items in the order in which the products take them: per segment, in step i, the
// K parts of tile i, then the V parts of tile i - 1. One thread.
// (Asking L2 for the next tile as well, by prefetch copies, was slower at every length:
// 16 sequences on a 128K prefix 178 us without, 200 us with.)
template <int HD, bool I8>
Q4G_DEV void produce(const SharedParams& p, const SharedMaps& maps, unsigned char* smem, State& sh, const Line& w) {
  using P = Plan<HD, I8>;
  constexpr int NS = I8 ? P::kCodeStages : P::kStages;
  uint64_t* const full = I8 ? sh.code_full : sh.full;
  uint64_t* const empty = I8 ? sh.code_empty : sh.empty;
  const int64_t end = line_begin(w, blockIdx.x + 1);
  uint32_t st = 0, phase = 1;  // the phase bit before a stage's first use: that wait is over at once
  uint32_t it = 0;
  bool ok = true;
  for (int64_t t = line_begin(w, blockIdx.x); t < end && ok;) {
    const Segment s = next_segment(p, w, t, end, blockIdx.x);
    if (s.tiles == 0) continue;
    for (int i = 0; i <= s.tiles && ok; ++i) {
      for (int part = 0; part < 2 && ok; ++part) {
        const int j = i - part;
        if (j < 0 || j >= s.tiles) continue;
        const void* const map = s.own ? (part ? &maps.own_v : &maps.own_k) : (part ? &maps.v : &maps.k);
        const int key = (int)s.key0 + j * kTileKeys;
        for (int c = 0; c < HD / 128; ++c, ++it) {
          if (!(ok = wait(sh, p, &empty[st], phase))) break;
          unsigned char* dst = smem + (I8 ? P::kCodes + st * P::kCodeStage : P::kRing + st * P::kStage);
          mbar_arrive_expect_tx(&full[st], I8 ? P::kCodeStage : P::kStage);
#pragma unroll
          for (int half = 0; half < (I8 ? 1 : 2); ++half, dst += P::kSlab) {
            const int x = c * 128 + half * 64;
            if (s.own) tma_load_4d(dst, map, x, s.h, key, s.b, &full[st]);
            else tma_load_3d(dst, map, x, s.h, key, &full[st]);
          }
          if (++st == NS) st = 0, phase ^= 1;
        }
      }
    }
  }
  // Given up: the copies in flight still write this CTA's shared memory. Each is the last
  // of its stage, so its phase stays.
  if (!ok)
    for (uint32_t k = it > NS ? it - NS : 0; k < it; ++k) mbar_wait_bounded(&full[k % NS], (k / NS) & 1, p.wait_ns);
}

// All products, by one thread.
template <int HD, bool I8>
Q4G_DEV void multiply(const SharedParams& p, unsigned char* smem, State& sh, const Line& w) {
  using P = Plan<HD, I8>;
  constexpr int NS = P::kStages, C = HD / 128;
  const uint32_t ring = smem_u32(smem) + P::kRing, q = smem_u32(smem) + P::kQ, pr = smem_u32(smem) + P::kP;
  const uint32_t s_col = sh.tmem, o_col = sh.tmem + 2 * kGroupRows;
  const int64_t end = line_begin(w, blockIdx.x + 1);
  uint32_t st = 0, phase = 0, tile = 0, seg = 0;
  bool ok = true;
  for (int64_t t = line_begin(w, blockIdx.x); t < end && ok;) {
    const Segment s = next_segment(p, w, t, end, blockIdx.x);
    if (s.tiles == 0) continue;
    const uint32_t n = (s.n_rows + 15) & ~15;
    const uint32_t id_s = tc_idesc_f16(n, false, false), id_o = tc_idesc_f16(n, true, true);
    if (!(ok = wait(sh, p, &sh.q_ready, seg & 1))) break;
    ++seg;
    // Step i: S^T of tile i, then O^T += V^T P^T of tile i - 1, whose softmax ran while S^T
    // of tile i was made. (Part by part in turn, with a tile more between the two, was 7%
    // slower on 16 sequences and a 32K prefix: every part then pays the wait for its load.)
    for (int i = 0; i <= s.tiles && ok; ++i) {
      if (i < s.tiles) {
        const uint32_t g = tile + i, s_at = s_col + (g & 1) * kGroupRows;
        if (g >= 2 && !(ok = wait(sh, p, &sh.s_free[g & 1], (g / 2 - 1) & 1))) break;
        for (int c = 0; c < C; ++c) {
          if (!(ok = wait(sh, p, &sh.full[st], phase))) break;
          tc_fence_after();
          const uint32_t a = ring + st * P::kStage, b = q + 2 * c * P::kQSlab;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_f16(s_at, tc_desc(a + (k >> 2) * P::kSlab + (k & 3) * 32, 0),
                       tc_desc(b + (k >> 2) * P::kQSlab + (k & 3) * 32, 0), id_s, c > 0 || k > 0);
          tc_commit(&sh.empty[st]);
          if (++st == NS) st = 0, phase ^= 1;
        }
        if (!ok) break;
        tc_commit(&sh.s_full[g & 1]);
      }
      if (i > 0) {
        const uint32_t g = tile + i - 1, pt = pr + (g & 1) * P::kPBytes;
        if (!(ok = wait(sh, p, &sh.p_full[g & 1], (g / 2) & 1))) break;
        // the live keys, rounded up to 16
        const int live = min(kTileKeys, (int)(s.key_end - s.key0) - (i - 1) * kTileKeys);
        const int steps = (live + 15) >> 4;
        for (int c = 0; c < C; ++c) {
          if (!(ok = wait(sh, p, &sh.full[st], phase))) break;
          if (!I8 && s.own && live < steps * 16) {
            // what lies behind a sequence's own rows may be anything, and zero times a NaN
            // is not zero
            for (int x = live * 8; x < steps * 128; ++x)
              for (int half = 0; half < 2; ++half)
                *reinterpret_cast<uint4*>(smem + P::kRing + st * P::kStage + half * P::kSlab + x * 16) =
                    make_uint4(0, 0, 0, 0);
            fence_async_smem();
          }
          tc_fence_after();
          const uint32_t a = ring + st * P::kStage, o_at = o_col + c * kGroupRows;
          if (steps == kTileKeys / 16) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc_mma_f16(o_at, tc_desc(a + k * 2048, P::kSlab), tc_desc(pt + k * 2048, 0), id_o, i > 1 || k > 0);
          } else {
            for (int k = 0; k < steps; ++k)
              tc_mma_f16(o_at, tc_desc(a + k * 2048, P::kSlab), tc_desc(pt + k * 2048, 0), id_o, i > 1 || k > 0);
          }
          tc_commit(&sh.empty[st]);
          if (++st == NS) st = 0, phase ^= 1;
        }
        if (!ok) break;
        tc_commit(&sh.pv_done[g & 1]);
      }
    }
    tile += s.tiles;
  }
  if (!ok) {  // given up: products in flight still use shared and tensor memory
    tc_commit(&sh.drain);
    mbar_wait_bounded(&sh.drain, 0, p.wait_ns);
  }
}

// int8 codes into fp16: with the sign bit flipped a code c is the byte c + 128, and the
// fp16 pattern 0x6400 | byte is 1024 + byte, so one subtraction gives c, exactly.
Q4G_DEV uint32_t widen2(uint32_t u, uint32_t sel) {
  const uint32_t h = __byte_perm(u, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kGroup = kConvertWarps / 2 * 32;

template <int HD>
Q4G_DEV void convert(const SharedParams& p, unsigned char* smem, State& sh, const Line& w) {
  using P = Plan<HD, true>;
  constexpr int NS = P::kStages, NC = P::kCodeStages, C = HD / 128;
  const int tid = threadIdx.x - 32 * (4 + kSoftmaxWarps), lane = tid & 31, group = tid / kGroup;
  const int64_t end = line_begin(w, blockIdx.x + 1);
  uint32_t items = 0;
  for (int64_t t = line_begin(w, blockIdx.x); t < end;) items += 2 * C * next_segment(p, w, t, end, blockIdx.x).tiles;
  for (uint32_t it = group; it < items; it += 2) {
    const uint32_t cs = it % NC, st = it % NS;
    if (!wait_warp(sh, p, &sh.code_full[cs], (it / NC) & 1)) return;
    if (it >= NS && !wait_warp(sh, p, &sh.empty[st], (it / NS - 1) & 1)) return;
    const unsigned char* const src = smem + P::kCodes + cs * P::kCodeStage;
    unsigned char* const dst = smem + P::kRing + st * P::kStage;
#pragma unroll 4
    for (int x = tid % kGroup; x < kTileKeys * 8; x += kGroup) {
      const int row = x >> 3, g = x & 7;  // 16 codes: columns 16 g of the row
      uint4 u = *reinterpret_cast<const uint4*>(src + x * 16);
      u.x ^= 0x80808080u, u.y ^= 0x80808080u, u.z ^= 0x80808080u, u.w ^= 0x80808080u;
      const uint4 a = make_uint4(widen2(u.x, 0x4140), widen2(u.x, 0x4342), widen2(u.y, 0x4140), widen2(u.y, 0x4342));
      const uint4 b = make_uint4(widen2(u.z, 0x4140), widen2(u.z, 0x4342), widen2(u.w, 0x4140), widen2(u.w, 0x4342));
      unsigned char* const out = dst + (g >> 2) * P::kSlab + row * 128;
      const int c0 = 2 * (g & 3), first = g >> 2;  // the two slabs' lanes store different chunks at a time
      *reinterpret_cast<uint4*>(out + (((c0 + first) ^ (row & 7)) * 16)) = first ? b : a;
      *reinterpret_cast<uint4*>(out + (((c0 + 1 - first) ^ (row & 7)) * 16)) = first ? a : b;
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh.full[st]);
      mbar_arrive(&sh.code_empty[cs]);
    }
  }
}

// One thread: a key of the tile (tensor-memory lane) and 32 of the 64 query rows.
template <int HD, bool I8>
Q4G_DEV void softmax(const SharedParams& p, unsigned char* smem, State& sh, const Line& w) {
  using P = Plan<HD, I8>;
  constexpr int C = HD / 128;
  const int tid = threadIdx.x - 128, lane = tid & 31, quarter = (tid >> 5) & 3, c0 = (tid >> 7) * 32;
  const int key = quarter * 32 + lane;
  const uint32_t lanes = sh.tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t s_col = lanes + c0, o_col = lanes + 2 * kGroupRows + c0;
  const int64_t end = line_begin(w, blockIdx.x + 1);
  uint32_t tile = 0;
  // once a wait has given up nothing waits any more, but every thread goes on to the end:
  // the barriers among these warps have no limit of their own
  bool ok = true;
  for (int64_t t = line_begin(w, blockIdx.x); t < end;) {
    const Segment s = next_segment(p, w, t, end, blockIdx.x);
    if (s.tiles == 0) continue;
    const int n = (s.n_rows + 15) & ~15;
    // the unit's query rows, zeros behind them; eight loads of a thread in flight. CTAs
    // start at different rows: most of them read the same ones at the same time
    constexpr int kRowsAtOnce = kSoftmaxThreads / (HD / 8);
    const int ch = tid % (HD / 8);
    const __half* const q_head = p.q + (int64_t)s.h * p.G * HD + ch * 8;
    unsigned char* const q_dst = smem + P::kQ + (ch >> 3) * P::kQSlab;
    const int turn = (blockIdx.x * 4) % n;
    const float inv_G = 1.0f / p.G;
    for (int r0 = tid / (HD / 8); r0 < n; r0 += 8 * kRowsAtOnce) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = r0 + i * kRowsAtOnce + turn;
        const int r = at < n ? at : at - n, rr = s.row0 + r;
        // rr / G: the quotient is off by less than 2^-23 of itself, rr < 2^18 and G <= 1024 put
        // (rr + 1/2) / G at least 2^-11 from a whole number while it is below 2^18 / G
        const int b = s.own ? s.b : (int)((rr + 0.5f) * inv_G), g = s.own ? rr : rr - b * p.G;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < s.n_rows && at - turn < n) v[i] = __ldg(reinterpret_cast<const uint4*>(q_head + ((int64_t)b * p.n_q + g) * HD));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = r0 + i * kRowsAtOnce + turn;
        const int r = at < n ? at : at - n;
        if (at - turn < n) *reinterpret_cast<uint4*>(q_dst + r * 128 + (((ch & 7) ^ (r & 7)) * 16)) = v[i];
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_ready);

    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.f;
    int left = (int)(s.key_end - s.key0) - key;  // this thread's key of the tile is live while left > 0
    const int64_t row0 = ((int64_t)s.b * p.own_cap + s.key0 + key) * p.n_kv + s.h;  // s.b = 0 over the prefix
    const float* ks_at = (s.own ? p.ks[1] : p.ks[0]) + row0;
    const float* vs_at = (s.own ? p.vs[1] : p.vs[0]) + row0;
    for (int j = 0; j < s.tiles; ++j, ++tile, left -= kTileKeys) {
      const bool live = left > 0;
      float ks = kLog2e, vs = 1.f, lift = 0.f;  // lift: log2 of the V scale, for the reference only
      if constexpr (I8) {
        ks = live ? __ldg(ks_at) * kLog2e : 0.f;
        vs = live ? __ldg(vs_at) : 0.f;
        lift = __log2f(fmaxf(fabsf(vs), 9.094947e-13f));  // 2^-40 at least
        ks_at += kTileKeys * p.n_kv;
        vs_at += kTileKeys * p.n_kv;
      }
      const uint32_t buf = tile & 1;
      ok = ok && wait_warp(sh, p, &sh.s_full[buf], (tile / 2) & 1);
      tc_fence_after();
      float x[32];
      const bool active = c0 < n;
      if (active) {
        tmem_ld32(s_col + buf * kGroupRows, x);
        tmem_wait_ld(x);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_free[buf]);
      if (active) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float m[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[i + e] = live ? x[i + e] * ks : -INFINITY;
            m[e] = warp_max_f32(x[i + e] + lift);
          }
          if (lane == 0)
            *reinterpret_cast<float4*>(&sh.wmax[quarter][c0 + i]) = make_float4(m[0], m[1], m[2], m[3]);
        }
      }
      softmax_sync();
      bool raise = false;
      if (tid < n) {
        const float m = fmaxf(fmaxf(fmaxf(sh.wmax[0][tid], sh.wmax[1][tid]), fmaxf(sh.wmax[2][tid], sh.wmax[3][tid])),
                              -1e30f);
        const float old = sh.ref[tid];
        raise = j > 0 && m > old + kHeadroom;
        sh.factor[tid] = raise ? ex2(old - m) : 1.f;
        if (j == 0 || raise) sh.ref[tid] = m;
      }
      raise = softmax_any(raise);
      if (raise) ok = ok && wait_warp(sh, p, &sh.pv_done[buf ^ 1], ((tile - 1) / 2) & 1);  // O^T is free
      else if (j >= 2) ok = ok && wait_warp(sh, p, &sh.pv_done[buf], (tile / 2 - 1) & 1);  // this P^T is free
      if (active) {
        if (raise) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 2 * C; ++c) {
            const int half = (c & 1) * 16;
            const uint32_t at = o_col + (c >> 1) * kGroupRows + half;
            float o[16];
            tmem_ld16(at, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= sh.factor[c0 + half + i];
            tmem_st16(at, o);
          }
          tmem_wait_st();
          tc_fence_before();
#pragma unroll
          for (int i = 0; i < 32; ++i) l[i] *= sh.factor[c0 + i];
        }
        unsigned char* const row = smem + P::kP + buf * P::kPBytes + key * 128;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 ref = *reinterpret_cast<const float2*>(&sh.ref[c0 + i + e]);
            const float a = ex2(x[i + e] - ref.x + kOffset), b = ex2(x[i + e + 1] - ref.y + kOffset);
            l[i + e] += a;
            l[i + e + 1] += b;
            const __half2 ab = I8 ? __floats2half2_rn(a * vs, b * vs) : __floats2half2_rn(a, b);
            h[e / 2] = *reinterpret_cast<const uint32_t*>(&ab);
          }
          *reinterpret_cast<uint4*>(row + ((((c0 + i) >> 3) ^ (key & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[buf]);
    }

    // the segment's partial
    ok = ok && wait_warp(sh, p, &sh.pv_done[(tile - 1) & 1], ((tile - 1) / 2) & 1);
    tc_fence_after();
    softmax_sync();  // wmax is free
    float* const ml = (s.own ? p.own_ml : p.ml) + s.slot * (s.own ? p.own_rows : p.rows) * 2;
    float* const acc = (s.own ? p.own_acc : p.acc) + s.slot * (s.own ? p.own_rows : p.rows) * HD;
    if (c0 < n) {
      sh.wmax[quarter][c0 + lane] = lane_sums(l, lane);
#pragma unroll 1
      for (int c = 0; c < C; ++c) {
        float o[32];
        tmem_ld32(o_col + c * kGroupRows, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c0 + i < s.n_rows) acc[(int64_t)(c0 + i) * HD + c * 128 + key] = o[i];
      }
    }
    tc_fence_before();
    softmax_sync();
    if (tid < s.n_rows) {
      ml[2 * tid] = sh.ref[tid];
      ml[2 * tid + 1] = sh.wmax[0][tid] + sh.wmax[1][tid] + sh.wmax[2][tid] + sh.wmax[3][tid];
    }
  }
}

template <int HD, bool I8>
__global__ void __launch_bounds__(Plan<HD, I8>::kThreads, 1)
    shared_kernel(const __grid_constant__ SharedMaps maps, const SharedParams p) {
  using P = Plan<HD, I8>;
  extern __shared__ __align__(1024) unsigned char smem[];
  State& sh = *reinterpret_cast<State*>(smem + P::kState);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    sum_own_places(p, sh.own_places, lane);
  } else if (warp == 1) {
    tmem_alloc(&sh.tmem, 512);
  } else if (warp == 2 && lane == 0) {
    for (int i = 0; i < 5; ++i) {
      mbar_init(&sh.full[i], I8 ? kConvertWarps / 2 : 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.code_full[i], 1);
      mbar_init(&sh.code_empty[i], kConvertWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], kSoftmaxWarps);
      mbar_init(&sh.p_full[i], kSoftmaxWarps);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.q_ready, kSoftmaxWarps);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Line w = make_line(p, sh.own_places);
  pdl_launch_dependents();  // the join's CTAs take the places that CTAs of this grid leave
  // With int8 rows 640 threads start with 96 registers each: the softmax warps take 136,
  // 4 x 32 x (56 + 2 x 136 + 2 x 72) = 472 x 128 of 480 x 128.
  if (warp < 4) {
    if constexpr (I8) regs_dec<56>();
    if (warp == 0) {
      if (elect_one()) produce<HD, I8>(p, maps, smem, sh, w);
      __syncwarp();
    } else if (warp == 1) {
      if (elect_one()) multiply<HD, I8>(p, smem, sh, w);
      __syncwarp();
    }
  } else if (warp < 4 + kSoftmaxWarps) {
    if constexpr (I8) regs_inc<136>();
    softmax<HD, I8>(p, smem, sh, w);
  } else {
    if constexpr (I8) {
      regs_dec<72>();
      convert<HD>(p, smem, sh, w);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, 512);
  }
}

// ------------------------------------------------------------------ the join ----
constexpr int kJoinThreads = 512;
constexpr int kJoinCols = 128;                          // output columns per CTA
constexpr int kJoinLanes = kJoinCols / 4;               // threads across them: a warp
constexpr int kJoinParts = kJoinThreads / kJoinLanes;   // threads down the partials: the warps
constexpr int kJoinMax = 2 * 256;                       // partials of a row: CTAs of its two units

// out[row] = sum_i 2^(ref_i - R) O_i / sum_i 2^(ref_i - R) l_i over the row's partials,
// R the largest reference; in a fixed order. Grid: query rows, columns / 128. The weights
// are made once, one thread a partial, so that the loads of O depend on nothing.
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const SharedParams p) {
  __shared__ int32_t own_places[kMaxBatch + 1];
  __shared__ float red[2][kJoinThreads / 32];
  __shared__ float weight[kJoinMax];
  __shared__ float4 part[kJoinParts][kJoinLanes];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) sum_own_places(p, own_places, lane);
  __syncthreads();
  const Line w = make_line(p, own_places);
  const int b = blockIdx.x / p.n_q, hq = blockIdx.x % p.n_q, h = hq / p.G, g = hq % p.G;
  __half* const out = p.out + (int64_t)blockIdx.x * HD + blockIdx.y * kJoinCols;
  // the partials of the row: slots [s0, s0 + n0) of the prefix, [s1, s1 + n1) of its own rows
  int64_t s0 = 0, s1 = 0;
  int n0 = 0, n1 = 0, r0 = 0, r1 = g % kGroupRows;
  if (w.prefix > 0) {
    const int rr = b * p.G + g;
    const int64_t u = (int64_t)h * p.groups + rr / kGroupRows, t = u * w.prefix;
    const int c = line_cta(w, t + kUnitCost);
    r0 = rr % kGroupRows;
    s0 = u + c;
    n0 = line_cta(w, t + w.prefix - 1) - c + 1;
  }
  const int own = own_places[b + 1] - own_places[b];
  if (own > 0) {
    const int per = p.n_kv * p.own_groups, u = h * p.own_groups + g / kGroupRows;
    const int64_t t = (int64_t)p.n_kv * p.groups * w.prefix + (int64_t)own_places[b] * per + (int64_t)u * own;
    const int c = line_cta(w, t + kUnitCost);
    s1 = (int64_t)b * per + u + c;
    n1 = line_cta(w, t + own - 1) - c + 1;
  }
  const int n = n0 + n1;
  // references, sums and weights, one partial a thread (n <= 2 * CTAs <= kJoinMax)
  const float* const ml0 = p.ml + (s0 * p.rows + r0) * 2;
  const float* const ml1 = p.own_ml + (s1 * p.own_rows + r1) * 2;
  float2 ml[kJoinMax / kJoinThreads];
  float R = -INFINITY;
  pdl_wait();  // all above comes from the call's own arguments
#pragma unroll
  for (int k = 0; k < kJoinMax / kJoinThreads; ++k) {
    const int i = tid + k * kJoinThreads;
    ml[k] = make_float2(-INFINITY, 0.f);
    if (i < n)
      ml[k] = *reinterpret_cast<const float2*>(i < n0 ? ml0 + (int64_t)i * p.rows * 2
                                                      : ml1 + (int64_t)(i - n0) * p.own_rows * 2);
    R = fmaxf(R, ml[k].x);
  }
  R = warp_max(R);
  if (lane == 0) red[0][warp] = R;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) R = fmaxf(R, red[0][i]);
  float l = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinMax / kJoinThreads; ++k) {
    const int i = tid + k * kJoinThreads;
    if (i < n) {
      const float f = ex2(ml[k].x - R);
      weight[i] = f;
      l += f * ml[k].y;
    }
  }
  l = warp_sum(l);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  const float* const acc0 = p.acc + (s0 * p.rows + r0) * HD + blockIdx.y * kJoinCols + lane * 4;
  const float* const acc1 = p.own_acc + (s1 * p.own_rows + r1) * HD + blockIdx.y * kJoinCols + lane * 4;
  const int64_t step0 = (int64_t)p.rows * HD, step1 = (int64_t)p.own_rows * HD;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 10
  for (int i = warp; i < n; i += kJoinParts) {
    const float4 a = *reinterpret_cast<const float4*>(i < n0 ? acc0 + i * step0 : acc1 + (i - n0) * step1);
    const float f = weight[i];
    o.x += f * a.x, o.y += f * a.y, o.z += f * a.z, o.w += f * a.w;
  }
  part[warp][lane] = o;
  __syncthreads();
  if (warp == 0) {
    l = red[1][0];
#pragma unroll
    for (int i = 1; i < kJoinParts; ++i) {
      const float4 a = part[i][lane];
      l += red[1][i];
      o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
    }
    const float inv = n > 0 ? 1.f / l : 0.f;  // no key at all: zeros
    const __half2 lo = __floats2half2_rn(o.x * inv, o.y * inv), hi = __floats2half2_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(out + lane * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// -------------------------------------------------------------------- host ----
q4g_status bad(q4g_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once; NULL if the driver has none.
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeTiled)f;
  }();
  return fn;
}

// Rows [batch][rows][n_kv][hd] of fp16 or codes; a box is 128 keys of one KV head and 64
// fp16 columns (swizzled) or 128 codes. Keys past `rows` read as zeros. batch 0: [rows][n_kv][hd].
bool encode(CUtensorMap* m, const void* base, int hd, int n_kv, int64_t rows, int batch, bool i8) {
  const cuuint64_t e = i8 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)hd, (cuuint64_t)n_kv, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {hd * e, (cuuint64_t)n_kv * hd * e, (cuuint64_t)rows * n_kv * hd * e};
  const cuuint32_t box[4] = {i8 ? 128u : 64u, 1, kTileKeys, 1}, one[4] = {1, 1, 1, 1};
  return encode_tiled()(m, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, batch ? 4 : 3,
                        const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        i8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

template <int HD, bool I8>
cudaError_t launch(const SharedMaps& maps, const SharedParams& p, cudaStream_t st) {
  static std::mutex mu;
  static bool configured[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(shared_kernel<HD, I8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem_bytes<HD, I8>());
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  shared_kernel<HD, I8><<<p.ctas, Plan<HD, I8>::kThreads, smem_bytes<HD, I8>(), st>>>(maps, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.batch * p.n_q, HD / kJoinCols);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_join_kernel<HD>, p);
}

// Units, partial slots and the scratch layout; returns its bytes.
size_t plan_scratch(SharedParams& p, int hd, void* ws) {
  p.G = p.n_q / p.n_kv;
  const int rows = p.batch * p.G;
  p.groups = (rows + kGroupRows - 1) / kGroupRows;
  p.own_groups = (p.G + kGroupRows - 1) / kGroupRows;
  p.rows = rows < kGroupRows ? rows : kGroupRows;
  p.own_rows = p.G < kGroupRows ? p.G : kGroupRows;
  p.ctas = device_sm_count() < kJoinMax / 2 ? device_sm_count() : kJoinMax / 2;
  const size_t n = ((size_t)p.n_kv * p.groups + p.ctas) * p.rows;
  const size_t n_own = ((size_t)p.batch * p.n_kv * p.own_groups + p.ctas) * p.own_rows;
  size_t off = 0;
  auto take = [&](size_t floats) {
    float* at = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + off);
    off += (floats * sizeof(float) + 255) & ~(size_t)255;
    return at;
  };
  p.ml = take(2 * n);
  p.own_ml = take(2 * n_own);
  p.acc = take(n * hd);
  p.own_acc = take(n_own * hd);
  return off;
}

q4g_status check_heads(int32_t batch, int32_t n_q, int32_t n_kv, int32_t hd) {
  if (hd != 256 && hd != 512) return bad(Q4G_EINVAL, "head_dim must be 256 or 512");
  if (n_q < 1 || n_kv < 1 || n_q % n_kv || n_q > 1024)
    return bad(Q4G_EINVAL, "n_q must be a positive multiple of n_kv, at most 1024");
  if (batch < 1 || batch > kMaxBatch) return bad(Q4G_ERANGE, "batch outside [1, 256]");
  return Q4G_OK;
}

q4g_status run_shared(const uint16_t* q, int32_t batch, int32_t n_q, int32_t n_kv, int32_t hd, const void* kp,
                      const float* kps, const void* vp, const float* vps, int64_t prefix, const void* ko,
                      const float* kos, const void* vo, const float* vos, int64_t own_cap, const int32_t* own_len,
                      uint16_t* out, void* ws, size_t ws_bytes, bool i8, cudaStream_t st) {
  q4g_status s = check_heads(batch, n_q, n_kv, hd);
  if (s) return s;
  if (prefix < 0 || prefix > ((int64_t)1 << 30)) return bad(Q4G_ERANGE, "prefix_len outside [0, 2^30]");
  if (own_cap < 0 || own_cap > (1 << 24) || own_cap * batch > ((int64_t)1 << 30))
    return bad(Q4G_ERANGE, "own_capacity outside [0, 2^24] or batch * own_capacity above 2^30");
  // absent parts take no part in the checks
  if (prefix == 0) kp = vp = nullptr, kps = vps = nullptr;
  if (own_cap == 0) ko = vo = nullptr, kos = vos = nullptr, own_len = nullptr;
  if (!q || !out || !ws) return bad(Q4G_EINVAL, "NULL pointer");
  if (prefix > 0 && (!kp || !vp || (i8 && (!kps || !vps)))) return bad(Q4G_EINVAL, "prefix rows: NULL pointer");
  if (own_cap > 0 && (!ko || !vo || !own_len || (i8 && (!kos || !vos))))
    return bad(Q4G_EINVAL, "own rows: NULL pointer");
  const void* ptrs[] = {q, kp, vp, ko, vo, out, ws, kps, vps, kos, vos, own_len};
  const size_t align[] = {16, 16, 16, 16, 16, 16, 256, 4, 4, 4, 4, 4};
  for (int i = 0; i < 12; ++i)
    if (!aligned(ptrs[i], align[i])) return bad(Q4G_EINVAL, "misaligned pointer");
  SharedParams p{};
  p.batch = batch, p.n_q = n_q, p.n_kv = n_kv;
  if (plan_scratch(p, hd, ws) > ws_bytes) return bad(Q4G_EINVAL, "workspace too small");
  for (const void* x : ptrs)
    if (x && !on_current_device(x)) return bad(Q4G_EINVAL, "a pointer is not memory of the current device");
  if (!encode_tiled()) return bad(Q4G_ECUDA, "the driver has no tensor maps");
  p.q = reinterpret_cast<const __half*>(q);
  p.ks[0] = kps, p.ks[1] = kos, p.vs[0] = vps, p.vs[1] = vos;
  p.prefix = prefix;
  p.own_cap = (int32_t)own_cap;
  p.own_len = own_len;
  p.out = reinterpret_cast<__half*>(out);
  p.wait_ns = 2000000000ull;
  if (!(p.err = device_error_word())) return bad(Q4G_ECUDA, "error word unavailable");
  SharedMaps maps{};
  bool ok = true;
  if (prefix > 0) ok = encode(&maps.k, kp, hd, n_kv, prefix, 0, i8) && encode(&maps.v, vp, hd, n_kv, prefix, 0, i8);
  if (own_cap > 0)
    ok = ok && encode(&maps.own_k, ko, hd, n_kv, own_cap, batch, i8) &&
         encode(&maps.own_v, vo, hd, n_kv, own_cap, batch, i8);
  if (!ok) return bad(Q4G_ECUDA, "tensor map refused by the driver");
  cudaError_t e;
  if (hd == 512) e = i8 ? launch<512, true>(maps, p, st) : launch<512, false>(maps, p, st);
  else e = i8 ? launch<256, true>(maps, p, st) : launch<256, false>(maps, p, st);
  return e == cudaSuccess ? Q4G_OK : bad(Q4G_ECUDA, cudaGetErrorString(e));
}

}  // namespace

extern "C" size_t q4g_flash_decode_shared_workspace_bytes(int32_t batch, int32_t n_q, int32_t n_kv,
                                                          int32_t head_dim) {
  if (batch < 1 || n_q < 1 || n_kv < 1 || head_dim < 1 || n_q < n_kv) return 256;
  SharedParams p{};
  p.batch = batch, p.n_q = n_q, p.n_kv = n_kv;
  return plan_scratch(p, head_dim, nullptr);
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
