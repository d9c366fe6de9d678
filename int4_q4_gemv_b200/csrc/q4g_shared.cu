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
// is rare. Probabilities (times the V scale) enter the second product as fp16 hi + lo,
// 2^-22 relative, as in the one-sequence kernels: one fp16 each would put an error of the
// size of the fp16 output's own rounding on top of it. Sums and O^T are fp32. With int8
// rows the reference covers the weight p * scale, not p, so no scale overflows fp16.
//
// Work: a unit is a row group of a KV head over the prefix, or a sequence's heads over
// its own rows. Prefix units are cut into equally many pieces, so that the CTAs that
// read the same keys for different row groups do so at the same time and share them
// through L2 (cut as one line over all units they drifted apart, and 16 sequences on a
// 128K prefix read HBM four times over: 1.08 GB, 167 us). Own units are cut as a line of
// 128-key tiles over the CTAs, those without a prefix piece first. Every piece leaves one
// partial (reference, sum, O), and a second kernel joins each row's partials.
//
// Bound by HBM for one row group: a 128-key tile of hd 512 is 256 KB, 5.6 us of an SM's
// share of HBM (4 sequences of 16 heads on a 128K prefix: 56 us, 4.8 TB/s). With more, the
// products of a tile and 64 rows take 64 x 48 cycles, 1.6 us (a product with M = 128 reads
// 4 KB of A from shared memory, whatever n up to 64) for hi and 32 x 48 more for lo, 2.4 us,
// and the parts of V stay in the ring of 128 KB that much longer: a tile takes 4.1 us (16
// sequences: 131 us, or 158 at the 1.6 GHz that the power limit leaves to a run of seconds;
// with hi alone 103 and 126, at 1.4 times the error of the output's own rounding). Small calls
// are a chain of latencies: two sequences on 100 rows take 11.4 us, 8 on 4096 rows 15.2, of
// which about 3.4 are writing and joining 128 KB of partials a CTA.
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
constexpr int kConvertWarps = 12;  // int8 rows: a group of four for K parts, two that take turns for V parts
// Tensor memory columns: two S^T of 64, O^T, and for int8 rows two K parts of 128 x 128 fp16.
constexpr int kKeyCol = 384, kKeyCols = 64;
constexpr float kHeadroom = 8.f;  // a tile may pass the reference by 2^8
constexpr float kOffset = 7.f;    // probabilities are scaled by 2^7: 2^15 at most
constexpr float kLog2e = 1.4426950408889634f;

struct SharedParams {
  const float* ks[2];  // int8 rows: K and V scales, [0] the prefix's, [1] the sequences' own
  const float* vs[2];
  int32_t prefix, own_cap;
  const int32_t* own_len;
  int32_t batch, n_q, n_kv, G;  // G = n_q / n_kv
  // A prefix unit: up to 64 rows of a KV head, seqs whole sequences of G heads (G <= 64) or
  // 64 heads of one; groups of them. An own unit: up to 64 heads of a sequence; parts of them.
  int32_t seqs, parts, heads, groups;
  int32_t rows, own_rows;       // query rows that a partial of either kind holds
  int32_t ctas;
  int32_t prefix_tiles, pieces, prefix_ctas;  // pieces of a prefix unit; 0: the units as one line
  int32_t piece_tiles, longer;                // the first `longer` pieces of a unit have one tile more
  uint32_t piece_inv, group_inv;              // reciprocals of pieces and groups (small_quotient)
  // partials: (reference, sum) per row, then O per row; the prefix units' slots, then the own units'
  float *ml, *acc, *own_ml, *own_acc;
  __half* out;
  int32_t* err;
  uint64_t wait_ns;
  int32_t stall;  // test (set_shared_stall)
};

struct alignas(64) SharedMaps {
  CUtensorMap k, v, own_k, own_v, q, own_q;
};

// ------------------------------------------------------------------ the work ----
// On a line a unit takes its tiles and kUnitCost places before them: starting one costs
// about as long as that many tiles. A line of `total` places is cut into `ctas` pieces
// (no more than places, so that none is empty); a unit u and a piece c meet at most once
// and only grow along the line, so u + c numbers the partials, on both sides.
constexpr int kUnitCost = 1;
Q4G_DEV int places(int tiles) { return tiles > 0 ? tiles + kUnitCost : 0; }

// a / b for a >= 0, b > 0. A CTA's first own segment waits for about ten of these one after
// the other, and the compiler's take 40 (32 bits) to some hundred (64 bits) instructions:
// below 2^23 the quotient comes from an fp32 division, off by at most one either way
// (2 ulp of at most 2^23), and the remainder corrects it.
Q4G_DEV int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 23) == 0) {
    const int x = (int)a, y = (int)b, q = (int)__fdividef((float)x, (float)y), rest = x - q * y;
    return rest < 0 ? q - 1 : rest >= y ? q + 1 : q;
  }
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// a / b for a, b < 2^16, from inv = ceil(2^32 / b): the excess of a * inv is below 2^32 / b. A
// CTA starts with two of these.
Q4G_DEV int small_quotient(int a, uint32_t inv, int b) { return b == 1 ? a : (int)__umulhi((uint32_t)a, inv); }
Q4G_DEV int64_t cut_begin(int64_t total, int ctas, int c) { return ctas > 0 ? quotient(total * c, ctas) : 0; }
Q4G_DEV int cut_of(int64_t total, int ctas, int64_t t) { return (int)quotient((t + 1) * ctas - 1, total); }

// The own units' line: places [0, head) go to the CTAs without a prefix piece, the rest
// to those with one, so that all have about the same work.
struct Line {
  const int32_t* own_places;  // [batch + 1] places of one KV head's own rows, summed up
  int64_t total, head;
  int32_t head_ctas, tail_ctas;
};

Q4G_DEV int own_len_of(const SharedParams& p, int b) {
  return p.own_cap > 0 ? min(max(p.own_len[b], 0), p.own_cap) : 0;
}

// own_places[0..batch], by one warp; `len`: own_len_of(lane), loaded earlier.
Q4G_DEV void sum_own_places(const SharedParams& p, int32_t* own_places, int lane, int len) {
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    if (b0 > 0) len = b < p.batch ? own_len_of(p, b) : 0;
    int v = places((len + kTileKeys - 1) / kTileKeys);
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
  w.own_places = own_places;
  w.total = (int64_t)own_places[p.batch] * p.n_kv * p.parts;
  const int idle = p.ctas - p.prefix_ctas;
  const int64_t load = p.pieces > 0 ? p.piece_tiles + (p.longer > 0) + kUnitCost : 0;
  if (idle == 0) w.head = 0;
  else if (w.total <= idle * load || p.prefix_ctas == 0) w.head = w.total;
  else w.head = quotient(idle * (p.prefix_ctas * load + w.total), p.ctas);
  w.head_ctas = (int)min((int64_t)idle, w.head);
  w.tail_ctas = (int)min((int64_t)p.prefix_ctas, w.total - w.head);
  return w;
}
Q4G_DEV int line_piece(const Line& w, int64_t t) {
  return t < w.head ? cut_of(w.head, w.head_ctas, t) : w.head_ctas + cut_of(w.total - w.head, w.tail_ctas, t - w.head);
}

struct Segment {
  int16_t own, b, h, g0, n_rows;  // first sequence and head, query rows
  int key0, key_end, tiles;   // keys [key0, key_end) of the unit's rows
  int64_t slot;
};

// A CTA's segments, its prefix piece (or its part of the prefix line) first: they need no
// own length, so that the first can start while those are still on their way.
struct Work {
  int64_t t, end;
  int own;
  Q4G_DEV Work(const SharedParams& p) : own(0) {
    const int c = blockIdx.x;
    if (p.pieces > 0) {
      t = c, end = c < p.prefix_ctas ? c + 1 : c;
    } else {
      const int64_t total = (int64_t)p.n_kv * p.groups * places_h(p);
      t = p.prefix_ctas > 0 ? cut_begin(total, p.prefix_ctas, c) : 0;
      end = p.prefix_ctas > 0 ? cut_begin(total, p.prefix_ctas, c + 1) : 0;
    }
  }
  static Q4G_DEV int places_h(const SharedParams& p) { return places(p.prefix_tiles); }
  // The own units follow: from here on next() takes them.
  Q4G_DEV void start_own(const SharedParams& p, const Line& w) {
    own = 1;
    const int c = blockIdx.x, r = c - p.prefix_ctas;
    t = end = 0;
    if (r >= 0 && r < w.head_ctas) {
      t = cut_begin(w.head, w.head_ctas, r), end = cut_begin(w.head, w.head_ctas, r + 1);
    } else if (r < 0 && c < w.tail_ctas) {
      t = w.head + cut_begin(w.total - w.head, w.tail_ctas, c);
      end = w.head + cut_begin(w.total - w.head, w.tail_ctas, c + 1);
    }
  }
  // The next segment of the current kind; false: there is none. A whole warp calls it.
  Q4G_DEV bool next(const SharedParams& p, const Line& w, Segment& s) {
    for (;;) {
      if (t >= end) return false;
      s.own = own;
      int first, len;
      if (!own) {
        int u;
        if (p.pieces > 0) {
          u = small_quotient((int)t, p.piece_inv, p.pieces);
          const int k = (int)t - u * p.pieces;
          first = k * p.piece_tiles + min(k, p.longer);
          s.tiles = p.piece_tiles + (k < p.longer);
          s.slot = t;
          t = end;
          s.h = small_quotient(u, p.group_inv, p.groups);
        } else {
          const int n = places_h(p);
          u = (int)quotient(t, n);
          s.slot = (int64_t)u + blockIdx.x;
          advance(t - (int64_t)u * n, n, first, s.tiles);
          s.h = (int)quotient(u, p.groups);
        }
        const int grp = u - s.h * p.groups;
        s.b = p.parts == 1 ? grp * p.seqs : grp / p.parts;
        s.g0 = p.parts == 1 ? 0 : grp % p.parts * kGroupRows;
        s.n_rows = p.parts == 1 ? min(p.seqs, p.batch - s.b) * p.G : min(kGroupRows, p.G - s.g0);
        len = p.prefix;
      } else {
        const int per = p.n_kv * p.parts;
        int lo = -1;  // the last sequence that starts at or before t: it is not empty
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          const int b = b0 + (threadIdx.x & 31);
          lo += __popc(__ballot_sync(0xffffffffu, b < p.batch && (int64_t)w.own_places[b] * per <= t));
        }
        const int n = w.own_places[lo + 1] - w.own_places[lo];
        const int64_t y = t - (int64_t)w.own_places[lo] * per;
        const int u = (int)quotient(y, n);
        s.slot = (int64_t)lo * per + u + line_piece(w, t);
        s.b = lo;
        s.h = p.parts == 1 ? u : u / p.parts;
        s.g0 = p.parts == 1 ? 0 : u % p.parts * kGroupRows;
        s.n_rows = min(kGroupRows, p.G - s.g0);
        len = own_len_of(p, lo);
        advance(y - (int64_t)u * n, n, first, s.tiles);
      }
      if (s.tiles <= 0) continue;
      s.key0 = first * kTileKeys;
      s.key_end = min(len, s.key0 + s.tiles * kTileKeys);
      return true;
    }
  }
  // From place j of a unit of n places: its tiles [first, first + tiles) up to `end`.
  Q4G_DEV void advance(int64_t j, int n, int& first, int& tiles) {
    const int64_t e = min((int64_t)n, j + end - t);
    t += e - j;
    first = (int)max(j - kUnitCost, (int64_t)0);
    tiles = (int)e - kUnitCost - first;
  }
};

// ------------------------------------------------------------- shared memory ----
// fp16 rows: a ring stage holds a part, 128 keys x 128 columns, as two swizzled blocks of 64
// columns (V's two are the M = 128 of one product). (Parts of half that size in a ring of 9
// cost more issues than they saved in waiting: with hi alone 109 us against 104 on 16 sequences
// and a 128K prefix.) int8 rows arrive in rings of codes of their own, K's parts whole, V's by
// halves of 64 keys, and are widened: K into tensor memory, V into this ring.
template <int HD, bool I8>
struct Plan {
  static constexpr int kStages = I8 || HD == 512 ? 4 : 5;
  static constexpr int kHalves = I8 ? 2 : 1;  // V parts of 128 value dimensions
  // codes: stages of K parts and of V parts (those and V's ring stages even: each of the two
  // groups that widen V has its own)
  static constexpr int kKeyCodes = I8 ? (HD == 512 ? 2 : 4) : 0, kValueCodes = I8 ? 4 : 0;
  static constexpr int kThreads = 32 * (4 + kSoftmaxWarps + (I8 ? kConvertWarps : 0));
  static constexpr int kStage = kTileKeys * 256 / kHalves;  // bytes
  static constexpr int kBox = kStage / 2;                   // a block of 64 columns
  static constexpr int kKeyCode = kTileKeys * 128, kValueCode = kKeyCode / kHalves;
  static constexpr int kQSlab = kGroupRows * 128;
  static constexpr int kQ = 0;
  static constexpr int kP = kQ + HD / 64 * kQSlab;
  static constexpr int kPBytes = kTileKeys * 128;  // P^T: hi, then lo
  static constexpr int kRing = kP + 2 * kPBytes;
  static constexpr int kCodes = kRing + kStages * kStage;
  static constexpr int kValues = kCodes + kKeyCodes * kKeyCode;
  static constexpr int kState = kValues + kValueCodes * kValueCode;
  static_assert(I8 ? kStages % 2 == 0 && kValueCodes % 2 == 0 : HD / 128 <= kStages, "ring sizes");
};

constexpr int kQueue = 2;  // segments that the scheduling warp is ahead at most

// Barriers and small arrays of a CTA, apart from the ring's own barriers.
struct State {
  float wmax[4][kGroupRows];  // per key quarter: a tile's column maxima; at the end column sums
  float ref[kGroupRows];
  float factor[kGroupRows];
  Segment seg[kQueue];
  uint64_t seg_full[kQueue], seg_empty[kQueue];
  uint64_t s_full[2], s_free[2], p_full, pv_done, q_full, q_free, o_free, drain[2];
  int32_t own_places[kMaxBatch + 1];
  uint32_t tmem;
  uint32_t fills, last, items;  // of the copying thread, at its end
  int32_t clean_at;  // the ring stage of the first V part to clear
  volatile int abort;
};
// fp16 rows: the last tile's V parts to clear; int8 rows: the ring of codes, and that of
// their K parts, widened into tensor memory.
template <int HD, bool I8>
struct RowState {
  uint64_t clean_ask[HD / 128], clean_done[HD / 128];
};
template <int HD>
struct RowState<HD, true> {
  // codes of K and of V parts, and K parts widened into tensor memory
  static constexpr int NK = Plan<HD, true>::kKeyCodes, NV = Plan<HD, true>::kValueCodes;
  uint64_t kc_full[NK], kc_empty[NK], vc_full[NV], vc_empty[NV], k_full[2], k_empty[2];
};
template <int HD, bool I8>
struct RingState : State, RowState<HD, I8> {
  // a ring stage's fills with K and with V parts ([1]; all fills with int8 rows) have a
  // barrier each: one consumer then waits for all of a barrier's phases, in order
  uint64_t full[2][Plan<HD, I8>::kStages], empty[Plan<HD, I8>::kStages];
  uint64_t o_part[HD / 128];  // 128 value dimensions of a segment's O^T are complete
};

template <int HD, bool I8>
constexpr size_t smem_bytes() {
  return Plan<HD, I8>::kState + sizeof(RingState<HD, I8>);
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
  atomicOr(p.err, kErrShared);
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
// The scheduling warp works the segments out (their divisions and searches would cost each
// role more than a microsecond a segment) and queues them; tiles = 0 ends the queue.
struct Scheduler {
  Work work;
  Line line{};
  Segment s{};
  uint32_t n = 0;
  // The first prefix segment comes from the arguments alone and is queued by the thread that
  // makes the barriers, so that nobody sleeps for it.
  Q4G_DEV explicit Scheduler(const SharedParams& p) : work(p) {}
  Q4G_DEV void push_first(const SharedParams& p, State& sh) {
    if (!work.next(p, line, s)) return;
    sh.seg[0] = s;
    mbar_arrive(&sh.seg_full[0]);
  }
  Q4G_DEV bool push(const SharedParams& p, State& sh, int lane) {
    // this wait lasts as long as a segment, which may be a whole prefix (the others: a tile)
    bool room = n < kQueue;
    for (int k = 0; k < 30 && !room && !sh.abort; ++k)
      room = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.seg_empty[n % kQueue], (n / kQueue - 1) & 1, p.wait_ns));
    if (!room) {
      sh.abort = 1;
      if (lane == 0) atomicOr(p.err, kErrShared);
      return false;
    }
    if (lane == 0) {
      sh.seg[n % kQueue] = s;
      mbar_arrive(&sh.seg_full[n % kQueue]);  // releases the write above
    }
    ++n;
    return true;
  }
  Q4G_DEV void run(const SharedParams& p, State& sh, int lane, int len) {
    bool first = true;
    for (;;) {
      if (work.next(p, line, s)) {
        if (first && !work.own) n = 1;  // push_first() has queued it
        else if (!push(p, sh, lane)) return;
        first = false;
      } else if (!work.own) {
        sum_own_places(p, sh.own_places, lane, len);
        __syncwarp();
        line = make_line(p, sh.own_places);
        work.start_own(p, line);
      } else {
        break;
      }
    }
    s.tiles = 0;
    push(p, sh, lane);
  }
};
// A role's segment number i, false at the end (or when a wait has given up).
Q4G_DEV bool take(State& sh, const SharedParams& p, uint32_t i, Segment& s) {
  if (!wait(sh, p, &sh.seg_full[i % kQueue], (i / kQueue) & 1)) return false;
  s = sh.seg[i % kQueue];
  return s.tiles > 0;
}
// The same for a warp: all lanes agree, and have read the segment before one gives it back
// (a vote orders no memory, __syncwarp does).
Q4G_DEV bool take_warp(State& sh, const SharedParams& p, uint32_t i, Segment& s) {
  const bool more = __all_sync(0xffffffffu, take(sh, p, i, s));
  __syncwarp();
  return more;
}
Q4G_DEV void give_back(State& sh, uint32_t i) { mbar_arrive(&sh.seg_empty[i % kQueue]); }

// A role's place in a ring of N stages and the phase that its next wait is for.
template <int N>
struct Ring {
  int at = 0;
  uint32_t phase;
  Q4G_DEV explicit Ring(uint32_t first) : phase(first) {}
  Q4G_DEV void step() {
    if (++at == N) at = 0, phase ^= 1;
  }
};
// A ring in which K and V parts alternate as the producer lays them out, for one consumer of
// one kind: a phase bit per stage, as that kind's fills of a stage are counted.
template <int N>
struct PartRing {
  int at = 0;
  uint32_t bits = 0;
  Q4G_DEV uint32_t phase() const { return (bits >> at) & 1; }
  Q4G_DEV void step() {
    bits ^= 1u << at;
    if (++at == N) at = 0;
  }
  Q4G_DEV void skip(int n) {  // the other kind's parts, n <= N
    at += n;
    if (at >= N) at -= N;
  }
};

// All copies of keys and values, by one thread: in step i the K parts of tile i and the V
// parts of tile i - 1, whose products run beside each other. fp16 rows: one ring, all of K
// before V; int8 rows: a ring of codes for each, in turn. An issue takes about 0.1 us, so a
// part is one copy, and the queries are left to the thread that multiplies with them.
// (Asking L2 for the next tile as well, by prefetch copies, was slower at every length.)
template <int HD, bool I8>
Q4G_DEV void produce(const SharedParams& p, const SharedMaps& maps, unsigned char* smem, RingState<HD, I8>& sh) {
  using P = Plan<HD, I8>;
  constexpr int C = HD / 128, NK = I8 ? P::kKeyCodes : P::kStages, NV = I8 ? P::kValueCodes : 1;
  Ring<NK> rk(1);  // the phase before a stage's first use: that wait is over at once
  [[maybe_unused]] Ring<NV> rv(1);
  uint32_t seg = 0, items = 0;
  uint32_t fills = 0, last = 0;  // a bit per stage: K fills (and from bit 16 on V fills) so far odd; the last was V
  bool ok = true;
  Segment s{};
  while (ok && take(sh, p, seg, s)) {
    give_back(sh, seg);
    ++seg;
    const void* const k_map = s.own ? &maps.own_k : &maps.k;
    const void* const v_map = s.own ? &maps.own_v : &maps.v;
    const int b = s.own ? s.b : 0, h = s.h;
    for (int i = 0; i <= s.tiles && ok; ++i) {
      const int key = s.key0 + i * kTileKeys;
      if constexpr (I8) {
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
          if (i < s.tiles) {
            if (!(ok = wait(sh, p, &sh.kc_empty[rk.at], rk.phase))) break;
            mbar_arrive_expect_tx(&sh.kc_full[rk.at], P::kKeyCode);
            tma_load_5d(smem + P::kCodes + rk.at * P::kKeyCode, k_map, 0, key, c, h, b, &sh.kc_full[rk.at]);
            fills ^= 1u << rk.at;
            rk.step();
          }
          for (int half = 0; half < P::kHalves && i > 0; ++half) {
            if (!(ok = wait(sh, p, &sh.vc_empty[rv.at], rv.phase))) break;
            mbar_arrive_expect_tx(&sh.vc_full[rv.at], P::kValueCode);
            tma_load_5d(smem + P::kValues + rv.at * P::kValueCode, v_map, 0, key - kTileKeys + half * 64, c, h, b,
                        &sh.vc_full[rv.at]);
            fills ^= 1u << (16 + rv.at);
            rv.step();
          }
          if (!ok) break;
        }
      } else {
        for (int part = 0; part < 2 && ok; ++part) {
          if (part == 0 ? i == s.tiles : i == 0) continue;
          const void* const map = part ? v_map : k_map;
#pragma unroll 1
          for (int c = 0; c < C; ++c) {
            if (!(ok = wait(sh, p, &sh.empty[rk.at], rk.phase))) break;
            uint64_t* const bar = (part ? sh.full[1] : sh.full[0]) + rk.at;
            mbar_arrive_expect_tx(bar, P::kStage);
            tma_load_5d(smem + P::kRing + rk.at * P::kStage, map, 0, part ? key - kTileKeys : key, 2 * c, h, b, bar);
            fills ^= 1u << (16 * part + rk.at);
            last = (last & ~(1u << rk.at)) | ((uint32_t)part << rk.at);
            ++items;
            rk.step();
          }
        }
      }
    }
  }
  sh.fills = fills, sh.last = last, sh.items = items;
}

// After a wait has given up and every role has ended: copies in flight still write this CTA's
// shared memory. Each is the last of its stage (and, of a stage with one barrier for K and one
// for V, kind), so its phase stays. (The queries' are waited for where they are made.)
template <int HD, bool I8>
Q4G_DEV void drain_copies(const SharedParams& p, RingState<HD, I8>& sh) {
  using P = Plan<HD, I8>;
  const uint32_t fills = sh.fills;
  if constexpr (I8) {  // a stage that was never filled has no phase to wait for: that wait is over at once
    for (int k = 0; k < P::kKeyCodes; ++k) mbar_wait_bounded(&sh.kc_full[k], ((fills >> k) & 1) ^ 1, p.wait_ns);
    for (int k = 0; k < P::kValueCodes; ++k) mbar_wait_bounded(&sh.vc_full[k], ((fills >> (16 + k)) & 1) ^ 1, p.wait_ns);
  } else {
    for (int k = 0; k < P::kStages && k < (int)sh.items; ++k) {
      const int kind = (sh.last >> k) & 1;
      mbar_wait_bounded((kind ? sh.full[1] : sh.full[0]) + k, ((fills >> (16 * kind + k)) & 1) ^ 1, p.wait_ns);
    }
  }
}

// What lies behind a sequence's own rows may be anything, and zero times a NaN is not zero:
// in the last V tile the rows up to the next 16 (those that the products take) are cleared,
// when the thread that makes the products has seen them arrive, by the softmax warps, which
// only wait for it then. (Codes are finite, and their scales are masked.)
template <bool I8>
Q4G_DEV bool needs_clean(const Segment& s) { return !I8 && s.own && (s.key_end & 15) != 0; }

// The products, by two threads of two warps: the issuing thread, not the tensor core, is what
// a product waits for (one thread with descriptors made for each product and a wait every 8
// took 73 cycles a product; with one addition per descriptor 61; two threads 48, n = 64).
//
// S^T of a segment's tiles; the segment's queries.
template <int HD, bool I8>
Q4G_DEV void multiply_keys(const SharedParams& p, const SharedMaps& maps, unsigned char* smem, RingState<HD, I8>& sh) {
  using P = Plan<HD, I8>;
  constexpr int C = HD / 128;
  [[maybe_unused]] PartRing<P::kStages> r;
  [[maybe_unused]] Ring<2> rk(0);
  const uint64_t ring = tc_desc(smem_u32(smem) + P::kRing, 0), q = tc_desc(smem_u32(smem) + P::kQ, 0);
  const uint32_t s_col = sh.tmem;
  uint32_t tile = 0, seg = 0;
  bool ok = true;
  Segment s{};
  while (ok && take(sh, p, seg, s)) {
    give_back(sh, seg);
    const uint32_t id = tc_idesc_f16((s.n_rows + 15) & ~15, false, false);
    if (seg > 0 && !(ok = wait(sh, p, &sh.q_free, (seg - 1) & 1))) break;
    mbar_arrive_expect_tx(&sh.q_full, HD * 2 * p.heads * (s.own ? 1 : p.seqs));
#pragma unroll 1
    for (int c = 0; c < HD / 64; ++c)
      tma_load_4d(smem + P::kQ + c * P::kQSlab, s.own ? &maps.own_q : &maps.q, c * 64, s.g0, s.h, s.b, &sh.q_full);
    if (!(ok = wait(sh, p, &sh.q_full, seg & 1))) {
      mbar_wait_bounded(&sh.q_full, seg & 1, p.wait_ns);  // the copies write this CTA's shared memory
      break;
    }
    for (int i = 0; i < s.tiles && ok; ++i, ++tile) {
      const uint32_t s_at = s_col + (tile & 1) * kGroupRows;
      if (tile >= 2 && !(ok = wait(sh, p, &sh.s_free[tile & 1], (tile / 2 - 1) & 1))) break;
#pragma unroll 1
      for (int c = 0; c < C; ++c) {
        if constexpr (I8) {
          if (!(ok = wait(sh, p, &sh.k_full[rk.at], rk.phase))) break;
          tc_fence_after();
          const uint32_t a = sh.tmem + kKeyCol + rk.at * kKeyCols;
          const uint64_t b = q + c * (2 * P::kQSlab >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_f16_ta(s_at, a + k * 8, b + (k >> 2) * (P::kQSlab >> 4) + (k & 3) * 2, id, c > 0 || k > 0);
          tc_commit(&sh.k_empty[rk.at]);
          rk.step();
        } else {
          if (!(ok = wait(sh, p, &sh.full[0][r.at], r.phase()))) break;
          tc_fence_after();
          const uint64_t a = ring + r.at * (P::kStage >> 4), b = q + c * (2 * P::kQSlab >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_f16(s_at, a + (k >> 2) * (P::kBox >> 4) + (k & 3) * 2, b + (k >> 2) * (P::kQSlab >> 4) + (k & 3) * 2,
                       id, c > 0 || k > 0);
          tc_commit(&sh.empty[r.at]);
          r.step();
        }
      }
      if (!ok) break;
      tc_commit(&sh.s_full[tile & 1]);
      if (i == s.tiles - 1) tc_commit(&sh.q_free);
      if constexpr (!I8) {  // the parts of V that follow: the tile's before, and the last one's
        if (i > 0) r.skip(C);
        if (i == s.tiles - 1) r.skip(C);
      }
    }
    ++seg;
  }
}

// O^T += V^T P^T.
template <int HD, bool I8>
Q4G_DEV void multiply_values(const SharedParams& p, unsigned char* smem, RingState<HD, I8>& sh) {
  using P = Plan<HD, I8>;
  constexpr int C = HD / 128;
  PartRing<P::kStages> r;
  const uint64_t ring = tc_desc(smem_u32(smem) + P::kRing, P::kBox), pt = tc_desc(smem_u32(smem) + P::kP, 0);
  const uint32_t o_col = sh.tmem + 2 * kGroupRows;
  uint32_t tile = 0, seg = 0, cleaned = 0;
  bool ok = true;
  Segment s{};
  while (ok && take(sh, p, seg, s)) {
    give_back(sh, seg);
    const uint32_t id = tc_idesc_f16((s.n_rows + 15) & ~15, true, true);
    const bool clean = needs_clean<I8>(s);
    if (!I8) r.skip(C);  // the first tile's K parts
    if (seg > 0 && !(ok = wait(sh, p, &sh.o_free, (seg - 1) & 1))) break;
    for (int i = 0; i < s.tiles && ok; ++i, ++tile) {
      const bool last = i == s.tiles - 1;
      if (!I8 && !last) r.skip(C);  // the next tile's K parts
      if (!(ok = wait(sh, p, &sh.p_full, tile & 1))) break;
      // the live keys, rounded up to 16
      const int live = min(kTileKeys, s.key_end - s.key0 - i * kTileKeys);
      const int steps = (live + 15) >> 4;
      if constexpr (!I8) {
        if (last && clean) {  // all parts at once: the ring holds them
          PartRing<P::kStages> ahead = r;
          sh.clean_at = ahead.at;
          for (int c = 0; c < C && ok; ++c, ahead.step())
            if ((ok = wait(sh, p, &sh.full[1][ahead.at], ahead.phase()))) mbar_arrive(&sh.clean_ask[c]);
          if (!ok) break;
        }
      }
#pragma unroll 1
      for (int c = 0; c < P::kHalves * C; ++c) {
        if (!(ok = wait(sh, p, &sh.full[1][r.at], r.phase()))) break;
        constexpr int kSteps = 8 / P::kHalves;
        const int d = c / P::kHalves, half = c % P::kHalves;
        if constexpr (!I8) {
          if (last && clean && !(ok = wait(sh, p, &sh.clean_done[d], cleaned & 1))) break;
        }
        tc_fence_after();
        const uint64_t a = ring + r.at * (P::kStage >> 4), b = pt + half * (kSteps * 128);
        const uint32_t o_at = o_col + d * kGroupRows;
        auto product = [&](int k) {
          tc_mma_f16(o_at, a + k * 128, b + k * 128, id, i > 0 || half > 0 || k > 0);
          tc_mma_f16(o_at, a + k * 128, b + (P::kPBytes >> 4) + k * 128, id, true);
        };
        if (steps == kTileKeys / 16) {
#pragma unroll
          for (int k = 0; k < kSteps; ++k) product(k);
        } else {
#pragma unroll 1
          for (int k = 0; k < kSteps && half * kSteps + k < steps; ++k) product(k);
        }
        tc_commit(&sh.empty[r.at]);
        if (last && half == P::kHalves - 1) tc_commit(&sh.o_part[d]);  // 128 of the value dimensions are complete
        r.step();
      }
      if (!ok) break;
      tc_commit(&sh.pv_done);
    }
    if (clean) ++cleaned;
    ++seg;
  }
}

// int8 codes into fp16: with the sign bit flipped a code c is the byte c + 128, and the
// fp16 pattern 0x6400 | byte is 1024 + byte, so one subtraction gives c, exactly.
Q4G_DEV uint32_t widen2(uint32_t u, uint32_t sel) {
  const uint32_t h = __byte_perm(u, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kGroup = 128;  // threads that widen a part

// 16 codes into 16 fp16 values.
Q4G_DEV void widen16(uint4 u, uint32_t (&h)[8]) {
  const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
#pragma unroll
  for (int k = 0; k < 4; ++k) h[2 * k] = widen2(w[k], 0x4140), h[2 * k + 1] = widen2(w[k], 0x4342);
}

// int8 rows out of L2 take longer than fp16 rows (64 sequences on a 32K prefix: 144 us against
// 130): the roles use half of the issue slots and wait for one another. Measured on the way, 64 sequences on a 32K prefix: all parts
// widened through shared memory's one ring by two groups 149 us, K and V by groups of their
// own 138, V without selects and by halves 122; a second group for K 120 there, but 73
// against 70 us for 8 sequences on a 128K prefix. With lo beside hi in P^T 144 and 80.
//
// A stage of codes is given back when what they became is written: every lane has used its
// loads then. (Given back after the loads, before a wait and their use, the next copy could
// overwrite codes: wrong values in one block of value dimensions, seldom.)
//
// K parts become operand A in tensor memory (a thread is a key).
template <int HD>
Q4G_DEV void convert_keys(const SharedParams& p, unsigned char* smem, RingState<HD, true>& sh) {
  using P = Plan<HD, true>;
  const int tid = threadIdx.x & (kGroup - 1), lane = tid & 31;
  const uint32_t key_lanes = sh.tmem + ((uint32_t)(tid & ~31) << 16) + kKeyCol;
  Ring<P::kKeyCodes> rc(0);
  Ring<2> rk(1);
  Segment s;
  for (uint32_t seg = 0; take_warp(sh, p, seg, s); ++seg) {
    if (lane == 0) give_back(sh, seg);
#pragma unroll 1
    for (int c = 0; c < s.tiles * (HD / 128); ++c) {
      if (!wait_warp(sh, p, &sh.kc_full[rc.at], rc.phase)) return;
      const unsigned char* const src = smem + P::kCodes + rc.at * P::kKeyCode + tid * 128;
      if (!wait_warp(sh, p, &sh.k_empty[rk.at], rk.phase)) return;
      tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 u[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) u[x] = *reinterpret_cast<const uint4*>(src + (((half * 4 + x) ^ (tid & 7)) * 16));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t h[8];
            widen16(u[2 * x + g], h);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[g * 8 + k] = __uint_as_float(h[k]);
          }
          tmem_st16(key_lanes + rk.at * kKeyCols + half * 32 + x * 16, v);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full[rk.at]), mbar_arrive(&sh.kc_empty[rc.at]);
      rc.step();
      rk.step();
    }
  }
}

// V parts become the swizzled blocks in shared memory that fp16 rows have, by halves of 64
// keys; two groups take turns at the halves. A thread has 16 of the 128 columns in every
// 16th key. Eight lanes have the first half of a key's columns and the second half of its
// neighbour's: reads and both writes of 16 bytes then fall on different banks.
template <int HD>
Q4G_DEV void convert_values(const SharedParams& p, unsigned char* smem, RingState<HD, true>& sh, int group) {
  using P = Plan<HD, true>;
  const int tid = threadIdx.x & (kGroup - 1), lane = tid & 31;
  const int g = tid & 7, row = (tid >> 3) ^ (g >> 2), c0 = 2 * (g & 3);
  const int from = row * 128 + ((g ^ (row & 7)) * 16);
  const int to = (g >> 2) * P::kBox + row * 128, to0 = to + ((c0 ^ (row & 7)) * 16), to1 = to0 ^ 16;
  Ring<P::kValueCodes> rc(0);
  Ring<P::kStages> rv(1);
  Segment s;
  if (group == 1) rc.step(), rv.step();
  for (uint32_t seg = 0; take_warp(sh, p, seg, s); ++seg) {
    if (lane == 0) give_back(sh, seg);
#pragma unroll 1
    for (int c = 0; c < s.tiles * (HD / 128); ++c) {
      if (!wait_warp(sh, p, &sh.vc_full[rc.at], rc.phase)) return;
      const unsigned char* const src = smem + P::kValues + rc.at * P::kValueCode + from;
      uint4 u[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) u[x] = *reinterpret_cast<const uint4*>(src + x * 2048);
      if (!wait_warp(sh, p, &sh.empty[rv.at], rv.phase)) return;
      unsigned char* const dst = smem + P::kRing + rv.at * P::kStage;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t h[8];
        widen16(u[x], h);
        *reinterpret_cast<uint4*>(dst + to0 + x * 2048) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(dst + to1 + x * 2048) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.full[1][rv.at]), mbar_arrive(&sh.vc_empty[rc.at]);
      rc.step(), rc.step();
      rv.step(), rv.step();
    }
  }
}

// One thread: a key of the tile (tensor-memory lane) and 32 of the 64 query rows.
template <int HD, bool I8>
Q4G_DEV void softmax(const SharedParams& p, unsigned char* smem, RingState<HD, I8>& sh) {
  using P = Plan<HD, I8>;
  constexpr int C = HD / 128;
  const int tid = threadIdx.x - 128, lane = tid & 31, quarter = (tid >> 5) & 3, c0 = (tid >> 7) * 32;
  const int key = quarter * 32 + lane;
  const uint32_t lanes = sh.tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t s_col = lanes + c0, o_col = lanes + 2 * kGroupRows + c0;
  uint32_t tile = 0;
  // once a wait has given up nothing waits any more, but every thread goes on to the end:
  // the barriers among these warps have no limit of their own
  bool ok = true;
  uint32_t cleaned = 0;
  for (uint32_t seg = 0;; ++seg) {
    Segment s;
    if (softmax_any(!__all_sync(0xffffffffu, take(sh, p, seg, s)))) break;  // all warps or none
    if (lane == 0) give_back(sh, seg);
    const int n = (s.n_rows + 15) & ~15;
    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.f;
    int left = s.key_end - s.key0 - key;  // this thread's key of the tile is live while left > 0
    const int64_t row0 = ((s.own ? (int64_t)s.b * p.own_cap : 0) + s.key0 + key) * p.n_kv + s.h;
    const float* ks_at = (s.own ? p.ks[1] : p.ks[0]) + row0;
    const float* vs_at = (s.own ? p.vs[1] : p.vs[0]) + row0;
    for (int j = 0; j < s.tiles; ++j, ++tile, left -= kTileKeys) {
      const bool live = left > 0;
      float ks = kLog2e, vs = 1.f, lift = 0.f;  // lift: log2 of the V scale, for the reference only
      if constexpr (I8) {
        ks = live ? *ks_at * kLog2e : 0.f;
        vs = live ? *vs_at : 0.f;
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
        raise = j > 0 && tid < s.n_rows && m > old + kHeadroom;  // rows of padding hold anything
        sh.factor[tid] = raise ? ex2(old - m) : 1.f;
        if (j == 0 || raise) sh.ref[tid] = m;
      }
      raise = softmax_any(raise);
      // P^T's buffer is free, and O^T may change here
      if (tile > 0) ok = ok && wait_warp(sh, p, &sh.pv_done, (tile - 1) & 1);
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
        unsigned char* const row = smem + P::kP + key * 128;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 ref = *reinterpret_cast<const float2*>(&sh.ref[c0 + i + e]);
            const float a = ex2(x[i + e] - ref.x + kOffset), b = ex2(x[i + e + 1] - ref.y + kOffset);
            l[i + e] += a;
            l[i + e + 1] += b;
            const float u = I8 ? a * vs : a, w = I8 ? b * vs : b;
            const __half2 h = __floats2half2_rn(u, w);
            const float2 f = __half22float2(h);
            const __half2 rest = __floats2half2_rn(u - f.x, w - f.y);
            hi[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
            lo[e / 2] = *reinterpret_cast<const uint32_t*>(&rest);
          }
          unsigned char* const at = row + ((((c0 + i) >> 3) ^ (key & 7)) * 16);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + P::kPBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full);
    }

    // the segment's partial, by blocks of 128 value dimensions as they are complete: thread =
    // value dimension and, of up to 32 rows, half of the blocks each; of more, half of the rows
    float* const ml = (s.own ? p.own_ml : p.ml) + s.slot * (s.own ? p.own_rows : p.rows) * 2;
    float* const acc = (s.own ? p.own_acc : p.acc) + s.slot * (s.own ? p.own_rows : p.rows) * HD + key;
    if constexpr (!I8) {
      if (needs_clean<I8>(s)) {
        const int from = s.key_end & (kTileKeys - 1), chunks = (16 - (from & 15)) * 16;  // of both boxes
        for (int c = 0; c < C; ++c) {
          ok = ok && wait_warp(sh, p, &sh.clean_ask[c], cleaned & 1);
          if (ok && tid < chunks) {  // (given up: clean_at may hold anything)
            const int at = (sh.clean_at + c) % P::kStages;
            *reinterpret_cast<uint4*>(smem + P::kRing + at * P::kStage + (tid & 1) * P::kBox + from * 128 + (tid >> 1) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.clean_done[c]);
        }
        ++cleaned;
      }
    }
    if (c0 < n) sh.wmax[quarter][c0 + lane] = lane_sums(l, lane);  // (while the last products run)
    const bool few = n <= 32;
    const int r0 = few ? 0 : c0, first = few && c0 > 0 ? C / 2 : 0, last = few && c0 == 0 ? C / 2 : C;
#pragma unroll 1
    for (int c = first; c < last; ++c) {
      ok = ok && wait_warp(sh, p, &sh.o_part[c], seg & 1);
      tc_fence_after();
      float o[32];
      tmem_ld32(lanes + 2 * kGroupRows + c * kGroupRows + r0, o);
      tmem_wait_ld(o);
      if (c == last - 1) {  // O^T may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_free);
      }
      float* const at = acc + r0 * HD + c * 128;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (r0 + i < s.n_rows) at[i * HD] = o[i];
    }
    softmax_sync();
    // (P^T is free for the next segment: every warp has waited for a last block)
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
  RingState<HD, I8>& sh = *reinterpret_cast<RingState<HD, I8>*>(smem + P::kState);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int len = 0;  // of own rows: warp 3's
  if (warp == 1) {
    tmem_alloc(&sh.tmem, 512);  // at once: with 227 KB of shared memory the CTA is alone on its SM
  } else if (warp == 2 && lane == 0) {
    // of a stalled ring only the third stage, so that others are in flight
    const int stall = blockIdx.x == 0 ? p.stall : 0;
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(&sh.full[0][i], 1 + (!I8 && stall == 1 && i == 2));
      mbar_init(&sh.full[1][i], I8 ? kGroup / 32 : 1 + (stall == 2 && i == 2));
      mbar_init(&sh.empty[i], 1);
    }
    if constexpr (I8) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.k_full[i], kGroup / 32);
        mbar_init(&sh.k_empty[i], 1);
      }
      for (int i = 0; i < P::kKeyCodes; ++i) {
        mbar_init(&sh.kc_full[i], 1 + (stall == 1 && i == P::kKeyCodes - 1));
        mbar_init(&sh.kc_empty[i], kGroup / 32);
      }
      for (int i = 0; i < P::kValueCodes; ++i) {
        mbar_init(&sh.vc_full[i], 1 + (stall == 2 && i == 2));
        mbar_init(&sh.vc_empty[i], kGroup / 32);
      }
    } else {
      for (int i = 0; i < HD / 128; ++i) {
        mbar_init(&sh.clean_ask[i], 1);
        mbar_init(&sh.clean_done[i], kSoftmaxWarps);
      }
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&sh.seg_full[i], 1);
      mbar_init(&sh.seg_empty[i], 3 + kSoftmaxWarps + (I8 ? kConvertWarps : 0) + (stall == 5));
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], kSoftmaxWarps);
    }
    mbar_init(&sh.p_full, kSoftmaxWarps + (stall == 4));
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.q_full, 1 + (stall == 3));
    mbar_init(&sh.q_free, 1);
    for (int i = 0; i < HD / 128; ++i) mbar_init(&sh.o_part[i], 1);
    mbar_init(&sh.o_free, kSoftmaxWarps);
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    sh.abort = 0;
    fence_mbar_init();
    Scheduler(p).push_first(p, sh);
    fence_async_smem();
  }
  pdl_wait();  // so far nothing of the kernel before was touched
  if (warp == 3 && lane < p.batch) len = own_len_of(p, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The join's CTAs take the places that CTAs of this grid leave. Not before pdl_wait(): the
  // join reads own_len ahead of its own wait, and what this grid waited for has written it.
  pdl_launch_dependents();
  // With int8 rows 768 threads start with 80 registers each: the softmax warps take 120,
  // (64 + 2 x 120 + 3 x 56) x 128 = 472 x 128 of 480 x 128.
  if (warp < 4) {
    if constexpr (I8) regs_dec<64>();
    if (warp == 0) {
      if (elect_one()) produce<HD, I8>(p, maps, smem, sh);
      __syncwarp();
    } else if (warp == 1) {
      if (elect_one()) multiply_keys<HD, I8>(p, maps, smem, sh);
      __syncwarp();
    } else if (warp == 2) {
      if (elect_one()) multiply_values<HD, I8>(p, smem, sh);
      __syncwarp();
    } else if (warp == 3) {
      Scheduler(p).run(p, sh, lane, len);
    }
  } else if (warp < 4 + kSoftmaxWarps) {
    if constexpr (I8) regs_inc<120>();
    softmax<HD, I8>(p, smem, sh);
  } else {
    if constexpr (I8) {
      regs_dec<56>();
      if (warp < 8 + kSoftmaxWarps) convert_keys<HD>(p, smem, sh);
      else convert_values<HD>(p, smem, sh, (warp >> 2) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (sh.abort) {  // no role issues any more, but copies and products in flight use shared and tensor memory
    if (warp == 0) {
      if (elect_one()) drain_copies<HD, I8>(p, sh);
      __syncwarp();
    } else if (warp <= 2) {
      if (elect_one()) {  // the thread that made the products
        tc_commit(&sh.drain[warp - 1]);
        mbar_wait_bounded(&sh.drain[warp - 1], 0, p.wait_ns);
      }
      __syncwarp();
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, 512);
  }
}

// ------------------------------------------------------------------ the join ----
constexpr int kJoinCols = 128;                          // output columns per CTA: four a lane
constexpr int kJoinMax = 2 * 256;                       // partials of a row: CTAs of its two units

// out[row] = sum_i 2^(ref_i - R) O_i / sum_i 2^(ref_i - R) l_i over the row's partials,
// R the largest reference; in a fixed order. Grid: query rows, columns / 128. The weights
// are made once, one thread a partial, so that the loads of O depend on nothing.
// kJoinParts warps, each with every kJoinParts-th partial.
template <int HD, int kJoinParts>
__global__ void __launch_bounds__(32 * kJoinParts) shared_join_kernel(const SharedParams p) {
  constexpr int kJoinThreads = 32 * kJoinParts, kJoinLanes = 32;
  __shared__ int32_t own_places[kMaxBatch + 1];
  __shared__ float red[2][kJoinThreads / 32];
  __shared__ float weight[kJoinMax];
  __shared__ float4 part[kJoinParts][kJoinLanes];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) sum_own_places(p, own_places, lane, lane < p.batch ? own_len_of(p, lane) : 0);
  __syncthreads();
  const Line w = make_line(p, own_places);
  const int b = blockIdx.x / p.n_q, hq = blockIdx.x % p.n_q, h = hq / p.G, g = hq % p.G;
  __half* const out = p.out + (int64_t)blockIdx.x * HD + blockIdx.y * kJoinCols;
  // the partials of the row: slots [s0, s0 + n0) of the prefix, [s1, s1 + n1) of its own rows
  int64_t s0 = 0, s1 = 0;
  int n0 = 0, n1 = 0, r0 = 0, r1 = g % kGroupRows;
  if (p.prefix_tiles > 0) {
    const int u = h * p.groups + (p.parts == 1 ? b / p.seqs : b * p.parts + g / kGroupRows);
    r0 = p.parts == 1 ? b % p.seqs * p.G + g : g % kGroupRows;
    if (p.pieces > 0) {
      s0 = (int64_t)u * p.pieces;
      n0 = p.pieces;
    } else {
      const int64_t len = places(p.prefix_tiles), total = len * p.n_kv * p.groups;
      const int c = cut_of(total, p.prefix_ctas, u * len + kUnitCost);
      s0 = (int64_t)u + c;
      n0 = cut_of(total, p.prefix_ctas, u * len + len - 1) - c + 1;
    }
  }
  const int own = own_places[b + 1] - own_places[b];
  if (own > 0) {
    const int per = p.n_kv * p.parts, u = h * p.parts + g / kGroupRows;
    const int64_t t = (int64_t)own_places[b] * per + (int64_t)u * own;
    const int c = line_piece(w, t + kUnitCost);
    s1 = (int64_t)b * per + u + c;
    n1 = line_piece(w, t + own - 1) - c + 1;
  }
  const int n = n0 + n1;
  const float* const acc0 = p.acc + (s0 * p.rows + r0) * HD + blockIdx.y * kJoinCols + lane * 4;
  const float* const acc1 = p.own_acc + (s1 * p.own_rows + r1) * HD + blockIdx.y * kJoinCols + lane * 4;
  const int64_t step0 = (int64_t)p.rows * HD, step1 = (int64_t)p.own_rows * HD;
  auto o_at = [&](int i) {
    return *reinterpret_cast<const float4*>(i < n0 ? acc0 + i * step0 : acc1 + (i - n0) * step1);
  };
  // references, sums and weights, a partial a thread and turn (n <= 2 * CTAs <= kJoinMax); a
  // warp's first rows of O are loaded beside them
  constexpr int kEarly = 5;
  float4 early[kEarly];
  const float* const ml0 = p.ml + (s0 * p.rows + r0) * 2;
  const float* const ml1 = p.own_ml + (s1 * p.own_rows + r1) * 2;
  float2 ml[kJoinMax / kJoinThreads];
  float R = -INFINITY;
  pdl_launch_dependents();
  pdl_wait();  // all above comes from the arguments and own_len, which is older than shared_kernel's trigger
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (warp + k * kJoinParts < n) early[k] = o_at(warp + k * kJoinParts);
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
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4 a, float f) { o.x += f * a.x, o.y += f * a.y, o.z += f * a.z, o.w += f * a.w; };
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (warp + k * kJoinParts < n) add(early[k], weight[warp + k * kJoinParts]);
#pragma unroll 5
  for (int i = warp + kEarly * kJoinParts; i < n; i += kJoinParts) add(o_at(i), weight[i]);
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

// A tensor map over fp16 values (boxes of 64 columns) or codes (128 columns), swizzled.
// dims and box from the columns outwards, `rank` of them; stride[i]: elements between
// neighbours of dimension i + 1. What a box has outside the tensor reads as zeros.
bool encode(CUtensorMap* m, const void* base, bool i8, int rank, const int64_t* dims, const int64_t* stride,
            const int32_t* box) {
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = (cuuint64_t)dims[i], b[i] = (cuuint32_t)box[i];
  for (int i = 0; i + 1 < rank; ++i) s[i] = (cuuint64_t)stride[i] * (i8 ? 1 : 2);
  return encode_tiled()(m, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                        const_cast<void*>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [batch][rows][n_kv][hd], the columns as blocks of 128 bytes: a box is `keys` keys
// of 128 columns, one block behind the other.
bool encode_rows(CUtensorMap* m, const void* base, bool i8, int hd, int n_kv, int64_t rows, int batch, int keys) {
  const int cols = i8 ? 128 : 64;
  const int64_t row = (int64_t)n_kv * hd, dims[] = {cols, rows, hd / cols, n_kv, batch},
                stride[] = {row, cols, hd, rows * row};
  const int32_t box[] = {cols, keys, 128 / cols, 1, 1};
  return encode(m, base, i8, 5, dims, stride, box);
}

constexpr int kMaxDevices = 64;
thread_local int stall_next = 0;  // set_shared_stall

template <int HD, int kJoinParts>
cudaError_t launch_join(const SharedParams& p, cudaStream_t st) {
  return launch_pdl(shared_join_kernel<HD, kJoinParts>, dim3(p.batch * p.n_q, HD / kJoinCols), 32 * kJoinParts, 0, st,
                    true, 1, p);
}

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
  e = launch_pdl(shared_kernel<HD, I8>, dim3(p.ctas), Plan<HD, I8>::kThreads, smem_bytes<HD, I8>(), st, true, 1, maps,
                 p);
  if (e != cudaSuccess) return e;
  // warps for about five partials each
  const int n = (p.pieces > 0 ? p.pieces : p.prefix_tiles > 0 ? 2 : 0) + (p.own_cap + kTileKeys - 1) / kTileKeys;
  if (n <= 20) return launch_join<HD, 4>(p, st);
  return n <= 40 ? launch_join<HD, 8>(p, st) : launch_join<HD, 16>(p, st);
}

// How the prefix units are cut: into equal pieces of `len` tiles, or, where whole pieces
// would leave more than a tenth of the CTAs without work, as one line. A longer piece
// leaves CTAs for the own rows, which otherwise come on top of somebody's piece: the
// length with the smallest estimate of the longest CTA's tiles is taken, own rows at
// half of their capacity (their lengths are on the device).
void plan_prefix(SharedParams& p, int64_t prefix, int64_t own_cap) {
  p.prefix = (int32_t)prefix;
  p.prefix_tiles = (int32_t)((prefix + kTileKeys - 1) / kTileKeys);
  p.pieces = p.prefix_ctas = 0;
  if (prefix == 0) return;
  const int64_t units = (int64_t)p.n_kv * p.groups, tiles = p.prefix_tiles, most = p.ctas / units;
  if (most < tiles && most * units * 10 < 9 * (int64_t)p.ctas) {
    p.prefix_ctas = p.ctas;  // units * (tiles + 1) > ctas places: no piece of the line is empty
    return;
  }
  const int64_t own = own_cap == 0 ? 0 : (int64_t)p.batch * p.n_kv * p.parts * ((own_cap / 2) / kTileKeys + 1 + kUnitCost);
  int64_t best = 0;
  const int64_t least = (tiles + most - 1) / most;
  for (int64_t len = least; len <= least + 4 && len <= tiles; ++len) {
    const int64_t pieces = (tiles + len - 1) / len, load = (tiles + pieces - 1) / pieces + kUnitCost;
    const int64_t idle = p.ctas - pieces * units, over = own - idle * load;
    // what the idle CTAs cannot take is shared by all, whole units at a time
    const int64_t cost = over <= 0 ? load : load + 1 + (over + p.ctas - 1) / p.ctas;
    if (best == 0 || cost < best) best = cost, p.pieces = (int32_t)pieces;
  }
  p.prefix_ctas = (int32_t)(p.pieces * units);
  p.piece_tiles = p.prefix_tiles / p.pieces;
  p.longer = p.prefix_tiles % p.pieces;
  p.piece_inv = (uint32_t)((((uint64_t)1 << 32) + p.pieces - 1) / p.pieces);
  p.group_inv = (uint32_t)((((uint64_t)1 << 32) + p.groups - 1) / p.groups);
}

// Units, partial slots and the scratch layout; returns its bytes.
size_t plan_scratch(SharedParams& p, int hd, void* ws) {
  p.G = p.n_q / p.n_kv;
  p.parts = (p.G + kGroupRows - 1) / kGroupRows;
  p.seqs = p.parts == 1 ? kGroupRows / p.G : 1;
  if (p.seqs > p.batch) p.seqs = p.batch;
  p.heads = p.parts == 1 ? p.G : kGroupRows;
  p.groups = p.parts == 1 ? (p.batch + p.seqs - 1) / p.seqs : p.batch * p.parts;
  p.rows = p.seqs * p.heads;
  p.own_rows = p.heads;
  p.ctas = device_sm_count() < kJoinMax / 2 ? device_sm_count() : kJoinMax / 2;
  const size_t n = ((size_t)p.n_kv * p.groups + p.ctas) * p.rows;
  const size_t n_own = ((size_t)p.batch * p.n_kv * p.parts + p.ctas) * p.own_rows;
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
  p.ks[0] = kps, p.ks[1] = kos, p.vs[0] = vps, p.vs[1] = vos;
  plan_prefix(p, prefix, own_cap);
  p.own_cap = (int32_t)own_cap;
  p.own_len = own_len;
  p.out = reinterpret_cast<__half*>(out);
  p.stall = stall_next;
  stall_next = 0;
  p.wait_ns = p.stall ? 20000000ull : 2000000000ull;
  if (!(p.err = device_error_word())) return bad(Q4G_ECUDA, "error word unavailable");
  SharedMaps maps{};
  // queries as [batch][n_kv][G][hd]: a box is the rows of a unit
  const int64_t q_dims[] = {hd, p.G, n_kv, batch}, q_stride[] = {hd, (int64_t)p.G * hd, (int64_t)n_q * hd};
  const int32_t q_box[] = {64, p.heads, 1, p.seqs}, own_q_box[] = {64, p.heads, 1, 1};
  bool ok = encode(&maps.q, q, false, 4, q_dims, q_stride, q_box) &&
            encode(&maps.own_q, q, false, 4, q_dims, q_stride, own_q_box);
  const int v_keys = i8 ? kTileKeys / 2 : kTileKeys;
  if (prefix > 0)
    ok = ok && encode_rows(&maps.k, kp, i8, hd, n_kv, prefix, 1, kTileKeys) &&
         encode_rows(&maps.v, vp, i8, hd, n_kv, prefix, 1, v_keys);
  if (own_cap > 0)
    ok = ok && encode_rows(&maps.own_k, ko, i8, hd, n_kv, own_cap, batch, kTileKeys) &&
         encode_rows(&maps.own_v, vo, i8, hd, n_kv, own_cap, batch, v_keys);
  if (!ok) return bad(Q4G_ECUDA, "tensor map refused by the driver");
  cudaError_t e;
  if (hd == 512) e = i8 ? launch<512, true>(maps, p, st) : launch<512, false>(maps, p, st);
  else e = i8 ? launch<256, true>(maps, p, st) : launch<256, false>(maps, p, st);
  return e == cudaSuccess ? Q4G_OK : bad(Q4G_ECUDA, cudaGetErrorString(e));
}

}  // namespace

void q4g::set_shared_stall(int kind) { stall_next = kind; }

extern "C" size_t q4g_flash_decode_shared_workspace_bytes(int32_t batch, int32_t n_q, int32_t n_kv,
                                                          int32_t head_dim) {
  // (a call with such sizes is refused)
  if (batch < 1 || batch > kMaxBatch || n_kv < 1 || n_q < n_kv || n_q > 1024 || head_dim < 1 || head_dim > 512) return 256;
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
