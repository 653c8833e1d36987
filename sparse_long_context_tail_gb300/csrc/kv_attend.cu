// Attention of new tokens over the 4-bit cache.
//
// For row (query i of request r, q head h), at position p = kv_len - q_len + i:
//   visible entries e: e <= p, and without a window or with p - e < window or
//   e < sinks;  out = sum_e softmax_e(scale q.k_e) v_e, lse = ln sum_e exp(scale q.k_e).
// Nothing visible: out = 0, lse = -inf.
//
// Bound and shape.  With the few rows a kv head has (gamma q heads x q_len new
// tokens) every cache byte is used for at most a few tens of products, so the
// call is bound by reading the cache.  To read it at the memory's rate every SM
// has to turn about 41 codes a clock into f16 and multiply them.  The matrix
// products run on mma.sync with the codes as operand A straight from registers
// (keys on M: S^T = K Q^T; dims on M: O^T = V^T P^T; rows on N, eight or
// sixteen): no code is written back to shared memory, which tcgen05 would need,
// and a pass over 16 entries of d = 128 costs 16 instructions, a third of their
// measured rate (2.0 clocks each per SM).
//
// Work.  A unit is (request, kv head, chunk of kRows rows); its tiles are the
// 32-entry runs that some row sees.  All units' tiles, in order, are dealt out to
// the workers in equal shares, from the lengths in device memory: ragged batches
// balance themselves and a captured call stays valid when the lengths change.  A
// worker is a CTA, whose teams take its tiles in turn and are joined through shared
// memory, or, where units are short, a single team that shares nothing.  A team is
// one warp, or as many as it takes for each to hold the weighted sums of its dims
// in 32 registers a lane (128 dims of eight rows, 64 of sixteen), so that sixteen
// warps fit an SM at every head size: each multiplies its dims of the queries and
// keys, the team adds the logits up through shared memory, and each weighs its dims
// of the values.  (Eight warps an SM with 250 registers instead took a third longer for 64
// requests with a window of 1024 at d = 256, and an eighth longer for four drafted tokens
// each of eight requests, when those took 46 and 31 us.)  Every team has its own ring of records filled by bulk
// copies (two records of 18 d bytes a tile).  A unit that lies in one worker's share is
// written out at once; of others every worker leaves its part (reference, sum, weighted
// sum, all fp32) in the workspace, and the last one to do so adds the parts up, in
// worker order whoever it is, so results repeat bit for bit.
//
// Measured on one GB300 (32 q heads, 8 kv heads, d = 128, bf16; device time of a call
// among others): 16 requests of 4096 to 131072 entries, 521 MB, 96 us, 5.4 TB/s or
// 0.80 of the copy rate; while tiles stream the SMs take in 6.2 TB/s, the rest is
// the start (kv_len, then page table, then the first records: 5.6 us) and the end.  One
// request of 131072 entries: 35.5 us.  One of 4096 entries with two heads of d = 64:
// 7.6 us, all of it latency.  Many short units (256 requests of up to 700 entries: 28
// us) and sixteen rows are bound by instructions: about 560 a warp for a whole tile
// (128 conversions, 128 scalings, 32 products, 32 to pair the values' entries), 1500
// to 2100 for a unit.
//
// Arithmetic.  A code times its scale has at most six significant bits and is
// exact in f16, and so is a query after division by the power of two of its
// row's largest element (elements 2^-14 below it lose their last bits: 2^-25 of
// the largest, under the fp32 sum's own rounding).  Logits, references, sums and the
// weighted sums are fp32.  The one rounding is that of the softmax weights to f16,
// 2^-11 relative; they are scaled by 2^12 against a reference that may lag the
// running maximum by 2^3, so that weights down to 2^-26 of the reference keep all
// their bits.  (Weights in two f16 parts would double the products over the values for
// an error that the rounding of a bf16 output hides.)
//
// Weights come from differences of a row's products, 2^((s - ref) f + 12) with s and ref
// as the matrix instructions give them (under 2^22) and f the row's logit factor: what
// rounds is the difference, whatever the size of the logits.  (With the reference times the
// factor folded into one constant, its last place is worth more than the f16 range of the
// weights from logits of about 10^7 on.)  So ref stays in units of s, also in the parts.  A
// row whose largest logit is past fp32 is NaN (`logit_of`).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

constexpr int kLogWarps = 3, kWarps = 1 << kLogWarps;   // of a CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;        // entries per tile (two records)
constexpr float kWeightExp = 12.f;   // weights are 2^(x - m + 12)
constexpr float kLag = 3.f;          // x may pass the reference m by this much
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ plan --

struct Request {
  int q0, q_len, n;           // first row, rows, cache entries
  int sink_t, lo_t, tiles;    // tiles [0, sink_t) and [lo_t, lo_t + tiles - sink_t)
  int lo, sinks;              // first entry inside some row's window; entries that stay visible before it
};

// What the device tables say about request r.  A table that makes no sense gives
// a request without rows or without entries, and an error in the status word.
__device__ __forceinline__ Request load_request(const KvAttendArgs& a, int r) {
  Request x;
  x.q0 = r;
  x.q_len = 1;
  x.n = a.kv_len[r];
  bool ok = true;
  if (a.cu_q) {
    x.q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    if (x.q0 < 0 || q1 < x.q0 || q1 > a.num_q || q1 - x.q0 > a.max_q) {
      ok = false;
      x.q0 = x.q_len = 0;
    } else {
      x.q_len = q1 - x.q0;
    }
  }
  if (x.n < 0 || x.n > ((int64_t)a.max_pages << a.page_shift)) {
    ok = false;
    x.n = 0;
  }
  if (!ok) set_status(a.status, UPF_ERR_INVALID_ARG);
  x.lo = a.window ? max(0, x.n - x.q_len - a.window + 1) : 0;
  x.sinks = min(a.sinks, x.lo);
  x.lo_t = x.lo / kTile;
  x.sink_t = min((x.sinks + kTile - 1) / kTile, x.lo_t);
  x.tiles = x.q_len > 0 ? x.sink_t + (x.n + kTile - 1) / kTile - x.lo_t : 0;
  return x;
}

// rho / gamma for a row of a request: the quotient is at most 1024 and gamma at most 256,
// so (rho + 1/2) / gamma is 2^-9 or more away from every integer and the fp32 product,
// off by under 2^-12, has the same whole part.
__device__ __forceinline__ int query_of(const KvAttendArgs& a, int rho) {
  return __float2int_rz((float(rho) + 0.5f) * a.inv_gamma);
}

__device__ __forceinline__ int chunks_of(const KvAttendArgs& a, const Request& x, int rows) {
  return (x.q_len * a.gamma + rows - 1) / rows;
}

// a / b, both >= 0, by the short division where it will do.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)(uint32_t(a) / uint32_t(b)) : a / b;
}

// Cost of a unit in the dealing, in tiles, beside its tiles: the rows' load, the
// first copies' latency and the writing out.
constexpr int kUnitCostCta = 24, kUnitCostTeam = 4;
// Workers are teams where units have fewer tiles than this on average.  256 short requests
// (4 tiles a unit): 28 us as teams, 54 as CTAs; 64 requests with a window (34 tiles, d = 256):
// 42.6 and 46.8; one request of 4096 entries (128 tiles): 14.5 and 7.7.
constexpr int kShortUnit = 64;

// Where workers are teams, a unit of at most this many tiles is not split: it belongs to
// the team whose share its first place lies in.  256 short requests: 28 us, 32 with
// every unit split where the shares end (parts to add up), 37 with units of up to 24 tiles
// kept whole (uneven shares).
constexpr int kWholeUnit = 8;

// How the tiles are dealt out.  Along the dealing a unit takes cost + tiles places.
struct Deal {
  bool teams;          // a worker is a team
  int cost;            // of a unit
  long long total;     // places of all units
  long long share;     // places of a worker
};

// The deal from the tiles and units of all requests; `before`: those of the requests
// before this thread's, turned into places.
__device__ __forceinline__ Deal make_deal(long long all_t, long long all_u, long long t, long long u, int teams, long long& before) {
  Deal d;
  d.teams = all_t < all_u * kShortUnit;
  d.cost = d.teams ? kUnitCostTeam : kUnitCostCta;
  d.total = all_t + all_u * d.cost;
  before = t + u * d.cost;
  const long long workers = d.teams ? (long long)gridDim.x * teams : gridDim.x;
  d.share = max(quotient(d.total + workers - 1, workers), (long long)(d.teams ? 1 : teams));
  return d;
}

__device__ __forceinline__ void scan_warp(long long& t, long long& u) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, t, s), z = __shfl_up_sync(0xFFFFFFFFu, u, s);
    if (lane >= s) {
      t += y;
      u += z;
    }
  }
}

// At most 32 requests: every warp works the deal out by itself, a request a lane (`mine`).
__device__ Deal deal_out_few(const KvAttendArgs& a, int rows, int teams, long long& before, Request& mine, bool& empty) {
  const int lane = threadIdx.x & 31;
  long long tiles = 0, units = 0;
  bool none = false;
  if (lane < a.R) {
    mine = load_request(a, lane);
    none = mine.tiles == 0;
    units = none ? 0 : (long long)a.H * chunks_of(a, mine, rows);
    tiles = units * mine.tiles;
  }
  empty = __any_sync(0xFFFFFFFFu, none);
  long long t = tiles, u = units;
  scan_warp(t, u);
  const long long all_t = __shfl_sync(0xFFFFFFFFu, t, 31), all_u = __shfl_sync(0xFFFFFFFFu, u, 31);
  return make_deal(all_t, all_u, t - tiles, u - units, teams, before);
}

// More: the CTA does, thread i looks at requests [i * per, (i + 1) * per).
// `mine`: the first of the thread's requests; `empty`: some request has no tiles.
__device__ Deal deal_out_many(const KvAttendArgs& a, int rows, int teams, int per, longlong2 (&warp_sums)[kWarps],
                              long long& before, Request& mine, bool& empty) {
  long long tiles = 0, units = 0;
  bool none = false;
  for (int j = 0; j < per; ++j) {
    const int r = threadIdx.x * per + j;
    if (r >= a.R) break;
    const Request x = load_request(a, r);
    if (j == 0) mine = x;
    if (x.tiles == 0) {
      none = true;
      continue;
    }
    const long long u = (long long)a.H * chunks_of(a, x, rows);
    units += u;
    tiles += u * x.tiles;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long t = tiles, u = units;
  scan_warp(t, u);
  if (lane == 31) warp_sums[warp] = make_longlong2(t, u);
  empty = __syncthreads_or(none);
  t -= tiles;
  u -= units;
  long long all_t = 0, all_u = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      t += warp_sums[w].x;
      u += warp_sums[w].y;
    }
    all_t += warp_sums[w].x;
    all_u += warp_sums[w].y;
  }
  return make_deal(all_t, all_u, t, u, teams, before);
}

// A row's logit factor: 2^exp times the mantissa of the scale.  Never 0: it multiplies the -inf
// of unseen entries; never infinite: the differences it multiplies may be 0.
__device__ __forceinline__ float factor_of(const KvAttendArgs& a, int exp) {
  if (exp > 127) return FLT_MAX;
  return fminf(a.scale_mant * __uint_as_float(uint32_t(max(exp, -126) + 127) << 23), FLT_MAX);
}

// The largest logit (times log2 e) of a row with factor f and reference s; NaN if it is past
// fp32, or if the factor is and the logit is not 0.  (The weights are right even then: differences
// of s are multiples of 2^-34, so that FLT_MAX takes them past the weights' range as the factor would.)
__device__ __forceinline__ float logit_of(float s, float f) {
  const float x = s * f;
  return fabsf(x) <= FLT_MAX && (f < FLT_MAX || s == 0.f) ? x : __int_as_float(0x7FFFFFFF);
}

// The workspace.  A worker has at most two units that others work on too: the one
// its share begins in the middle of, and the one that goes on after its share.
// The part of the latter (or of a unit that does both) is at 2 w + 1, that of the
// former at 2 w.
struct Parts {
  float* o;         // [part slots][rows][d]
  float2* ml;       // [part slots][rows]: reference, sum
  float* f;         // [CTAs][rows]: the rows' logit factors, for the second launch
  struct Note* notes;   // [CTAs], or null: no second launch
};

// Where few units are spread over many CTAs, adding their parts up is left to a second
// launch, which shares it among as many CTAs as the unit had (one request of 131072
// entries: 35.5 against 37.7 us at eight kv heads, 27.7 against 33.8 at two of d = 256; with
// 16 parts a unit or fewer the second launch costs more: 7.9 against 7.7 us for one
// request of 4096 entries, 44.7 against 42.6 for 64 with a window): for each CTA, the unit that goes on after its share.
struct Note {
  int first, last;        // CTAs of the unit (first < 0: no such unit)
  int h, row0, rows, q0;  // kv head, first row of the chunk, rows of the request, its first row in q
};

// Parts are counted in by at most kFan workers at a time, so that no worker has to
// add up more than kFan of them: workers first + kFan i .. of a unit count at the
// first of them, whose part then stands for them all, and these count at `first`
// in the second half of the counters.  The unit that goes on after a worker is the
// only one that counts at it.  Counters are zero between calls.
constexpr int kFan = 16;

// ---------------------------------------------------------------- kernel --

template <int kDim, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPart = kDim >= 128 ? 128 : kDim;      // dims per part of a record
  static constexpr int kSlice = NT == 1 ? kPart : 64;         // dims of a warp
  static constexpr int kHalves = kPart / kSlice;              // slices of a part
  static constexpr int kMembers = kDim / kSlice;              // warps of a team
  static constexpr int kLogTeams = kLogWarps - (kMembers == 4 ? 2 : kMembers == 2 ? 1 : 0), kTeams = 1 << kLogTeams;
  static constexpr int kSteps = kSlice / 16;                  // mma steps over a slice, and dim tiles of it
  static constexpr int kRecord = kv::record_bytes(kDim);
  static constexpr int kStage = 2 * kRecord;
  // two CTAs an SM: about 110 KB each
  static constexpr int kCtasPerSm = 2;
  static constexpr int kStages = kDim == 64 ? 6 : kMembers == 1 ? 3 : NT == 2 ? 5 : 2;
  static constexpr int kRing = kStages * kStage;              // of a team
  static constexpr int kExchange = kMembers > 1 ? 32 * 8 * NT * 4 : 0;   // a warp's logits of a tile
  static constexpr int kJoinRow = kSlice + 4;                 // floats; the pad spreads the rows over the banks
  // At the end of a unit a team's ring is empty and holds its warps' rows for the join.
  static_assert(kRows * kJoinRow * 4 <= kRing / kMembers && kRing / kMembers % 16 == 0, "a warp's join rows fit its share of the ring");
  static constexpr int kSmem = kTeams * kRing + kWarps * kExchange;
  static constexpr int kCtas = kCtasPerSm * kPlanSMs;
  static constexpr int kMaxWorkers = kCtas * kTeams;
  static_assert(2 * kMaxWorkers <= kKvCounters, "counters of the context");
  // The part that stands for the kFan workers from w on of a unit that begins at worker `first`
  // and has more.  Of such units, at most one has a later worker and one its first in a
  // run of kFan workers.
  static constexpr int kPartSlots = 2 * kMaxWorkers + 2 * (kMaxWorkers / kFan + 1);
  __device__ static int group_part(int w, int first) { return 2 * kMaxWorkers + 2 * (w / kFan) + (w == first); }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// As mma_f16, from zero.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ __half2 as_half2(uint32_t a) { return *reinterpret_cast<const __half2*>(&a); }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(as_half2(a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// (x & m) | (y & ~m)
__device__ __forceinline__ uint32_t merge_bits(uint32_t x, uint32_t y, uint32_t m) { return (x & m) | (y & ~m); }

// A unit in the dealing.
struct Unit {
  int r, h, c;        // request, kv head, chunk
  long long place;    // its first place
  Request x;
};

// The unit of request r (places from `before` on) that holds place `first`.
__device__ __forceinline__ Unit unit_at(const KvAttendArgs& a, int r, const Request& x, long long before, long long first,
                                        int cost, int rows) {
  const int chunks = chunks_of(a, x, rows), places = x.tiles + cost, unit = int(quotient(first - before, places));
  Unit u;
  u.r = r;
  u.h = unit / chunks;
  u.c = unit - u.h * chunks;
  u.place = before + (long long)unit * places;
  u.x = x;
  return u;
}

__device__ __forceinline__ void next_unit(const KvAttendArgs& a, Unit& u, int cost, int rows) {
  u.place += u.x.tiles + cost;
  if (++u.c < chunks_of(a, u.x, rows)) return;
  u.c = 0;
  if (++u.h < a.H) return;
  u.h = 0;
  do {
    if (++u.r >= a.R) {
      u.place = LLONG_MAX;
      return;
    }
    u.x = load_request(a, u.r);
  } while (u.x.tiles == 0);
}

// What a row's weighted sum is multiplied by, and its lse, from its largest logit (`logit_of`)
// and the sum of its weights.
__device__ __forceinline__ float inverse_of(const KvAttendArgs& a, float logit, float all) {
  return all == 0.f ? 0.f : isnan(logit) ? logit : a.v_mul / all;
}
__device__ __forceinline__ float lse_of(float logit, float all) {
  return all == 0.f ? -INFINITY : (logit - kWeightExp + log2f(all)) * kLn2;
}

// Adds up n parts of a unit's workers first .. last in order, by `count` threads: those of
// workers w0, w0 + 1, ... or, if `groups`, those that stand for kFan workers each.
// Of its outputs (four dims of a row each) from .. to - 1; the sum goes to out and lse
// or, if `into` >= 0, to that part.  `factors`: of the unit's rows.  2^k lanes add up one output, each every 2^k-th
// part; what they load does not hang on what they loaded before.
template <typename T, int kDim, int NT>
__device__ void add_parts(const KvAttendArgs& a, const Parts& parts, const Note& u, int w0, int n, bool groups, int into,
                          const float* factors, int from, int to, int thread, int count) {
  using S = Shape<kDim, NT>;
  constexpr int kBatch = 4;
  int lanes = 1;
  while (lanes < 32 && 2 * lanes * (to - from) <= count && lanes < n) lanes *= 2;
  const int sub = thread & (lanes - 1);
  // every lane makes every round: the shuffles need all of them
  for (int at0 = from; at0 < to; at0 += count / lanes) {
    const int i = at0 + thread / lanes;
    const bool mine = i < to;
    const int row = mine ? i / (kDim / 4) : 0, j = mine ? i % (kDim / 4) : 0;
    const float f = factors[row];
    float m = -FLT_MAX, all = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = sub; k0 < n; k0 += kBatch * lanes) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int k = k0 + x * lanes, w = groups ? w0 + k * kFan : w0 + k;
        ml[x] = make_float2(-FLT_MAX, 0.f);
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < n) {   // from L2: other SMs wrote them
          const size_t at = (size_t)(groups && w < u.last ? S::group_part(w, u.first) : 2 * w + (w < u.last)) * S::kRows + row;
          ml[x] = __ldcg(parts.ml + at);
          v[x] = __ldcg(reinterpret_cast<const float4*>(parts.o + at * kDim) + j);
        }
      }
      float top = m;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) top = fmaxf(top, ml[x].x);
      const float c = ptx::ex2_approx((m - top) * f);
      m = top;
      all *= c;
      sum.x *= c;
      sum.y *= c;
      sum.z *= c;
      sum.w *= c;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const float y = ptx::ex2_approx((ml[x].x - top) * f);
        all += ml[x].y * y;
        sum.x += v[x].x * y;
        sum.y += v[x].y * y;
        sum.z += v[x].z * y;
        sum.w += v[x].w * y;
      }
    }
    for (int d = 1; d < lanes; d <<= 1) {
      const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, d), top = fmaxf(m, m2);
      const float c = ptx::ex2_approx((m - top) * f);
      m = top;
      all *= c;
      sum.x *= c;
      sum.y *= c;
      sum.z *= c;
      sum.w *= c;
      all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
      sum.x += __shfl_xor_sync(0xFFFFFFFFu, sum.x, d);
      sum.y += __shfl_xor_sync(0xFFFFFFFFu, sum.y, d);
      sum.z += __shfl_xor_sync(0xFFFFFFFFu, sum.z, d);
      sum.w += __shfl_xor_sync(0xFFFFFFFFu, sum.w, d);
    }
    if (!mine || sub) continue;
    if (into >= 0) {
      const size_t at = (size_t)into * S::kRows + row;
      reinterpret_cast<float4*>(parts.o + at * kDim)[j] = sum;
      if (j == 0) parts.ml[at] = make_float2(m, all);
      continue;
    }
    const int rho = u.row0 + row, q = query_of(a, rho), head = a.qhead[u.h * a.gamma + rho - q * a.gamma];
    const int64_t at = u.q0 + q;
    const float logit = logit_of(m, f), inv = inverse_of(a, logit, all);
    uint2 w;
    w.x = kv::float2_to_pair(sum.x * inv, sum.y * inv, static_cast<const T*>(nullptr));
    w.y = kv::float2_to_pair(sum.z * inv, sum.w * inv, static_cast<const T*>(nullptr));
    reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * a.out_stride + head * kDim)[j] = w;
    if (a.lse && j == 0) a.lse[at * a.Hq + head] = lse_of(logit, all);
  }
}

// One more at the counter: what this CTA's threads wrote before the barrier before
// this is seen by whoever reads the counter after.
__device__ __forceinline__ int count_in(int32_t* counter) {
  int n;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
  return n;
}

// Counts this worker's part of a unit in; the worker that completes the count adds
// the parts up.  sync: a barrier of the worker's threads; said: a word of theirs in
// shared memory; factors: of the unit's rows, written by the worker's threads.
template <typename T, int kDim, int NT, typename Sync>
__device__ __forceinline__ void finish_unit(const KvAttendArgs& a, const Parts& parts, const Unit& u, const Deal& deal, int worker, int thread,
                            int count, volatile int* said, const float* factors, Sync&& sync) {
  using S = Shape<kDim, NT>;
  const long long place = u.place + deal.cost;
  const int first = int(quotient(place, deal.share));
  const int last = min(int(quotient(place + u.x.tiles - 1, deal.share)), int(gridDim.x) * (deal.teams ? S::kTeams : 1) - 1);
  const int n = last - first + 1, row0 = u.c * S::kRows;
  const Note note{first, last, u.h, row0, u.x.q_len * a.gamma, u.x.q0};
  const int outputs = min(S::kRows, note.rows - row0) * (kDim / 4);
  auto arrive = [&](int32_t* counter) {   // how many came before
    sync();
    if (thread == 0) *said = count_in(counter);
    sync();
    return *said;
  };
  // level 0: the runs of kFan workers of a unit with more than that; level 1: the unit
  for (int level = n > kFan ? 0 : 1; level < 2; ++level) {
    const bool groups = level == 1 && n > kFan;
    const int w0 = level == 0 ? first + (worker - first) / kFan * kFan : first;
    const int members = groups ? (n + kFan - 1) / kFan : min(level == 0 ? kFan : n, last - w0 + 1);
    if (level == 0 && members == 1) continue;   // its part stands for itself
    int32_t* const counter = a.counters + (groups ? S::kMaxWorkers : 0) + w0;
    if (arrive(counter) != members - 1) break;
    if (thread == 0) *counter = 0;
    add_parts<T, kDim, NT>(a, parts, note, w0, members, groups, level == 0 ? S::group_part(w0, first) : -1, factors, 0, outputs,
                           thread, count);
    sync();   // the next unit's factors may be written
  }
}

// A team's barriers: one warp, or kMembers warps on the named barrier 1 + team.
template <int kMembers>
__device__ __forceinline__ void team_sync(int team) {
  if constexpr (kMembers == 1) __syncwarp();
  else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + team), "n"(32 * kMembers) : "memory");
}

// The same, and whether x holds in any thread of the team.
template <int kMembers>
__device__ __forceinline__ bool team_any(int team, bool x) {
  if constexpr (kMembers == 1) {
    return __any_sync(0xFFFFFFFFu, x);
  } else {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(x)), "r"(1 + team), "n"(32 * kMembers)
        : "memory");
    return r != 0;
  }
}

template <typename T, int kDim, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<kDim, NT>::kCtasPerSm)) kv_attend_kernel(const __grid_constant__ KvAttendArgs a, const __grid_constant__ Parts parts) {
  using S = Shape<kDim, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[S::kTeams][S::kStages];
  __shared__ longlong2 warp_sums[kWarps];
  __shared__ Unit starts[S::kTeams];
  __shared__ float sh_m[S::kTeams][S::kRows], sh_l[S::kTeams][S::kRows], sh_f[S::kTeams][S::kRows];
  __shared__ float sh_top[S::kRows], sh_all[S::kRows];
  __shared__ int sh_count[S::kTeams];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / S::kMembers, member = warp % S::kMembers;
  const int part = member / S::kHalves, half = member % S::kHalves;   // this warp's slice
  const int g = lane >> 2, t4 = lane & 3;
  if (member == 0 && lane == 0)
    for (int s = 0; s < S::kStages; ++s) ptx::mbar_init(ptx::smem_u32(&bars[team][s]), 1);
  ptx::fence_barrier_init();
  __syncthreads();   // the barriers are there for the team's other warps
  pdl_wait();

  // ---- this worker's share
  long long before;
  Request mine;
  bool empty;
  Deal deal;
  Unit u;
  int worker;
  if (a.R <= 32) {
    deal = deal_out_few(a, S::kRows, S::kTeams, before, mine, empty);
    worker = deal.teams ? blockIdx.x * S::kTeams + team : blockIdx.x;
    const long long first = worker * deal.share;
    // the last request with tiles that begins at or before the first place
    const uint32_t from = __ballot_sync(0xFFFFFFFFu, lane < a.R && mine.tiles > 0 && before <= first);
    const int r = from ? 31 - __clz(from) : 0;
    const long long at = __shfl_sync(0xFFFFFFFFu, before, r);
    if (first < deal.total) u = unit_at(a, r, load_request(a, r), at, first, deal.cost, S::kRows);
  } else {
    const int per = (a.R + kThreads - 1) / kThreads;
    deal = deal_out_many(a, S::kRows, S::kTeams, per, warp_sums, before, mine, empty);
    worker = deal.teams ? blockIdx.x * S::kTeams + team : blockIdx.x;
    const int workers = deal.teams ? S::kTeams : 1;   // of this CTA
    for (int j = 0; j < per; ++j) {
      // the thread whose requests hold a worker's first place finds its unit
      const int r = threadIdx.x * per + j;
      if (r >= a.R) break;
      const Request x = j ? load_request(a, r) : mine;
      if (x.tiles == 0) continue;
      const long long end = before + (long long)(x.tiles + deal.cost) * a.H * chunks_of(a, x, S::kRows);
      for (int w = 0; w < workers; ++w) {
        const long long first = (long long)(blockIdx.x * workers + w) * deal.share;
        if (first >= before && first < end) starts[w] = unit_at(a, r, x, before, first, deal.cost, S::kRows);
      }
      before = end;
    }
    __syncthreads();
    u = starts[deal.teams ? team : 0];
  }
  const int lg = deal.teams ? 0 : S::kLogTeams, group = 1 << lg, rank = deal.teams ? 0 : team;   // teams of a worker; which this is
  // rows that see nothing because their request has no entries
  for (int r = blockIdx.x; empty && r < a.R; r += gridDim.x) {
    const Request x = load_request(a, r);
    if (x.tiles) continue;
    for (int i = threadIdx.x; i < x.q_len * a.Hq * (kDim / 2); i += kThreads) {
      const int row = i / (kDim / 2), q = row / a.Hq, h = row - q * a.Hq;
      const int64_t at = x.q0 + q;
      reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * a.out_stride + h * kDim)[i % (kDim / 2)] = 0;
      if (a.lse && i % (kDim / 2) == 0) a.lse[at * a.Hq + h] = -INFINITY;
    }
  }
  if (parts.notes && threadIdx.x == 0) parts.notes[blockIdx.x].first = -1;
  const long long my_first = worker * deal.share, my_end = min(my_first + deal.share, deal.total);
  if (my_first >= deal.total) return;   // a whole CTA, or a team that meets no other again

  uint8_t* const ring = smem + team * S::kRing;
  uint8_t* const join = ring + member * (S::kRing / S::kMembers);
  float4* const exchange = reinterpret_cast<float4*>(smem + S::kTeams * S::kRing + team * S::kMembers * S::kExchange) + lane;
  const uint32_t bar0 = ptx::smem_u32(&bars[team][0]), ring0 = ptx::smem_u32(ring);
  // where in a record this lane's keys, values and their scales are
  const int k_at = part * (8 * S::kPart) + g * (S::kPart / 2) + t4 * (S::kPart / 8) + half * 8;
  const int ks_at = 16 * kDim + g * (kDim / 16) + part * 8 + (S::kPart == 128 ? 2 * t4 + half : t4);
  const int v_at = 8 * kDim + part * (8 * S::kPart) + lane * (S::kPart / 8) + half * 4;
  const int vs_at = 17 * kDim + part * S::kPart + (S::kPart == 128 ? g : g >> 1) * 8 + 2 * t4;
  const int dim0 = part * 128 + g * (S::kPart / 8) + half * 8;   // first of the lane's 2 kSteps dims of the output
  int stage = 0;                  // next stage to take
  uint32_t phase = 0;             // of its barrier
  uint32_t usable_ring = ~0u;     // two bits per stage: which of its records may be looked at
  bool dead = false;

  for (; u.place < my_end; next_unit(a, u, deal.cost, S::kRows)) {
    int begin = int(max(0LL, my_first - u.place - deal.cost));
    int end = int(min((long long)u.x.tiles, my_end - u.place - deal.cost));
    if (deal.teams && u.x.tiles <= kWholeUnit) {
      begin = 0;
      end = u.place < my_first ? 0 : u.x.tiles;
    }
    if (end <= begin) continue;

    // ---- the unit's rows, asked for before the copies so that they do not queue behind them
    const int row0 = u.c * S::kRows, rows = u.x.q_len * a.gamma;   // rows of the request
    const int base = u.x.n - u.x.q_len;                            // position of query 0
    // Words of the lane's quarter of each slice, its own slice's first (the others count for the
    // largest element only).
    constexpr int kWords = S::kSlice / 8;
    uint32_t raw[NT][S::kMembers][kWords];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rho = row0 + nt * 8 + g;
      const bool real = rho < rows;
      const int i = real ? query_of(a, rho) : 0, j = real ? rho - i * a.gamma : 0;
      const T* src = static_cast<const T*>(a.q) + (int64_t)(u.x.q0 + i) * a.q_stride + (int)a.qhead[u.h * a.gamma + j] * kDim;
#pragma unroll
      for (int p = 0; p < S::kMembers; ++p) {
        const int slice = (member + p) % S::kMembers;
        const uint4* v = reinterpret_cast<const uint4*>(src + slice / S::kHalves * 128 + t4 * (S::kPart / 4) +
                                                        slice % S::kHalves * 16);
#pragma unroll
        for (int x = 0; x < kWords / 4; ++x) {
          const uint4 y = real ? v[x] : make_uint4(0, 0, 0, 0);
          raw[nt][p][4 * x] = y.x;
          raw[nt][p][4 * x + 1] = y.y;
          raw[nt][p][4 * x + 2] = y.z;
          raw[nt][p][4 * x + 3] = y.w;
        }
      }
    }

    // ---- the copies.  The lanes know the records of the team's next 16 tiles: lane 2 i + b the
    // b-th record of the i-th.  The team's first warp has them copied.
    const int todo = dead || begin + rank >= end ? 0 : (end - begin - rank + group - 1) >> lg;   // this team's tiles
    int left = todo, src = 16, refill = begin + rank;
    const uint8_t* record = nullptr;
    uint32_t usable = 0;
    auto entry_of = [&](int t) { return (t < u.x.sink_t ? t : t - u.x.sink_t + u.x.lo_t) * kTile; };
    auto issue = [&](int s) {   // the next tile into stage s
      if (left == 0) return;
      --left;
      if (src == 16) {
        src = 0;
        const int tile = refill + ((lane >> 1) << lg);
        refill += 16 << lg;
        bool ok = false;
        if (tile < end) {
          const int e0 = entry_of(tile) + (lane & 1) * 16;
          if (e0 < u.x.n && (e0 + 15 >= u.x.lo || e0 < u.x.sinks)) {
            const int page = a.page_table[(int64_t)u.r * a.page_stride + (e0 >> a.page_shift)];
            const int64_t b = ((int64_t)page << (a.page_shift - 4)) + ((e0 & ((1 << a.page_shift) - 1)) >> 4);
            ok = page >= 0 && b < (a.num_slots >> 4);
            if (!ok) set_status(a.status, UPF_ERR_INVALID_ARG);
            record = a.data + (b * a.H + u.h) * S::kRecord;
          }
        }
        usable = __ballot_sync(0xFFFFFFFFu, ok);
      }
      const uint32_t two = usable & 3u;
      usable >>= 2;
      if (two != 3u) usable_ring &= ~((two ^ 3u) << (2 * s));
      if (member == 0 && (lane >> 1) == src) {
        const uint32_t bar = bar0 + 8 * s;
        if ((lane & 1) == 0) ptx::mbar_arrive_expect_tx(bar, two == 3u ? 2 * S::kRecord : two ? S::kRecord : 0);
        if ((two >> (lane & 1)) & 1u)
          ptx::bulk_load(ring0 + s * S::kStage + (lane & 1) * S::kRecord, record, S::kRecord, bar);
      }
      ++src;
    };
    for (int i = 0, s = stage; i < S::kStages; ++i) {
      issue(s);
      if (++s == S::kStages) s = 0;
    }
    __syncwarp();

    // ---- the rows as operand B, divided by the power of two of their largest element
    uint32_t qf[S::kSteps][NT][2];
    float f[NT][2];          // logit factor of rows 2 t4, 2 t4 + 1 of each eight
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t top = 0;
#pragma unroll
      for (int p = 0; p < S::kMembers; ++p)
#pragma unroll
        for (int x = 0; x < kWords; ++x) top = kv::max_abs2(top, raw[nt][p][x], static_cast<const T*>(nullptr));
      const float2 tops = kv::pair_to_float2(top, static_cast<const T*>(nullptr));
      float amax = fmaxf(fabsf(tops.x), fabsf(tops.y));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // 2^-e with e the exponent of the largest element (0 for a row of zeros)
      int e = int(__float_as_uint(amax) >> 23) - 127;
      e = amax == 0.f ? 0 : max(-126, min(e, 126));
      // An infinite query makes every logit infinite or NaN, and their softmax NaN; where all are -inf, NaN
      // queries tell that from entries that are not seen.
      const float down = __uint_as_float(amax <= FLT_MAX ? uint32_t(127 - e) << 23 : 0x7FFFFFFFu);
#pragma unroll
      for (int x = 0; x < kWords; ++x) {
        const float2 y = kv::pair_to_float2(raw[nt][0][x], static_cast<const T*>(nullptr));
        qf[x / 2][nt][x & 1] = pack_f16(y.x * down, y.y * down);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) f[nt][b] = factor_of(a, a.scale_exp + __shfl_sync(0xFFFFFFFFu, e, (2 * t4 + b) * 4));
    }
    const int p_min = base + query_of(a, row0), p_max = base + query_of(a, min(rows, row0 + S::kRows) - 1);
    // does row y of this lane's columns (nt, b) see entry e?
    auto sees = [&](int nt, int b, int e) {
      const int y = row0 + nt * 8 + 2 * t4 + b, p = base + query_of(a, y);
      return y < rows && e <= p && (a.window == 0 || p - e < a.window || e < a.sinks);
    };

    // weights are 2^((s - ref) f + 12); the reference moves when s passes `limit`
    float o[S::kSteps][NT][4];
    float ref[NT][2], limit[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        ref[nt][b] = limit[nt][b] = -FLT_MAX;
        l[nt][b] = 0.f;
#pragma unroll
        for (int mt = 0; mt < S::kSteps; ++mt) o[mt][nt][b] = o[mt][nt][b + 2] = 0.f;
      }

    // One tile from the records at `rec`; masked: some row does not see some entry of it, or a record of
    // it may not be looked at (bits of `two`).  `late`: this warp's wait for the tile ran out;
    // returns whether any of the team's did (then nothing is added).
    auto work = [&](auto masked, const uint8_t* rec, int e0, uint32_t two, bool late) {
      constexpr bool kMasked = decltype(masked)::value;
      // ---- logits: S^T[entry][row]
      float s[2][NT][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint8_t* const rb = rec + b * S::kRecord;
        constexpr int kW = S::kSlice / 32;   // words of a lane's quarter row: 2 or 4
        uint32_t w[2][kW];
        __half2 sc[2];                       // scales of the quarter's first and second group
#pragma unroll
        for (int y8 = 0; y8 < 2; ++y8) {
          const uint8_t* const src = rb + k_at + y8 * (4 * S::kPart);
          const uint8_t* const scale = rb + ks_at + y8 * (kDim / 2);
          if constexpr (kW == 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(src);
            w[y8][0] = y.x;
            w[y8][1] = y.y;
            w[y8][2] = y.z;
            w[y8][3] = y.w;
            sc[y8] = as_half2(kv::e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(scale)));
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            w[y8][0] = y.x;
            w[y8][1] = y.y;
            sc[y8] = as_half2(kv::e4m3x2_to_f16x2(*scale));
          }
        }
#pragma unroll
        for (int x = 0; x < kW; ++x) {   // eight dims of the lane: two steps
          uint32_t x0[4], x1[4];
          kv::e2m1x8_to_f16(w[0][x], x0);
          kv::e2m1x8_to_f16(w[1][x], x1);
          const bool second = kW == 4 && x >= 2;
          const __half2 s0 = second ? __high2half2(sc[0]) : __low2half2(sc[0]);
          const __half2 s1 = second ? __high2half2(sc[1]) : __low2half2(sc[1]);
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint32_t af[4] = {hmul2(x0[2 * st], s0), hmul2(x1[2 * st], s1), hmul2(x0[2 * st + 1], s0),
                                    hmul2(x1[2 * st + 1], s1)};
            const int step = 2 * x + st;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (step == 0) mma_f16_zero(s[b][nt], af, qf[step][nt]);
              else mma_f16(s[b][nt], af, qf[step][nt]);
            }
          }
        }
      }
      if constexpr (S::kMembers > 1) {
        // the members' logits add up in the same order for all of them
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            exchange[(member * 2 * NT + b * NT + nt) * 32] = make_float4(s[b][nt][0], s[b][nt][1], s[b][nt][2], s[b][nt][3]);
        if (team_any<S::kMembers>(team, late)) return true;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float4 y = exchange[(b * NT + nt) * 32];
#pragma unroll
            for (int p = 1; p < S::kMembers; ++p) {
              const float4 z = exchange[(p * 2 * NT + b * NT + nt) * 32];
              y.x += z.x;
              y.y += z.y;
              y.z += z.z;
              y.w += z.w;
            }
            s[b][nt][0] = y.x;
            s[b][nt][1] = y.y;
            s[b][nt][2] = y.z;
            s[b][nt][3] = y.w;
          }
      }
      // ---- weights, in f16 as operand B of the second product
      if constexpr (kMasked) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((two >> b) & 1u) || !sees(nt, i & 1, e0 + 16 * b + g + 8 * (i >> 1))) s[b][nt][i] = -INFINITY;
      }
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          over |= fmaxf(fmaxf(s[0][nt][i], s[1][nt][i]), fmaxf(s[0][nt][i + 2], s[1][nt][i + 2])) > limit[nt][i];
      if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float x = fmaxf(fmaxf(s[0][nt][b], s[0][nt][b + 2]), fmaxf(s[1][nt][b], s[1][nt][b + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
            if (x > limit[nt][b]) {
              const float k = ptx::ex2_approx((ref[nt][b] - x) * f[nt][b]);
              ref[nt][b] = x;
              limit[nt][b] = __fadd_rd(x, __fdividef(kLag, f[nt][b]));   // down: the weights' range ends there
              l[nt][b] *= k;
#pragma unroll
              for (int mt = 0; mt < S::kSteps; ++mt) {
                o[mt][nt][b] *= k;
                o[mt][nt][b + 2] *= k;
              }
            }
          }
        __syncwarp();   // the matrix instructions below take whole warps
      }
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = ptx::ex2_approx(__fmaf_rn(s[b][nt][i] - ref[nt][i & 1], f[nt][i & 1], kWeightExp));
            l[nt][i & 1] += w[i];
          }
          pf[b][nt][0] = transpose8x8(pack_f16(w[0], w[1]));
          pf[b][nt][1] = transpose8x8(pack_f16(w[2], w[3]));
        }
      // ---- weighted sum: O^T[dim][row]
      uint32_t bad = 0;   // a NaN scale among the values of a tile with unseen entries
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint8_t* const rb = rec + b * S::kRecord;
        constexpr int kW = S::kSlice / 64;   // words of a lane's dims of an entry: 1 or 2
        uint32_t w[2][2][kW];                // [entries 2 t4.. or 2 t4 + 8..][entry of the two]
        __half2 sc[2];
#pragma unroll
        for (int y8 = 0; y8 < 2; ++y8) {
          const uint8_t* const src = rb + v_at + y8 * (4 * S::kPart);
          if constexpr (kW == 2) {
            const uint4 y = *reinterpret_cast<const uint4*>(src);
            w[y8][0][0] = y.x;
            w[y8][0][1] = y.y;
            w[y8][1][0] = y.z;
            w[y8][1][1] = y.w;
          } else if constexpr (S::kHalves == 1) {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            w[y8][0][0] = y.x;
            w[y8][1][0] = y.y;
          } else {
            w[y8][0][0] = *reinterpret_cast<const uint32_t*>(src);
            w[y8][1][0] = *reinterpret_cast<const uint32_t*>(src + 8);
          }
          uint32_t raw_sc = *reinterpret_cast<const uint16_t*>(rb + vs_at + y8 * (S::kPart / 2));
          if constexpr (kMasked) {
            // 0 * NaN would reach the rows that do not see the entry: take the scale as 0 and
            // give the NaN to the rows that do see it below
            if ((raw_sc & 0x7Fu) == 0x7Fu) {
              raw_sc &= 0xFF00u;
              bad = 1;
            }
            if ((raw_sc & 0x7F00u) == 0x7F00u) {
              raw_sc &= 0x00FFu;
              bad = 1;
            }
          }
          sc[y8] = as_half2(kv::e4m3x2_to_f16x2(uint16_t(raw_sc)));
        }
        if constexpr (kMasked) __syncwarp();
#pragma unroll
        for (int x = 0; x < kW; ++x) {
          // low nibbles of both entries side by side (even dims), then the high ones
          uint32_t lo[2][4], hi[2][4];
#pragma unroll
          for (int y8 = 0; y8 < 2; ++y8) {
            kv::e2m1x8_to_f16(merge_bits(w[y8][0][x], w[y8][1][x] << 4, 0x0F0F0F0Fu), lo[y8]);
            kv::e2m1x8_to_f16(merge_bits(w[y8][0][x] >> 4, w[y8][1][x], 0x0F0F0F0Fu), hi[y8]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t af[4] = {hmul2(lo[0][j], sc[0]), hmul2(hi[0][j], sc[0]), hmul2(lo[1][j], sc[1]),
                                    hmul2(hi[1][j], sc[1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[4 * x + j][nt], af, pf[b][nt]);
          }
        }
      }
      if (kMasked && __any_sync(0xFFFFFFFFu, bad)) {
        for (int b = 0; b < 2; ++b)
          for (int row = 0; row < 16; ++row) {
            const int e = e0 + 16 * b + row;
            const int grp = part * (S::kPart / 16) + (S::kPart == 128 ? g : g >> 1);
            const bool nan = (rec[b * S::kRecord + kv::v_scale(kDim, row, grp)] & 0x7F) == 0x7F;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int d = 0; d < 2; ++d)
                if (nan && ((two >> b) & 1u) && sees(nt, d, e))
#pragma unroll
                  for (int mt = 0; mt < S::kSteps; ++mt) o[mt][nt][d] = o[mt][nt][d + 2] = __int_as_float(0x7FFFFFFF);
          }
      }
      return false;
    };

    // tiles [whole0, whole0 + wholes) lie inside every row's window and before every row's position
    const int whole0 = u.x.sink_t - u.x.lo_t + (a.window ? (max(0, p_max - a.window + 1) + kTile - 1) / kTile : 0);
    const uint32_t wholes = max(0, u.x.sink_t - u.x.lo_t + (p_min + 1) / kTile - whole0);
    for (int i = 0, t = begin + rank; i < todo; ++i, t += group) {
      bool late = !ptx::mbar_wait_poll(bar0 + 8 * stage, phase, a.wait_limit, 64);
      late = __any_sync(0xFFFFFFFFu, late);   // one answer, and the lanes together again for the matrix instructions
      if (S::kMembers > 1 || !late) {
        const uint8_t* const rec = ring + stage * S::kStage;
        const uint32_t two = (usable_ring >> (2 * stage)) & 3u;
        if (two == 3u && uint32_t(t - whole0) < wholes) {
          late = work(std::false_type(), rec, 0, 3u, late);
        } else {
          late = work(std::true_type(), rec, entry_of(t), two, late);
          usable_ring |= 3u << (2 * stage);
        }
      }
      if (late) {
        // a copy did not come in time: no more work, the team's own copies are waited for
        if (lane == 0) set_status(a.status, UPF_ERR_TIMEOUT);
        dead = true;
        for (int flying = todo - left - i; flying > 0; --flying) {
          ptx::mbar_wait(bar0 + 8 * stage, phase, kDefaultWaitCycles);
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        break;
      }
      team_sync<S::kMembers>(team);
      issue(stage);
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }

    // ---- write the unit, or this worker's part of it
    const bool goes_on = end < u.x.tiles, alone = !goes_on && begin == 0;
    const size_t slot = (size_t)2 * worker + (goes_on ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][b] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][b], d);
    if (deal.teams) {
      // straight from the registers: a lane holds 2 kSteps dims of its two columns
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int row = nt * 8 + 2 * t4 + b, rho = row0 + row;
          if (rho >= rows) continue;
          const float all = l[nt][b];
          if (alone) {
            const int qi = query_of(a, rho), head = a.qhead[u.h * a.gamma + rho - qi * a.gamma];
            const int64_t at = u.x.q0 + qi;
            const float logit = logit_of(ref[nt][b], f[nt][b]), inv = inverse_of(a, logit, all);
            uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * a.out_stride + head * kDim + dim0);
#pragma unroll
            for (int mt = 0; mt < S::kSteps; mt += 4) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = kv::float2_to_pair(o[mt + i][nt][b] * inv, o[mt + i][nt][b + 2] * inv, static_cast<const T*>(nullptr));
              *reinterpret_cast<uint4*>(dst + mt) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (g == 0 && member == 0 && a.lse) a.lse[at * a.Hq + head] = lse_of(logit, all);
          } else {
            float* const dst = parts.o + (slot * S::kRows + row) * kDim + dim0;
#pragma unroll
            for (int mt = 0; mt < S::kSteps; mt += 2)
              *reinterpret_cast<float4*>(dst + 2 * mt) =
                  make_float4(o[mt][nt][b], o[mt][nt][b + 2], o[mt + 1][nt][b], o[mt + 1][nt][b + 2]);
            if (g == 0 && member == 0) {
              parts.ml[slot * S::kRows + row] = make_float2(ref[nt][b], all);
              sh_f[team][row] = f[nt][b];
            }
          }
        }
    } else {
      if (member == 0 && g == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            sh_m[team][nt * 8 + 2 * t4 + b] = ref[nt][b];
            sh_l[team][nt * 8 + 2 * t4 + b] = l[nt][b];
            sh_f[team][nt * 8 + 2 * t4 + b] = f[nt][b];   // the same for every team
          }
      }
      __syncthreads();
      if (threadIdx.x < S::kRows) {
        const float fr = sh_f[0][threadIdx.x];
        float top = -FLT_MAX, all = 0.f;
#pragma unroll
        for (int w = 0; w < S::kTeams; ++w) top = fmaxf(top, sh_m[w][threadIdx.x]);
#pragma unroll
        for (int w = 0; w < S::kTeams; ++w) all += sh_l[w][threadIdx.x] * ptx::ex2_approx((sh_m[w][threadIdx.x] - top) * fr);
        sh_top[threadIdx.x] = top;
        sh_all[threadIdx.x] = all;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float scale[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float top = -FLT_MAX;
#pragma unroll
          for (int w = 0; w < S::kTeams; ++w) top = fmaxf(top, sh_m[w][nt * 8 + 2 * t4 + b]);
          scale[b] = ptx::ex2_approx((ref[nt][b] - top) * f[nt][b]);
        }
#pragma unroll
        for (int mt = 0; mt < S::kSteps; ++mt) {
          float* const dst = reinterpret_cast<float*>(join) + (nt * 8 + 2 * t4) * S::kJoinRow + mt * 16 + g * 2;
          *reinterpret_cast<float2*>(dst) = make_float2(o[mt][nt][0] * scale[0], o[mt][nt][2] * scale[0]);
          *reinterpret_cast<float2*>(dst + S::kJoinRow) = make_float2(o[mt][nt][1] * scale[1], o[mt][nt][3] * scale[1]);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < S::kRows * kDim / 2; i += kThreads) {
        const int row = i / (kDim / 2), j = i % (kDim / 2) / (S::kSlice / 2), y = i % (S::kSlice / 2);   // y: dims (mt = y / 8, g = y % 8) of slice j
        const int rho = row0 + row;
        if (rho >= rows) continue;
        const int dim = j / S::kHalves * 128 + (y % 8) * (S::kPart / 8) + j % S::kHalves * 8 + 2 * (y / 8);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < S::kTeams; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(smem + w * S::kRing + j * (S::kRing / S::kMembers) +
                                                            (row * S::kJoinRow + 2 * y) * 4);
          sum.x += v.x;
          sum.y += v.y;
        }
        const float all = sh_all[row];
        if (alone) {
          const int qi = query_of(a, rho), head = a.qhead[u.h * a.gamma + rho - qi * a.gamma];
          const int64_t at = u.x.q0 + qi;
          const float logit = logit_of(sh_top[row], sh_f[0][row]), inv = inverse_of(a, logit, all);
          *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * a.out_stride + head * kDim + dim) =
              kv::float2_to_pair(sum.x * inv, sum.y * inv, static_cast<const T*>(nullptr));
          if (a.lse && dim == 0) a.lse[at * a.Hq + head] = lse_of(logit, all);
        } else {
          *reinterpret_cast<float2*>(parts.o + (slot * S::kRows + row) * kDim + dim) = sum;
          if (dim == 0) {
            parts.ml[slot * S::kRows + row] = make_float2(sh_top[row], all);
            if (goes_on) parts.f[blockIdx.x * S::kRows + row] = sh_f[0][row];
          }
        }
      }
      // the rings take copies again, sh_m, sh_l, sh_top and sh_all new values
      ptx::fence_proxy_async_smem();
      __syncthreads();
    }
    if (parts.notes && !deal.teams) {
      if (goes_on && threadIdx.x == 0) {
        const long long place = u.place + deal.cost;
        parts.notes[blockIdx.x] = Note{int(quotient(place, deal.share)), int(quotient(place + u.x.tiles - 1, deal.share)),
                                       u.h, row0, rows, u.x.q0};
      }
    } else if (!alone) {
      finish_unit<T, kDim, NT>(a, parts, u, deal, worker, deal.teams ? member * 32 + lane : threadIdx.x,
                               deal.teams ? 32 * S::kMembers : kThreads, &sh_count[deal.teams ? team : 0], sh_f[deal.teams ? team : 0], [&] {
                                 if (deal.teams) team_sync<S::kMembers>(team);
                                 else __syncthreads();
                               });
    }
  }
}

// The second launch: each warp of the CTAs first .. last - 1 of a unit takes its portion
// of the outputs.
template <typename T, int kDim, int NT>
__global__ void __launch_bounds__(kThreads) kv_attend_join_kernel(const __grid_constant__ KvAttendArgs a,
                                                                  const __grid_constant__ Parts parts) {
  using S = Shape<kDim, NT>;
  pdl_wait();
  const Note u = parts.notes[blockIdx.x];
  if (u.first < 0) return;
  const int outputs = min(S::kRows, u.rows - u.row0) * (kDim / 4), portions = (u.last - u.first) * kWarps;
  const int each = (outputs + portions - 1) / portions;
  const int from = ((blockIdx.x - u.first) * kWarps + (threadIdx.x >> 5)) * each;
  add_parts<T, kDim, NT>(a, parts, u, u.first, u.last - u.first + 1, false, -1, parts.f + u.first * S::kRows, from,
                         min(outputs, from + each), threadIdx.x & 31, 32);
}

template <int kDim, int NT>
constexpr size_t part_rows() {
  return (size_t)Shape<kDim, NT>::kPartSlots * Shape<kDim, NT>::kRows;
}

template <typename T, int kDim, int NT>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t s) {
  using S = Shape<kDim, NT>;
  Parts parts;
  parts.o = static_cast<float*>(a.ws);
  parts.ml = reinterpret_cast<float2*>(parts.o + part_rows<kDim, NT>() * kDim);
  // once a device (setting it twice does no harm)
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (a.device & 63);
  cudaError_t e = cudaSuccess;
  if (a.device > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kv_attend_kernel<T, kDim, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  // Most CTAs that can come to work on one unit, if the units are about as long as one another:
  // all CTAs by the units, or the longest unit by the least share.
  const long long units = (long long)a.R * a.H * ((a.max_q * a.gamma + S::kRows - 1) / S::kRows);
  const long long longest = a.window ? (long long)a.window + a.sinks + a.max_q : (long long)a.max_pages << a.page_shift;
  const bool second = std::min(S::kCtas / units, longest / (kTile * S::kTeams)) > kFan;
  parts.f = reinterpret_cast<float*>(parts.ml + part_rows<kDim, NT>());
  parts.notes = second ? reinterpret_cast<Note*>(parts.f + S::kCtas * S::kRows) : nullptr;
  e = launch_kernel(kv_attend_kernel<T, kDim, NT>, S::kCtas, kThreads, S::kSmem, s, true, a, parts);
  if (e != cudaSuccess || !second) return e;
  return launch_kernel(kv_attend_join_kernel<T, kDim, NT>, S::kCtas, kThreads, 0, s, true, a, parts);
}

template <int kDim>
cudaError_t launch_dim(const KvAttendArgs& a, bool f16, cudaStream_t s) {
  if (a.gamma * a.max_q <= 8) return f16 ? launch<__half, kDim, 1>(a, s) : launch<__nv_bfloat16, kDim, 1>(a, s);
  return f16 ? launch<__half, kDim, 2>(a, s) : launch<__nv_bfloat16, kDim, 2>(a, s);
}

template <int kDim, int NT>
constexpr size_t ws_bytes() {
  using S = Shape<kDim, NT>;
  return part_rows<kDim, NT>() * (kDim * sizeof(float) + sizeof(float2)) + S::kCtas * (S::kRows * sizeof(float) + sizeof(Note));
}

template <int kDim>
size_t ws_bytes_dim(int rows) {
  return rows <= 8 ? ws_bytes<kDim, 1>() : ws_bytes<kDim, 2>();
}

}  // namespace

size_t kv_attend_workspace_bytes(int gamma, int max_q, int d) {
  const int rows = gamma * max_q;
  return d == 64 ? ws_bytes_dim<64>(rows) : d == 128 ? ws_bytes_dim<128>(rows) : ws_bytes_dim<256>(rows);
}

cudaError_t launch_kv_attend(const KvAttendArgs& a, bool f16, cudaStream_t s) {
  return a.d == 64 ? launch_dim<64>(a, f16, s) : a.d == 128 ? launch_dim<128>(a, f16, s) : launch_dim<256>(a, f16, s);
}

}  // namespace upf
