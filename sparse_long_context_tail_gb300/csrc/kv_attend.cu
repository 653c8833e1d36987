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
// the CTAs in equal shares, from the lengths in device memory: ragged batches
// balance themselves and a captured call stays valid when the lengths change.  A
// CTA's warps take its tiles in turn, each with its own ring of records filled by
// bulk copies (two records of 18 d bytes a tile), its own running reference and
// sums; at the end of a unit the CTA joins its warps through shared memory.  A
// unit that lies in one CTA's share is written out at once; others leave a part
// (reference, sum, weighted sum, all fp32) per CTA in the workspace, which
// kv_attend_join_kernel adds up in a fixed order, so results repeat bit for bit.
//
// Arithmetic.  A code times its scale has at most six significant bits and is
// exact in f16, and so is a query after division by the power of two of its
// row's largest element (elements 2^-14 below it lose their last bits: 2^-25 of
// the largest, under the fp32 sum's own rounding).  Logits, references, sums and the
// weighted sums are fp32.  The one rounding is that of the softmax weights to f16,
// 2^-11 relative; they are scaled by 2^12 against a reference that may lag the
// running maximum by 2^3, so that weights down to 2^-26 of the reference keep all
// their bits.
#include <cfloat>

#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

constexpr int kWarps = 4;        // of a CTA
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

__device__ __forceinline__ int chunks_of(const KvAttendArgs& a, const Request& x, int rows) {
  return (x.q_len * a.gamma + rows - 1) / rows;
}

// Tiles of all requests up to the first that a thread looks at, and the total.
// Thread i looks at requests [i * per, (i + 1) * per).
template <int kCount>
__device__ long long scan_tiles(const KvAttendArgs& a, int rows, int per, long long (&warp_sums)[kCount / 32],
                                long long& total) {
  long long mine = 0;
  for (int j = 0; j < per; ++j) {
    const int r = threadIdx.x * per + j;
    if (r >= a.R) break;
    const Request x = load_request(a, r);
    mine += (long long)x.tiles * a.H * chunks_of(a, x, rows);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, s);
    if (lane >= s) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
  total = 0;
#pragma unroll
  for (int w = 0; w < kCount / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before;
}

// Tiles per CTA: an equal share, and at least one for every warp.
__device__ __forceinline__ long long share_of(long long total, int ctas) {
  const long long s = (total + ctas - 1) / ctas;
  return s < kWarps ? kWarps : s;
}

// The workspace.  A CTA works on at most two units that others work on too: the
// one its share begins in the middle of, and the one that goes on after its
// share.  The part of the latter (or of a unit that does both) is at 2 c + 1, that
// of the former at 2 c, and the CTAs c0 .. c1 - 1 of a shared unit, for which it is
// the latter, note it for the join.
struct Shared {
  int c0, c1;             // CTAs of the unit (c0 < 0: no unit goes on after this CTA's share)
  int h, row0, rows, q0;  // kv head, first row of the chunk, rows of the request, its first row in q
};

struct Parts {
  float* o;         // [2 ctas][rows][d]
  float2* ml;       // [2 ctas][rows]: reference, sum
  Shared* shared;   // [ctas]
};

// ------------------------------------------------------------ main kernel --

template <int kDim, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kParts = kDim >= 128 ? kDim / 128 : 1;
  static constexpr int kPart = kDim / kParts;          // dims per part: 64 or 128
  static constexpr int kSteps = kPart / 16;            // mma steps over the dims of a part, and dim tiles of it
  static constexpr int kRecord = kv::record_bytes(kDim);
  static constexpr int kStage = 2 * kRecord;
  static constexpr int kStages = kDim == 64 ? 4 : 2;
  static constexpr bool kQueryInSmem = kDim * NT > 256;
  static constexpr int kCtasPerSm = kDim == 64 ? 4 : kDim == 128 ? (NT == 1 ? 4 : 3) : 2;
  static constexpr int kJoinRow = kPart + 4;           // floats; the pad spreads the rows over the banks
  static constexpr int kJoinBytes = kWarps * kRows * kJoinRow * 4;
  static constexpr int kQueryBytes = kQueryInSmem ? kRows * kDim * 2 : 0;
  static constexpr int kSmem = kWarps * kStages * kStage + kJoinBytes + kQueryBytes;
  static constexpr int kCtas = kCtasPerSm * kPlanSMs;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// (x & m) | (y & ~m)
__device__ __forceinline__ uint32_t merge_bits(uint32_t x, uint32_t y, uint32_t m) { return (x & m) | (y & ~m); }

// Where in the tiles of all units a CTA or warp stands.
struct Cursor {
  int r, h, c;        // request, kv head, chunk
  int t, end;         // tile of the unit, and the end of this CTA's tiles of it
  long long left;     // tiles of the CTA's share from t on
  Request x;
};

// Enter the unit at (r, h, c) from tile t; units without tiles are passed over.
__device__ __forceinline__ void enter(const KvAttendArgs& a, Cursor& k, int rows) {
  while (k.left > 0 && k.r < a.R) {
    if (k.c == 0 && k.h == 0) k.x = load_request(a, k.r);
    if (k.x.tiles > 0 && k.c < chunks_of(a, k.x, rows)) {
      k.end = int(min((long long)k.x.tiles, k.t + k.left));
      return;
    }
    k.c = 0;
    if (++k.h == a.H || k.x.tiles == 0 || k.x.q_len == 0) {
      k.h = 0;
      ++k.r;
    }
  }
  k.left = 0;
}

__device__ __forceinline__ void next_unit(const KvAttendArgs& a, Cursor& k, int from, int rows) {
  k.left -= k.end - from;
  k.t = 0;
  ++k.c;
  enter(a, k, rows);
}

template <typename T, int kDim, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<kDim, NT>::kCtasPerSm)) kv_attend_kernel(const KvAttendArgs a, const Parts parts) {
  using S = Shape<kDim, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][S::kStages];
  __shared__ long long warp_sums[kWarps];
  __shared__ Cursor start;
  __shared__ float sh_m[kWarps][S::kRows], sh_l[kWarps][S::kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  pdl_trigger();

  // ---- this CTA's share
  const int per = (a.R + kThreads - 1) / kThreads;
  long long total;
  const long long before = scan_tiles<kThreads>(a, S::kRows, per, warp_sums, total);
  const long long share = share_of(total, gridDim.x);
  const long long first = blockIdx.x * share;
  // rows that see nothing because their request has no entries
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const Request x = load_request(a, r);
    if (x.tiles) continue;
    for (int i = threadIdx.x; i < x.q_len * a.Hq * (kDim / 2); i += kThreads) {
      const int row = i / (kDim / 2), q = row / a.Hq, h = row - q * a.Hq;
      const int64_t at = x.q0 + q;
      reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * a.out_stride + h * kDim)[i % (kDim / 2)] = 0;
      if (a.lse && i % (kDim / 2) == 0) a.lse[at * a.Hq + h] = -INFINITY;
    }
  }
  if (first >= total) {
    if (threadIdx.x == 0) parts.shared[blockIdx.x].c0 = -1;
    return;
  }
  {
    // the thread whose requests hold tile `first` finds its place
    long long at = before;
    for (int j = 0; j < per; ++j) {
      const int r = threadIdx.x * per + j;
      if (r >= a.R) break;
      Cursor k;
      k.x = load_request(a, r);
      const int chunks = chunks_of(a, k.x, S::kRows);
      const long long n = (long long)k.x.tiles * a.H * chunks;
      if (first >= at && first < at + n) {
        const long long in = first - at;
        const int unit = int(in / k.x.tiles);
        k.r = r;
        k.h = unit / chunks;
        k.c = unit % chunks;
        k.t = int(in % k.x.tiles);
        k.left = min(share, total - first);
        k.end = int(min((long long)k.x.tiles, k.t + k.left));
        start = k;
      }
      at += n;
    }
  }
  if (lane == 0)
    for (int s = 0; s < S::kStages; ++s) ptx::mbar_init(ptx::smem_u32(&bars[warp][s]), 1);
  ptx::fence_barrier_init();
  __syncthreads();

  uint8_t* const ring = smem + warp * (S::kStages * S::kStage);
  float* const join = reinterpret_cast<float*>(smem + kWarps * S::kStages * S::kStage);
  __half* const sq = reinterpret_cast<__half*>(smem + kWarps * S::kStages * S::kStage + S::kJoinBytes);
  const uint32_t bar0 = ptx::smem_u32(&bars[warp][0]), ring0 = ptx::smem_u32(ring);

  // ---- the copies: a second cursor ahead of the one that is being worked on
  Cursor ic = start;
  int it = ic.t + warp;          // the warp's next tile to fetch
  int held = -1;                 // first of the 16 tiles whose records the lanes know
  uint32_t block = 0;            // lane: record of tile held + kWarps * (lane / 2), half lane % 2
  uint32_t usable = 0, usable_ring = 0;   // bit per lane; two bits per stage
  int issued = 0, taken = 0, fill = 0;
  bool dead = false;

  auto issue = [&]() {
    if (dead) return;
    while (ic.left > 0 && it >= ic.end) {
      next_unit(a, ic, ic.t, S::kRows);
      it = warp;
      held = -1;
    }
    if (ic.left <= 0) return;
    if (held < 0 || it >= held + 16 * kWarps) {
      held = it;
      const int tile = it + kWarps * (lane >> 1);
      bool ok = false;
      if (tile < ic.end) {
        const int e0 = (tile < ic.x.sink_t ? tile : tile - ic.x.sink_t + ic.x.lo_t) * kTile + (lane & 1) * 16;
        if (e0 < ic.x.n && (e0 + 15 >= ic.x.lo || e0 < ic.x.sinks)) {
          const int page = a.page_table[(int64_t)ic.r * a.page_stride + (e0 >> a.page_shift)];
          const int64_t b = ((int64_t)page << (a.page_shift - 4)) + ((e0 & ((1 << a.page_shift) - 1)) >> 4);
          ok = page >= 0 && b < (a.num_slots >> 4);
          if (!ok) set_status(a.status, UPF_ERR_INVALID_ARG);
          block = uint32_t(b);
        }
      }
      usable = __ballot_sync(0xFFFFFFFFu, ok);
    }
    const int src = (it - held) / kWarps * 2;
    const uint32_t two = (usable >> src) & 3u;
    const uint32_t b0 = __shfl_sync(0xFFFFFFFFu, block, src), b1 = __shfl_sync(0xFFFFFFFFu, block, src + 1);
    usable_ring = (usable_ring & ~(3u << (2 * fill))) | (two << (2 * fill));
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * fill, dst = ring0 + fill * S::kStage;
      ptx::mbar_arrive_expect_tx(bar, S::kRecord * __popc(two));
      if (two & 1u) ptx::bulk_load(dst, a.data + ((int64_t)b0 * a.H + ic.h) * S::kRecord, S::kRecord, bar);
      if (two & 2u) ptx::bulk_load(dst + S::kRecord, a.data + ((int64_t)b1 * a.H + ic.h) * S::kRecord, S::kRecord, bar);
    }
    __syncwarp();
    it += kWarps;
    ++issued;
    if (++fill == S::kStages) fill = 0;
  };
  for (int s = 0; s < S::kStages; ++s) issue();

  int stage = 0;
  uint32_t phase = 0;
  Cursor k = start;
  while (k.left > 0) {
    // ---- the unit's rows
    const int row0 = k.c * S::kRows, rows = k.x.q_len * a.gamma;   // rows of the request
    const int base = k.x.n - k.x.q_len;                            // position of query 0
    uint32_t qf[S::kQueryInSmem ? 1 : S::kParts * S::kSteps][NT][2];
    float f[NT][2];          // logit factor of rows 2 t4, 2 t4 + 1 of each eight
    int pos[NT][2];          // their positions (-1: no such row)
    if constexpr (S::kQueryInSmem) __syncthreads();   // the last unit's reads are done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rho = row0 + nt * 8 + g;
      const bool real = rho < rows;
      const int i = real ? rho / a.gamma : 0, j = real ? rho - i * a.gamma : 0;
      const T* src = static_cast<const T*>(a.q) + (int64_t)(k.x.q0 + i) * a.q_stride + (int)a.qhead[k.h * a.gamma + j] * kDim;
      constexpr int kWords = S::kPart / 8;   // 32-bit words of this lane's quarter of a part
      uint32_t w[S::kParts][kWords];
      float amax = 0.f;
#pragma unroll
      for (int p = 0; p < S::kParts; ++p) {
        const uint4* v = reinterpret_cast<const uint4*>(src + p * 128 + t4 * (S::kPart / 4));
#pragma unroll
        for (int u = 0; u < kWords / 4; ++u) {
          const uint4 y = real ? v[u] : make_uint4(0, 0, 0, 0);
          w[p][4 * u] = y.x;
          w[p][4 * u + 1] = y.y;
          w[p][4 * u + 2] = y.z;
          w[p][4 * u + 3] = y.w;
        }
#pragma unroll
        for (int u = 0; u < kWords; ++u) {
          const float2 y = kv::pair_to_float2(w[p][u], static_cast<const T*>(nullptr));
          amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // 2^-e and 2^e with e the exponent of the largest element (0 for a row of zeros)
      int e = int(__float_as_uint(amax) >> 23) - 127;
      e = amax == 0.f ? 0 : max(-126, min(e, 126));
      const float down = __uint_as_float(uint32_t(127 - e) << 23), up = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
      for (int p = 0; p < S::kParts; ++p)
#pragma unroll
        for (int u = 0; u < kWords; ++u) {
          const float2 y = kv::pair_to_float2(w[p][u], static_cast<const T*>(nullptr));
          const uint32_t v = pack_f16(y.x * down, y.y * down);
          if constexpr (S::kQueryInSmem) {
            // every warp writes the same values; read back as [step][nt][lane] pairs
            reinterpret_cast<uint32_t*>(sq)[(((p * S::kSteps + u / 2) * NT + nt) * 32 + lane) * 2 + (u & 1)] = v;
          } else {
            qf[p * S::kSteps + u / 2][nt][u & 1] = v;
          }
        }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        f[nt][b] = a.scale_log2 * __shfl_sync(0xFFFFFFFFu, up, (2 * t4 + b) * 4);
        const int rr = row0 + nt * 8 + 2 * t4 + b;
        pos[nt][b] = rr < rows ? base + rr / a.gamma : -1;
      }
    }
    if constexpr (S::kQueryInSmem) __syncthreads();
    const int last_row = min(rows, row0 + S::kRows) - 1;
    const int p_min = base + row0 / a.gamma, p_max = base + last_row / a.gamma;

    float o[S::kParts * S::kSteps][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -FLT_MAX;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < S::kParts * S::kSteps; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
    }

    for (int t = k.t + warp; t < k.end; t += kWarps) {
      if (dead) {   // a copy did not come in time: no more work, only its own copies are waited for
        if (taken < issued) ptx::mbar_wait(bar0 + 8 * stage, phase, kDefaultWaitCycles);
      } else if (!ptx::mbar_wait_poll(bar0 + 8 * stage, phase, a.wait_limit, 64)) {
        dead = true;
        if (lane == 0) set_status(a.status, UPF_ERR_TIMEOUT);
        ptx::mbar_wait(bar0 + 8 * stage, phase, kDefaultWaitCycles);
      }
      dead = __any_sync(0xFFFFFFFFu, dead);
      const uint32_t two = (usable_ring >> (2 * stage)) & 3u;
      const uint8_t* const rec = ring + stage * S::kStage;
      if (!dead) {
        const int e0 = (t < k.x.sink_t ? t : t - k.x.sink_t + k.x.lo_t) * kTile;
        const bool whole = two == 3u && e0 + kTile - 1 <= p_min &&
                           (a.window == 0 || p_max - e0 < a.window || e0 + kTile <= a.sinks);
        // ---- logits: S^T[entry][row]
        float s[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint8_t* const rb = rec + b * S::kRecord;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][nt][i] = 0.f;
#pragma unroll
          for (int p = 0; p < S::kParts; ++p) {
            constexpr int kW = S::kPart / 32;   // words of a lane's quarter row: 2 or 4
            uint32_t w[2][kW], sc[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint8_t* const src = rb + p * (8 * S::kPart) + (g + 8 * half) * (S::kPart / 2) + t4 * (S::kPart / 8);
              if constexpr (kW == 4) {
                const uint4 y = *reinterpret_cast<const uint4*>(src);
                w[half][0] = y.x;
                w[half][1] = y.y;
                w[half][2] = y.z;
                w[half][3] = y.w;
                sc[half] = kv::e4m3x2_to_f16x2(
                    *reinterpret_cast<const uint16_t*>(rb + kv::k_scale(kDim, g + 8 * half, p * 8 + 2 * t4)));
              } else {
                const uint2 y = *reinterpret_cast<const uint2*>(src);
                w[half][0] = y.x;
                w[half][1] = y.y;
                sc[half] = kv::e4m3x2_to_f16x2(rb[kv::k_scale(kDim, g + 8 * half, t4)]);
              }
            }
#pragma unroll
            for (int u = 0; u < kW; ++u) {   // eight dims of the lane: two steps
              uint32_t x0[4], x1[4];
              kv::e2m1x8_to_f16(w[0][u], x0);
              kv::e2m1x8_to_f16(w[1][u], x1);
              // at d >= 128 the second half of the quarter is the second group
              const uint32_t sel = (kW == 4 && u >= 2) ? 0x3232u : 0x1010u;
              const uint32_t s0 = __byte_perm(sc[0], 0, sel), s1 = __byte_perm(sc[1], 0, sel);
#pragma unroll
              for (int st = 0; st < 2; ++st) {
                const uint32_t af[4] = {hmul2(x0[2 * st], s0), hmul2(x1[2 * st], s1), hmul2(x0[2 * st + 1], s0),
                                        hmul2(x1[2 * st + 1], s1)};
                const int step = p * S::kSteps + 2 * u + st;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if constexpr (S::kQueryInSmem) {
                    const uint2 y = reinterpret_cast<const uint2*>(sq)[(step * NT + nt) * 32 + lane];
                    const uint32_t bf[2] = {y.x, y.y};
                    mma_f16(s[b][nt], af, bf);
                  } else {
                    mma_f16(s[b][nt], af, qf[step][nt]);
                  }
                }
              }
            }
          }
        }
        // ---- weights: 2^(x - m + 12), in f16 as operand B of the second product
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][nt][i] *= f[nt][i & 1];
        if (!whole) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = e0 + 16 * b + g + 8 * (i >> 1), p = pos[nt][i & 1];
                const bool see = ((two >> b) & 1u) && e <= p && (a.window == 0 || p - e < a.window || e < a.sinks);
                if (!see) s[b][nt][i] = -INFINITY;
              }
        }
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) over |= fmaxf(s[0][nt][i], s[1][nt][i]) > m[nt][i & 1] + kLag;
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float x = fmaxf(fmaxf(s[0][nt][b], s[0][nt][b + 2]), fmaxf(s[1][nt][b], s[1][nt][b + 2]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
              const float m2 = fmaxf(m[nt][b], x), c = ptx::ex2_approx(m[nt][b] - m2);
              m[nt][b] = m2;
              l[nt][b] *= c;
#pragma unroll
              for (int mt = 0; mt < S::kParts * S::kSteps; ++mt) {
                o[mt][nt][b] *= c;
                o[mt][nt][b + 2] *= c;
              }
            }
        }
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = ptx::ex2_approx(s[b][nt][i] + (kWeightExp - m[nt][i & 1]));
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
#pragma unroll
          for (int p = 0; p < S::kParts; ++p) {
            constexpr int kW = S::kPart / 64;   // words of a chunk: 1 or 2
            uint32_t w[2][2][kW], sc[2];        // [entries 2 t4.. or 2 t4 + 8..][entry of the two]
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint8_t* const src = rb + 8 * kDim + p * (8 * S::kPart) + half * (4 * S::kPart) + lane * (8 * kW);
              if constexpr (kW == 2) {
                const uint4 y = *reinterpret_cast<const uint4*>(src);
                w[half][0][0] = y.x;
                w[half][0][1] = y.y;
                w[half][1][0] = y.z;
                w[half][1][1] = y.w;
              } else {
                const uint2 y = *reinterpret_cast<const uint2*>(src);
                w[half][0][0] = y.x;
                w[half][1][0] = y.y;
              }
              uint32_t raw = *reinterpret_cast<const uint16_t*>(rb + 17 * kDim + p * S::kPart + half * (S::kPart / 2) +
                                                                (kW == 2 ? g : g >> 1) * 8 + 2 * t4);
              if (!whole) {
                // 0 * NaN would reach the rows that do not see the entry: take the scale as 0 and
                // give the NaN to the rows that do see it below
                if ((raw & 0x7Fu) == 0x7Fu) {
                  raw &= 0xFF00u;
                  bad = 1;
                }
                if ((raw & 0x7F00u) == 0x7F00u) {
                  raw &= 0x00FFu;
                  bad = 1;
                }
              }
              sc[half] = kv::e4m3x2_to_f16x2(uint16_t(raw));
            }
#pragma unroll
            for (int u = 0; u < kW; ++u) {
              // low nibbles of both entries side by side (even dims), then the high ones
              uint32_t lo[2][4], hi[2][4];
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                kv::e2m1x8_to_f16(merge_bits(w[half][0][u], w[half][1][u] << 4, 0x0F0F0F0Fu), lo[half]);
                kv::e2m1x8_to_f16(merge_bits(w[half][0][u] >> 4, w[half][1][u], 0x0F0F0F0Fu), hi[half]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t af[4] = {hmul2(lo[0][j], sc[0]), hmul2(hi[0][j], sc[0]), hmul2(lo[1][j], sc[1]),
                                        hmul2(hi[1][j], sc[1])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(o[p * S::kSteps + 4 * u + j][nt], af, pf[b][nt]);
              }
            }
          }
        }
        if (!whole && __any_sync(0xFFFFFFFFu, bad)) {
          for (int b = 0; b < 2; ++b)
            for (int row = 0; row < 16; ++row) {
              const int e = e0 + 16 * b + row;
#pragma unroll
              for (int p = 0; p < S::kParts; ++p) {
                const int grp = p * (S::kPart / 16) + (S::kPart == 128 ? g : g >> 1);
                const bool nan = (rec[b * S::kRecord + kv::v_scale(kDim, row, grp)] & 0x7F) == 0x7F;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const int q = pos[nt][c];
                    const bool see = ((two >> b) & 1u) && e <= q && (a.window == 0 || q - e < a.window || e < a.sinks);
                    if (nan && see)
#pragma unroll
                      for (int mt = 0; mt < S::kSteps; ++mt) {
                        o[p * S::kSteps + mt][nt][c] = __int_as_float(0x7FFFFFFF);
                        o[p * S::kSteps + mt][nt][c + 2] = __int_as_float(0x7FFFFFFF);
                      }
                  }
              }
            }
        }
      }
      ++taken;
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
      __syncwarp();
      issue();
    }

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][b] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][b], d);
        if (g == 0) {
          sh_m[warp][nt * 8 + 2 * t4 + b] = m[nt][b];
          sh_l[warp][nt * 8 + 2 * t4 + b] = l[nt][b];
        }
      }
    __syncthreads();
    const bool alone = k.t == 0 && k.end == k.x.tiles;
    const bool goes_on = k.end < k.x.tiles;
    const size_t part = 2 * blockIdx.x + (goes_on ? 1 : 0);
    if (threadIdx.x == 0 && k.left == k.end - k.t) {   // the share's last unit
      Shared u;
      const long long t0 = min(first + share, total) - k.end;   // the unit's first tile
      u.c0 = goes_on ? int(t0 / share) : -1;
      u.c1 = int((t0 + k.x.tiles - 1) / share);
      u.h = k.h;
      u.row0 = row0;
      u.rows = rows;
      u.q0 = k.x.q0;
      parts.shared[blockIdx.x] = u;
    }
    float scale[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float top = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w][nt * 8 + 2 * t4 + b]);
        scale[nt][b] = ptx::ex2_approx(m[nt][b] - top);
      }
    for (int p = 0; p < S::kParts; ++p) {
      if (p) __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < S::kSteps; ++mt) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = o[mt][nt][i];
            if constexpr (S::kParts == 2)
              if (p) x[i] = o[S::kSteps + mt][nt][i];
            x[i] *= scale[nt][i & 1];
          }
          float* const dst = join + (warp * S::kRows + nt * 8 + 2 * t4) * S::kJoinRow + mt * 16 + g * 2;
          *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[2]);
          *reinterpret_cast<float2*>(dst + S::kJoinRow) = make_float2(x[1], x[3]);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < S::kRows * S::kPart / 2; i += kThreads) {
        const int row = i / (S::kPart / 2), y = i % (S::kPart / 2);   // y: dims (mt = y / 8, g = y % 8)
        const int rho = row0 + row;
        if (rho >= rows) continue;
        const int dim = p * 128 + (y % 8) * (S::kPart / 8) + 2 * (y / 8);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(join + (w * S::kRows + row) * S::kJoinRow + 2 * y);
          sum.x += v.x;
          sum.y += v.y;
        }
        float top = -FLT_MAX, all = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w][row]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += sh_l[w][row] * ptx::ex2_approx(sh_m[w][row] - top);
        if (alone) {
          const int qi = rho / a.gamma, head = a.qhead[k.h * a.gamma + rho - qi * a.gamma];
          const int64_t at = k.x.q0 + qi;
          const float inv = all == 0.f ? 0.f : a.v_mul / all;
          *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * a.out_stride + head * kDim + dim) =
              kv::float2_to_pair(sum.x * inv, sum.y * inv, static_cast<const T*>(nullptr));
          if (a.lse && p == 0 && y == 0) a.lse[at * a.Hq + head] = all == 0.f ? -INFINITY : (top - kWeightExp + log2f(all)) * kLn2;
        } else {
          *reinterpret_cast<float2*>(parts.o + (part * S::kRows + row) * kDim + dim) = sum;
          if (p == 0 && y == 0) parts.ml[part * S::kRows + row] = make_float2(top, all);
        }
      }
    }
    __syncthreads();   // the join buffer and sh_m, sh_l are free again
    next_unit(a, k, k.t, S::kRows);
  }
  while (taken < issued) {   // only after a wait that ran out
    ptx::mbar_wait(bar0 + 8 * stage, phase, kDefaultWaitCycles);
    ++taken;
    if (++stage == S::kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
}

// ------------------------------------------------------------------- join --

constexpr int kJoinThreads = 256;

// Adds up the parts of shared units.  CTA c takes its portion of the outputs of
// the unit that goes on after share c, so that the CTAs c0 .. c1 - 1 of a unit
// with many parts all work on it.  2^k lanes add up one pair of dims.
template <typename T, int kDim, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attend_join_kernel(const KvAttendArgs a, const Parts parts) {
  using S = Shape<kDim, NT>;
  pdl_wait();
  const Shared u = parts.shared[blockIdx.x];
  if (u.c0 < 0) return;
  const int rows = min(S::kRows, u.rows - u.row0), outputs = rows * (kDim / 2);
  const int workers = u.c1 - u.c0, each = (outputs + workers - 1) / workers;
  int lanes = 1;
  while (lanes < 32 && 2 * lanes * each <= kJoinThreads) lanes *= 2;
  const int sub = threadIdx.x & (lanes - 1);
  const int from = (blockIdx.x - u.c0) * each, to = min(outputs, from + each);
  // every lane makes every round: the shuffles need all of them
  for (int base = from; base < to; base += kJoinThreads / lanes) {
    const int i = base + threadIdx.x / lanes;
    const bool mine = i < to;
    const int row = mine ? i / (kDim / 2) : 0, j = mine ? i % (kDim / 2) : 0;
    float top = -FLT_MAX;
    for (int c = u.c0 + sub; c <= u.c1; c += lanes)
      top = fmaxf(top, parts.ml[(size_t)(2 * c + (c < u.c1)) * S::kRows + row].x);
    for (int d = 1; d < lanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float all = 0.f;
    float2 sum = make_float2(0.f, 0.f);
    for (int c = u.c0 + sub; c <= u.c1; c += lanes) {
      const size_t at = (size_t)(2 * c + (c < u.c1)) * S::kRows + row;
      const float2 ml = parts.ml[at], v = reinterpret_cast<const float2*>(parts.o + at * kDim)[j];
      const float w = ptx::ex2_approx(ml.x - top);
      sum.x += v.x * w;
      sum.y += v.y * w;
      all += ml.y * w;
    }
    for (int d = 1; d < lanes; d <<= 1) {
      sum.x += __shfl_xor_sync(0xFFFFFFFFu, sum.x, d);
      sum.y += __shfl_xor_sync(0xFFFFFFFFu, sum.y, d);
      all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
    }
    if (!mine || sub) continue;
    const int rho = u.row0 + row, q = rho / a.gamma, head = a.qhead[u.h * a.gamma + rho - q * a.gamma];
    const int64_t at = u.q0 + q;
    const float inv = all == 0.f ? 0.f : a.v_mul / all;
    reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at * a.out_stride + head * kDim)[j] =
        kv::float2_to_pair(sum.x * inv, sum.y * inv, static_cast<const T*>(nullptr));
    if (a.lse && j == 0) a.lse[at * a.Hq + head] = all == 0.f ? -INFINITY : (top - kWeightExp + log2f(all)) * kLn2;
  }
}

template <typename T, int kDim, int NT>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t s) {
  using S = Shape<kDim, NT>;
  Parts parts;
  parts.o = static_cast<float*>(a.ws);
  parts.ml = reinterpret_cast<float2*>(parts.o + (size_t)2 * S::kCtas * S::kRows * kDim);
  parts.shared = reinterpret_cast<Shared*>(parts.ml + (size_t)2 * S::kCtas * S::kRows);
  cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<T, kDim, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kv_attend_kernel<T, kDim, NT>, S::kCtas, kThreads, S::kSmem, s, false, a, parts);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv_attend_join_kernel<T, kDim, NT>, S::kCtas, kJoinThreads, 0, s, true, a, parts);
}

template <int kDim>
cudaError_t launch_dim(const KvAttendArgs& a, bool f16, cudaStream_t s) {
  if (a.gamma * a.max_q <= 8) return f16 ? launch<__half, kDim, 1>(a, s) : launch<__nv_bfloat16, kDim, 1>(a, s);
  return f16 ? launch<__half, kDim, 2>(a, s) : launch<__nv_bfloat16, kDim, 2>(a, s);
}

template <int kDim, int NT>
constexpr size_t ws_bytes() {
  using S = Shape<kDim, NT>;
  return (size_t)2 * S::kCtas * S::kRows * (kDim * sizeof(float) + sizeof(float2)) + S::kCtas * sizeof(Shared);
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
