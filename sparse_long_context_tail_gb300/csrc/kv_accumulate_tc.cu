// Attention weight that cache entries have drawn, for more than eight rows a kv head: prompts' last queries, drafted
// tokens, wide groups of q heads.
//
// Per 128 entries and kv head the logits are one tcgen05 product, S = K Q^T: the keys are operand A, the rows operand B,
// an entry is a TMEM lane, so that an entry's sum over the rows is a thread's sum along its lane.  Codes times
// scales go to TMEM straight from the registers that worked them out (tcgen05.st), as f16; from shared memory both
// operands of an M128 N128 product would take more of its bandwidth than there is.  The rows
// are made ready once by a launch of their own, in the swizzled layout that the product reads, and copied in bulk.
//
// A CTA (one an SM) has a run of 128-entry blocks of one request after another.  For each head and chunk of rows it goes
// through its blocks, so that rows are copied once a run; the entries' sums wait in shared memory.  Warps: two teams of
// four work out keys, two teams of four add up weights (every other product each), one issues
// the products, one the copies.  Tensor memory has a slot of keys a team (d = 128) and three of sums.
//
// What bounds it: with n rows a kv head every entry and head costs 2 d n flop, n exponentials and one pass over
// its codes.  A product of 128 rows at d = 128 takes 1090 cycles; its exponentials alone would take 512 (32 a clock and SM),
// the product about 560, the conversion of its keys 250 to 500.  With any one of these left out in a trial the time
// fell by 2 to 6 %: what is left is the hand-over between the roles.  32 queries of 4 q heads a kv head over
// 131072 entries of 8 heads: 43 us (800 TFLOP/s, 3.1 exponentials a ps), 128 queries 131 us.  Measured beside 42 and 128:
// both teams at one product, a half of its columns each: 53 and 171 us; three sum teams 46 and 140; two slots of
// sums and four of keys 48 and 150.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "kv_accumulate.cuh"
#include "sm100_ptx.cuh"

namespace upf {

namespace {

using namespace acc;

constexpr int kBlock = 128;                    // entries of a product
constexpr int kRows = 128;                     // most rows of a product
constexpr int kRowWarps = 32;                  // of a CTA that makes them ready
constexpr int kRun = 16;                       // blocks whose sums are in shared memory at once
constexpr int kKeyWarps = 8, kSumWarps = 8, kMmaWarp = 16, kTcWarps = 18 /* the last one copies */, kTcThreads = 32 * kTcWarps;
constexpr uint32_t kSlots = 2;                 // of rows

// The rows of all requests as operand B.  Those of request r and kv head h, padded to a multiple of 16, begin at row
// first_row(r) + h * padded; of d dims every 64 are a slab of their own, 128 bytes a row.
__host__ __device__ constexpr int pad16(int rows) { return (rows + 15) / 16 * 16; }
__device__ __forceinline__ int64_t first_row(const KvAccumulateArgs& a, int q0, int r) {
  return (int64_t)a.H * 16 * (((int64_t)a.gamma * q0) / 16 + r);
}
struct RowsMem {
  uint8_t* q;        // [rows][d] f16: per request and head [slab][row][64 dims], 16-byte pieces swizzled
  float* f;          // [rows] logit factors; with a minus: the row's weights are held at 1
  float* lse;        // [rows] -lse * log2 e
  int32_t* i;        // [rows] queries; -1: none
  int64_t rows;
};
__host__ __device__ inline RowsMem rows_mem(void* ws, int H, int gamma, int num_q, int R, int d) {
  RowsMem m;
  m.rows = (int64_t)H * 16 * ((int64_t)gamma * num_q / 16 + R + 1);
  m.q = static_cast<uint8_t*>(ws);
  m.f = reinterpret_cast<float*>(m.q + m.rows * d * 2);
  m.lse = m.f + m.rows;
  m.i = reinterpret_cast<int32_t*>(m.lse + m.rows);
  return m;
}

// A CTA per chunk of rows of a request and kv head, the padding's among them.
//
// Rows are divided by a power of two so that f16 holds them: one of the whole chunk, which makes its largest element
// 2^14 to 2^15, so that a logit factor is the same for all columns (32 queries of 131072 entries: 57 us with a factor
// a column, 53 with one).  f16 ends at 2^-24, so the rounding of a row 2^14 smaller, whose
// largest element is 1 to 2, is 2^-25 of that at most, as it is where each row has its own power.
// Rows further apart do have their own.
template <typename T, int kDim>
__global__ void __launch_bounds__(32 * kRowWarps) kv_accumulate_rows_kernel(const KvAccumulateArgs a, const RowsMem m) {
  constexpr const T* kT = nullptr;
  constexpr int kEach = kDim / 32;             // dims of a lane
  constexpr int kTop = 14;                     // exponent of the largest element
  constexpr int kOwn = kRows / kRowWarps;      // rows of a warp
  __shared__ int most, least;                  // of the exponents of the rows that count
  __shared__ int back;                         // do they begin before those of an earlier request end
  pdl_wait();
  pdl_trigger();         // only now: the second launch reads and writes what launches before this one do
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int looked = 0, top = 0;     // requests looked at, and where the rows of this thread's among them end
  for (int r = blockIdx.y; r < a.R; r += gridDim.y) {
    for (int j = looked + threadIdx.x; a.cu_q && j < r; j += 32 * kRowWarps) {
      Request y;
      top = end_of(y, look_at(a, j, y), top);
    }
    looked = r;
    const Request x = load_request<false>(a, r, top);
    const int rows = x.q_len * a.gamma, padded = pad16(rows), chunks = (padded + kRows - 1) / kRows;
    for (int hc = blockIdx.x; hc < a.H * chunks; hc += gridDim.x) {
      const int h = hc / chunks, row0 = (hc - h * chunks) * kRows, row1 = min(padded, row0 + kRows);
      const int64_t region = first_row(a, x.q0, r) + (int64_t)h * padded;
      // the warp's rows, all on their way before the first is looked at
      uint32_t q[kOwn][kEach / 2];
      float lse[kOwn];
      int query[kOwn];
#pragma unroll
      for (int y = 0; y < kOwn; ++y) {
        const int rho = row0 + warp + y * kRowWarps;
        const bool real = rho < rows;
        query[y] = real ? rho / a.gamma : -1;
        const int i = max(query[y], 0), head = a.qhead[h * a.gamma + (real ? rho - i * a.gamma : 0)];
        const int64_t at = x.q0 + i;
        lse[y] = real ? a.lse[at * a.Hq + head] : -INFINITY;
#pragma unroll
        for (int k = 0; k < kEach / 2; ++k)
          q[y][k] = real ? reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + at * a.q_stride + head * kDim)[lane * (kEach / 2) + k] : 0u;
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        most = INT_MIN;
        least = INT_MAX;
        back = 0;
      }
      __syncthreads();
      RowConstants c[kOwn];
      int hi = INT_MIN, lo = INT_MAX;
#pragma unroll
      for (int y = 0; y < kOwn; ++y) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kEach / 2; ++k) top = kv::max_abs2(top, q[y][k], kT);
        const float2 tops = kv::pair_to_float2(top, kT);
        const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, max(__float_as_uint(fabsf(tops.x)), __float_as_uint(fabsf(tops.y))));
        c[y] = row_constants(a, query[y] >= 0, amax, lse[y]);
        if (c[y].bad && lane == 0) set_status(a.status, UPF_ERR_NONFINITE);
        if (!c[y].on || c[y].zero) continue;
        hi = max(hi, c[y].e);
        lo = min(lo, c[y].e);
      }
      if (top > x.q0) back = 1;
      if (lane == 0 && hi >= lo) {
        atomicMax(&most, hi);
        atomicMin(&least, lo);
      }
      __syncthreads();
      if (back) continue;      // their places are another's
      const bool same = most < least || most - least <= kTop;     // none, or near one another
#pragma unroll
      for (int y = 0; y < kOwn; ++y) {
        const int rho = row0 + warp + y * kRowWarps;
        if (rho >= row1) break;
        const int e = (same ? (most < least ? 0 : most) : c[y].e) - kTop;
        // 2^-e in two factors: it may be past fp32
        const float down0 = __uint_as_float(uint32_t(127 - e / 2) << 23), down1 = __uint_as_float(uint32_t(127 - (e - e / 2)) << 23);
        uint32_t v[kEach / 2];
#pragma unroll
        for (int k = 0; k < kEach / 2; ++k) {
          const float2 z = kv::pair_to_float2(q[y][k], kT);
          v[k] = c[y].on ? pack_f16(z.x * down0 * down1, z.y * down0 * down1) : 0u;
        }
        // dims lane * kEach ..: slab, and the byte within the row's 128
        const int dim = lane * kEach, slab = dim / 64, byte = dim % 64 * 2;
        uint8_t* const dst = m.q + (region * kDim + ((int64_t)slab * padded + rho) * 64) * 2 + ((byte >> 4 ^ (rho & 7)) << 4) + (byte & 15);
        if constexpr (kEach == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
        else if constexpr (kEach == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(v[0], v[1]);
        else *reinterpret_cast<uint32_t*>(dst) = v[0];
        if (lane == 0) {
          const float f = factor_of(a, a.scale_exp + e);
          m.f[region + rho] = c[y].on && is_far(c[y].hi) ? -f : f;
          m.lse[region + rho] = c[y].on ? -(c[y].hi + c[y].low) : -INFINITY;      // a row that does not count has the weight 0
          m.i[region + rho] = query[y];      // one that does not count sees NaNs, too
        }
      }
    }
  }
}

template <int kDim>
struct TcShape {
  static constexpr int kSlabs = kDim / 64;
  static constexpr int kKeyCols = kDim / 2;                    // TMEM columns of a block's keys
  static constexpr int kRowBytes = kRows * kDim * 2;           // of a chunk of rows
  static constexpr int kConstBytes = kRows * 12;
  // Four slots of keys where tensor memory has room: a group works out its next block while the products with the last
  // are under way.
  static constexpr uint32_t kKeySlots = kDim == 64 ? 4 : 2, kSumSlots = kDim == 256 ? 2 : 3;
  static constexpr int kSumCol = kKeySlots * kKeyCols;         // first TMEM column of the sums
  static_assert(kSumCol + kSumSlots * kRows <= 512, "tensor memory");
  // a key warp's ring: of two tiles the codes, then the scales; 16-byte pieces
  static constexpr int kRowPieces = Shape<kDim>::kPart / 32;
  static constexpr int kRingItem = 2 * 9 * kDim, kAhead = kDim == 64 ? 6 : kDim == 128 ? 4 : 2, kRingBytes = kAhead * kRingItem;
  // rows side by side begin at the same bank every 128 bytes: a row's pieces are swapped by that
  __host__ __device__ static constexpr int swap(int row) { return row / (4 / (kRowPieces / 2)) % kRowPieces; }
  // rows (1024-byte aligned), their constants, the entries' sums (a column half each), the rings
  static constexpr int kConstAt = kSlots * kRowBytes, kSumAt = kConstAt + kSlots * kConstBytes;
  static constexpr int kRingAt = kSumAt + 2 * kRun * kBlock * 4;
  static constexpr int kSmem = kRingAt + kKeyWarps * kRingBytes + 1024;
  static_assert(kSmem <= 224 * 1024, "shared memory");
};

__device__ __forceinline__ void copy_async16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 8 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// D[tmem] = A[tmem] * B[smem]^T, f16 inputs, fp32 accumulation; kAdd: += .
template <bool kAdd>
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}
// As ptx::idesc_bf16_f32 with f16 operands.
__device__ __forceinline__ uint32_t idesc_f16(uint32_t n) { return (1u << 4) | (n >> 3 << 17) | (kBlock >> 4 << 24); }

// A request's blocks that some row sees: [0, sink_b) and [lo_b, ..).
struct Blocks {
  int sink_b, lo_b, count;
  __device__ __forceinline__ int entry(int b) const { return (b < sink_b ? b : b - sink_b + lo_b) * kBlock; }
};
__device__ __forceinline__ Blocks blocks_of(const KvAccumulateArgs& a, const Request& x) {
  const View v = view_of(a, x);
  Blocks b;
  b.lo_b = v.w0 / kBlock;
  b.sink_b = min((v.sinks + kBlock - 1) / kBlock, b.lo_b);
  b.count = x.q_len ? b.sink_b + (x.n + kBlock - 1) / kBlock - b.lo_b : 0;
  return b;
}

template <int kDim>
__global__ void __launch_bounds__(kTcThreads, 1) kv_accumulate_tc_kernel(const KvAccumulateArgs a, const RowsMem m) {
  using S = Shape<kDim>;
  using C = TcShape<kDim>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (1024 - (ptx::smem_u32(smem_raw) & 1023)) % 1024;
  float* const sums = reinterpret_cast<float*>(smem + C::kSumAt);      // [2][kRun * kBlock]
  __shared__ Starts<kTcThreads> starts;
  __shared__ __align__(8) uint64_t bars[2 * C::kKeySlots + 2 * kSlots + 2 * C::kSumSlots];
  __shared__ uint32_t tmem_word;
  __shared__ int failed;
  __shared__ uint32_t row_copies, products;      // begun so far
  __shared__ unsigned long long records[kRun][kBlock / 16];     // bit 0: there is none, and the cache's first stands in
  // from a shuffle, so that what depends on the warp alone is known to be the same in all lanes
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto keys_full = [&](uint32_t s) { return bar0 + 8 * s; };
  auto keys_free = [&](uint32_t s) { return bar0 + 8 * (C::kKeySlots + s); };
  const uint32_t bar1 = bar0 + 16 * C::kKeySlots;
  auto rows_full = [&](uint32_t s) { return bar1 + 8 * s; };
  auto rows_free = [&](uint32_t s) { return bar1 + 8 * (kSlots + s); };
  auto sums_full = [&](uint32_t s) { return bar1 + 8 * (2 * kSlots + s); };
  auto sums_free = [&](uint32_t s) { return bar1 + 8 * (2 * kSlots + C::kSumSlots + s); };
  if (tid == 0) {
    for (uint32_t s = 0; s < C::kKeySlots; ++s) {
      ptx::mbar_init(keys_full(s), 4);
      ptx::mbar_init(keys_free(s), 1);
    }
    for (uint32_t s = 0; s < kSlots; ++s) {
      ptx::mbar_init(rows_full(s), 1);
      ptx::mbar_init(rows_free(s), 1 + kSumWarps);
    }
    for (uint32_t s = 0; s < C::kSumSlots; ++s) {
      ptx::mbar_init(sums_full(s), 1);
      ptx::mbar_init(sums_free(s), kSumWarps / 2);
    }
    failed = 0;
    row_copies = products = 0;
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_word), 512);
    ptx::tmem_relinquish();
  }
  ptx::fence_barrier_init();
  int* const tops = reinterpret_cast<int*>(smem + C::kRingAt);      // the rings come later
  const Deal deal = deal_out<kTcThreads, true>(a, starts, tops, [&](const Request& x) { return blocks_of(a, x).count; });   // barriers inside
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_word;
  fade_unseen<kTcThreads, true>(a, [&](const Request& x, int& from, int& to) {
    const Blocks b = blocks_of(a, x);
    from = b.sink_b * kBlock;
    to = b.lo_b * kBlock;
  });
  const long long share = (deal.total + gridDim.x - 1) / gridDim.x;
  long long u = blockIdx.x * share;
  const long long end = min(u + share, deal.total);
  // phases of the rings, each role its own
  uint32_t key_n = 0, row_n = 0, sum_n = 0;      // blocks, chunks, products so far
  auto wait = [&](uint32_t bar, uint32_t phase) {
    if (ptx::mbar_try_wait(bar, phase)) return true;
    const long long t0 = clock64();
    while (!ptx::mbar_try_wait_hint(bar, phase, 200)) {
      if (*reinterpret_cast<volatile int*>(&failed)) return false;
      if (clock64() - t0 > a.wait_limit) {
        *reinterpret_cast<volatile int*>(&failed) = 1;
        set_status(a.status, UPF_ERR_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  bool rows_waited = false;
  int r = 0;
  Request x{};
  long long first = 0;
  int top = 0;
  if (u < end && !find_request<kTcThreads, true>(a, starts, tops, deal, u, r, x, first, top, [&](const Request& y) { return blocks_of(a, y).count; })) u = end;
  while (u < end) {
    const Blocks blocks = blocks_of(a, x);
    const View view = view_of(a, x);
    const int begin = int(u - first), stop = int(min(end - first, (long long)blocks.count));
    const int rows = x.q_len * a.gamma, padded = pad16(rows), chunks = (padded + kRows - 1) / kRows;
    const int64_t region = first_row(a, x.q0, r);
    for (int run0 = begin; run0 < stop; run0 += kRun) {
      const int run = min(kRun, stop - run0);
      for (int i = tid; i < run * (kBlock / 16); i += kTcThreads) {
        const uint8_t* const rec = record_at<kDim>(a, r, x, view, blocks.entry(run0 + i / (kBlock / 16)) + i % (kBlock / 16) * 16);
        records[i / (kBlock / 16)][i % (kBlock / 16)] = reinterpret_cast<unsigned long long>(rec ? rec : a.data) | !rec;
      }
      for (int i = tid; i < 2 * kRun * kBlock; i += kTcThreads) sums[i] = 0.f;
      __syncthreads();
      if (warp < kKeyWarps) {
        // ---- keys: this warp's 32 entries of every other block, an entry a lane
        const int quarter = warp & 3;
        const uint32_t team = warp >> 2;
        uint8_t* const ring = smem + C::kRingAt + warp * C::kRingBytes;
        const int total = a.H * chunks * run;        // products of the run; the i-th is of block i % run
        // the group's products: those whose number from the kernel's start is its team's modulo two
        const int i0 = int((team - key_n) & 1);
        struct At {
          int i, b, c, h;      // product; its block, chunk of rows and head
        };
        auto next = [&](At& x) {
          x.i += 2;
          x.b += 2;
          while (x.b >= run) {
            x.b -= run;
            if (++x.c == chunks) {
              x.c = 0;
              ++x.h;
            }
          }
        };
        // ---- copies of the warp's two tiles' codes and scales, kAhead products before they are worked out.  A lane's
        // pieces lie side by side in the cache; in the ring those of a row are swapped so that lanes
        // that read one piece of 32 rows meet all banks.
        // a run of 512 bytes has the pieces of whole rows, and rows in the same place of it are swapped alike
        static_assert(C::swap(512 / (S::kPart / 2)) == 0, "swaps repeat");
        const uint32_t codes_to = ptx::smem_u32(ring) + (lane / C::kRowPieces * C::kRowPieces + (lane % C::kRowPieces ^ C::swap(lane / C::kRowPieces))) * 16;
        const uint32_t scales_to = ptx::smem_u32(ring) + 16 * kDim + lane * 16;
        At to{i0 - 2, i0 - 2, 0, 0};
        next(to);
        int to_slot = 0;
        auto copy = [&] {
          if (to.i < total) {
            const uint32_t dst = codes_to + to_slot * C::kRingItem;
            const int64_t from = to.h * S::kRecord + lane * 16;
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
              const uint8_t* const src = reinterpret_cast<const uint8_t*>(records[to.b][quarter * 2 + tile] & ~1ull) + from;
#pragma unroll
              for (int k = 0; k < 8 * kDim; k += 512) copy_async16(dst + tile * 8 * kDim + k, src + k);
              if (lane < kDim / 16) copy_async16(scales_to + to_slot * C::kRingItem + tile * kDim, src + 16 * kDim);
            }
            if (++to_slot == C::kAhead) to_slot = 0;
            next(to);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < C::kAhead; ++k) copy();
        int from_slot = 0;
        const int row = lane & 15;
        At x{i0 - 2, i0 - 2, 0, 0};
        for (next(x); x.i < total; next(x)) {
          const uint32_t n = key_n + x.i, slot = n % C::kKeySlots;
          asm volatile("cp.async.wait_group %0;" ::"n"(C::kAhead - 1) : "memory");
          __syncwarp();
          const bool there = !(records[x.b][quarter * 2 + (lane >> 4)] & 1);
          const uint8_t* const item = ring + from_slot * C::kRingItem;
          if (++from_slot == C::kAhead) from_slot = 0;
          bool ok = true;
#pragma unroll
          for (int half = 0; half < kDim / 64; ++half) {    // 64 dims: 32 columns
            uint32_t v[32];
            const uint32_t scales = there ? *reinterpret_cast<const uint32_t*>(item + 16 * kDim + (lane >> 4) * kDim + row * (kDim / 16) + half * 4) : 0u;
            const uint32_t s01 = kv::e4m3x2_to_f16x2(uint16_t(scales)), s23 = kv::e4m3x2_to_f16x2(uint16_t(scales >> 16));
            const __half2 s[4] = {__low2half2(as_half2(s01)), __high2half2(as_half2(s01)), __low2half2(as_half2(s23)), __high2half2(as_half2(s23))};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int piece = half * 2 + k, part = piece / C::kRowPieces;
              const uint4 c = *reinterpret_cast<const uint4*>(item + (((lane >> 4) * S::kParts + part) * 16 + row) * (S::kPart / 2) +
                                                              (piece % C::kRowPieces ^ C::swap(row)) * 16);
              const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint32_t hh[4];
                kv::e2m1x8_to_f16(w[y], hh);
#pragma unroll
                for (int z = 0; z < 4; ++z) v[k * 16 + y * 4 + z] = hmul2(hh[z], s[k * 2 + y / 2]);
              }
            }
            if (half == 0) {      // the first 64 dims are worked out before the slot is free
              ok = __all_sync(0xFFFFFFFFu, wait(keys_free(slot), (n / C::kKeySlots & 1) ^ 1));   // all lanes or none
              if (!ok) break;
              ptx::tc_fence_after();
            }
            tmem_st32(tmem + (uint32_t(quarter * 32) << 16) + slot * C::kKeyCols + half * 32, v);
          }
          if (!ok) break;
          __syncwarp();      // the item may be copied over
          copy();
          tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(keys_full(slot));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      } else if (warp < kKeyWarps + kSumWarps) {
        // ---- weights: this warp's 32 entries of its team's products, every other one
        const int quarter = warp & 3, team = (warp - kKeyWarps) >> 2;
        uint32_t rn = row_n, sn = sum_n;
        bool ok = true;
        for (int hc = 0; hc < a.H * chunks && ok; ++hc, ++rn) {
          const int c = hc % chunks, cols = min(kRows, padded - c * kRows);
          const uint32_t rs = rn % kSlots;
          ok = __all_sync(0xFFFFFFFFu, wait(rows_full(rs), rn / kSlots & 1));
          const float* const cf = reinterpret_cast<const float*>(smem + C::kConstAt + rs * C::kConstBytes);
          // a broadcast from shared memory takes as long as it has words, so the factor is one where the rows allow it:
          // all have the same, and none's weights are held at 1 (its factor has a minus)
          bool same = true;
          if (ok && lane * 4 < cols) {
            const float4 f = *reinterpret_cast<const float4*>(cf + lane * 4);
            same = f.x == fabsf(cf[0]) && f.y == f.x && f.z == f.x && f.w == f.x;
          }
          same = __all_sync(0xFFFFFFFFu, same);
          const uint64_t one_f = ok ? ptx::pack2(cf[0], cf[0]) : 0;
          for (int b = int((team - sn) & 1); b < run && ok; b += 2) {
            const uint32_t n = sn + b, ss = n % C::kSumSlots;
            const int e0 = blocks.entry(run0 + b), e = e0 + quarter * 32 + lane;
            const bool whole = all_seen(a, x, view, e0, e0 + kBlock);
            // The queries that see this entry: `count` from `from` on.  (With each row's four comparisons instead 53 us for 43: the CTA
            // with the blocks that rows see in part is the last one.)
            const int from = max(0, e - view.base);
            const uint32_t count = a.window == 0 || e < a.sinks ? INT_MAX : max(0, e - view.base + a.window - from);
            if (!(ok = __all_sync(0xFFFFFFFFu, wait(sums_full(ss), n / C::kSumSlots & 1)))) break;
            ptx::tc_fence_after();
            const uint32_t at = tmem + (uint32_t(quarter * 32) << 16) + C::kSumCol + ss * kRows;
            uint64_t total = 0;      // over the even and over the odd columns
            // four logits as weights, added up
            auto add = [&](auto plain, const float* v, int j) {      // plain: one factor, none held at 1, all seen
              constexpr bool kPlain = decltype(plain)::value;
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(cf + kRows + j);
              ulonglong2 f;
              if constexpr (kPlain) f = make_ulonglong2(one_f, one_f);
              else {
                f = *reinterpret_cast<const ulonglong2*>(cf + j);
                f.x &= 0x7FFFFFFF7FFFFFFFull, f.y &= 0x7FFFFFFF7FFFFFFFull;     // without the minus
              }
              float w[4];
              ptx::unpack2(ptx::fma2(ptx::pack2(v[0], v[1]), f.x, l.x), w[0], w[1]);
              ptx::unpack2(ptx::fma2(ptx::pack2(v[2], v[3]), f.y, l.y), w[2], w[3]);
              if constexpr (!kPlain) {
                float minus[4];
                ptx::unpack2(l.x, minus[0], minus[1]);
                ptx::unpack2(l.y, minus[2], minus[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = held(w[k], minus[k]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = ptx::ex2_approx(w[k]);
              if constexpr (!kPlain) {
                const int4 i = *reinterpret_cast<const int4*>(cf + 2 * kRows + j);
                w[0] = uint32_t(i.x - from) < count ? w[0] : 0.f;
                w[1] = uint32_t(i.y - from) < count ? w[1] : 0.f;
                w[2] = uint32_t(i.z - from) < count ? w[2] : 0.f;
                w[3] = uint32_t(i.w - from) < count ? w[3] : 0.f;
              }
              total = ptx::add2(total, ptx::add2(ptx::pack2(w[0], w[1]), ptx::pack2(w[2], w[3])));
            };
            const bool plain = whole && same;
            int j = 0;
            if (plain && cols == kRows) {      // 32 columns are on their way while others are added up
              float v0[32], v1[32];
              ptx::tmem_ld32(at, v0);
              ptx::tmem_wait_ld();
#pragma unroll
              for (j = 0; j < kRows; j += 64) {
                ptx::tmem_ld32(at + j + 32, v1);
#pragma unroll
                for (int k = 0; k < 32; k += 4) add(std::true_type(), v0 + k, j + k);
                ptx::tmem_wait_ld();
                if (j + 64 < kRows) ptx::tmem_ld32(at + j + 64, v0);
#pragma unroll
                for (int k = 0; k < 32; k += 4) add(std::true_type(), v1 + k, j + 32 + k);
                ptx::tmem_wait_ld();
              }
            }
            if (plain)
              for (; j < cols; j += 16) {
                float v[16];
                ptx::tmem_ld16(at + j, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k += 4) add(std::true_type(), v + k, j + k);
              }
            for (; j < cols; j += 8) {
              float v[8];
              tmem_ld8(at + j, v);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; k += 4) add(std::false_type(), v + k, j + k);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sums_free(ss));
            float even, odd;
            ptx::unpack2(total, even, odd);
            sums[team * kRun * kBlock + b * kBlock + quarter * 32 + lane] += even + odd;
          }
          sn += run;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(rows_free(rs));
        }
      } else if (warp == kMmaWarp) {
        // the whole warp runs the loops, so that what the products take is known to be the same in all lanes
        uint32_t kn = key_n, rn = row_n, sn = sum_n;
        bool ok = true;
        for (int hc = 0, c = 0; hc < a.H * chunks && ok; ++hc, ++rn) {
          const int cols = min(kRows, padded - c * kRows);
          if (++c == chunks) c = 0;
          const uint32_t rs = rn % kSlots, idesc = idesc_f16(cols);
          if (!(ok = __all_sync(0xFFFFFFFFu, wait(rows_full(rs), rn / kSlots & 1)))) break;
          uint64_t rows_at[C::kSlabs];         // a step of 16 dims is two further on (of 16 bytes)
#pragma unroll
          for (int s = 0; s < C::kSlabs; ++s) rows_at[s] = ptx::sdesc_kmajor_sw128(ptx::smem_u32(smem + rs * C::kRowBytes) + s * cols * 128);
          for (int b = 0; b < run; ++b, ++kn, ++sn) {
            const uint32_t ks = kn % C::kKeySlots, ss = sn % C::kSumSlots;
            if (!(ok = __all_sync(0xFFFFFFFFu, wait(sums_free(ss), (sn / C::kSumSlots & 1) ^ 1) && wait(keys_full(ks), kn / C::kKeySlots & 1)))) break;
            ptx::tc_fence_after();
            const uint32_t to = tmem + C::kSumCol + ss * kRows, keys = tmem + ks * C::kKeyCols;
            if (ptx::elect_one()) {
              mma_f16_ts<false>(to, keys, rows_at[0], idesc);
#pragma unroll
              for (int k = 1; k < kDim / 16; ++k) mma_f16_ts<true>(to, keys + k * 8, rows_at[k / 4] + k % 4 * 2, idesc);
              ptx::mma_commit(keys_free(ks));
              ptx::mma_commit(sums_full(ss));
              if (b == run - 1) ptx::mma_commit(rows_free(rs));
            }
            __syncwarp();
          }
        }
        if (lane == 0) products = sn;
        __syncwarp();
      } else {
        // ---- copies of the rows and their constants
        if (lane == 0) {
          if (!rows_waited) pdl_wait();
          rows_waited = true;
          for (int hc = 0; hc < a.H * chunks; ++hc) {
            const uint32_t n = row_n + hc, rs = n % kSlots;
            const int h = hc / chunks, c = hc - h * chunks, cols = min(kRows, padded - c * kRows);
            if (!wait(rows_free(rs), (n / kSlots & 1) ^ 1)) break;
            const int64_t row0 = region + (int64_t)h * padded;
            ptx::mbar_arrive_expect_tx(rows_full(rs), cols * (kDim * 2 + 12));
            for (int s = 0; s < C::kSlabs; ++s)
              ptx::bulk_load(ptx::smem_u32(smem + rs * C::kRowBytes) + s * cols * 128,
                             m.q + (row0 * kDim + ((int64_t)s * padded + c * kRows) * 64) * 2, cols * 128, rows_full(rs));
            const uint32_t dst = ptx::smem_u32(smem + C::kConstAt + rs * C::kConstBytes);
            const int64_t at = row0 + c * kRows;
            ptx::bulk_load(dst, m.f + at, cols * 4, rows_full(rs));
            ptx::bulk_load(dst + kRows * 4, m.lse + at, cols * 4, rows_full(rs));
            ptx::bulk_load(dst + kRows * 8, m.i + at, cols * 4, rows_full(rs));
            row_copies = n + 1;
          }
        }
        __syncwarp();
      }
      key_n += a.H * chunks * run;
      sum_n += a.H * chunks * run;
      row_n += a.H * chunks;
      __syncthreads();
      if (failed) break;
      for (int i = tid; i < run * kBlock; i += kTcThreads) {
        const int e = blocks.entry(run0 + i / kBlock) + i % kBlock;
        if (e >= x.n) continue;
        const float v = records[i / kBlock][i % kBlock / 16] & 1 ? 0.f : sums[i] + sums[kRun * kBlock + i];
        const int64_t at = r * a.w_stride + e;
        a.w_out[at] = a.w_in ? __fmaf_rn(a.decay, a.w_in[at], v) : v;
      }
      __syncthreads();      // records and sums are the next run's
    }
    if (failed) break;
    u = first + stop;
    first += blocks.count;
    for (++r; u < end && r < a.R; ++r) {
      x = load_request<true>(a, r, top);
      const int count = blocks_of(a, x).count;
      if (u < first + count) break;
      first += count;
    }
    if (r >= a.R) break;
  }
  // the workspace is the caller's again only when the rows' launch is over, whether or not this CTA had any work
  if (tid == 32 * (kTcWarps - 1) && !rows_waited) pdl_wait();
  __syncthreads();
  // a wait that ran out leaves copies and products on their way: they are waited for as long as waits may take by default
  if (failed && tid == 0)
    for (uint32_t k = 1; k <= C::kSumSlots; ++k) {
      if (k <= kSlots && row_copies >= k) ptx::mbar_wait(rows_full((row_copies - k) % kSlots), (row_copies - k) / kSlots & 1, kDefaultWaitCycles);
      if (products >= k) ptx::mbar_wait(sums_full((products - k) % C::kSumSlots), (products - k) / C::kSumSlots & 1, kDefaultWaitCycles);
    }
  __syncthreads();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

template <typename T, int kDim>
cudaError_t launch(const KvAccumulateArgs& a, cudaStream_t s) {
  const RowsMem m = rows_mem(a.ws, a.H, a.gamma, a.num_q, a.R, kDim);
  // once per device and process: this launches nothing
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (a.device & 63);
  cudaError_t e;
  if (a.device > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kv_accumulate_tc_kernel<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<kDim>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int per = int(std::min<int64_t>((int64_t)a.H * ((pad16(a.gamma * a.max_q) + kRows - 1) / kRows), 4 * kPlanSMs));
  e = launch_kernel(kv_accumulate_rows_kernel<T, kDim>, dim3(per, std::min(a.R, std::max(1, 2 * kPlanSMs / per))), 32 * kRowWarps, 0, s, true, a, m);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)a.R * ((((int64_t)a.max_pages << a.page_shift) + kBlock - 1) / kBlock);
  return launch_kernel(kv_accumulate_tc_kernel<kDim>, dim3(unsigned(std::min<long long>(kPlanSMs, blocks))), kTcThreads, TcShape<kDim>::kSmem, s, true, a, m);
}

}  // namespace

size_t kv_accumulate_tc_workspace_bytes(int H, int gamma, int num_q, int R, int d) {
  return size_t(rows_mem(nullptr, H, gamma, num_q, R, d).rows) * (2 * d + 12);
}

cudaError_t launch_kv_accumulate_tc(const KvAccumulateArgs& a, bool f16, cudaStream_t s) {
  if (f16) return a.d == 64 ? launch<__half, 64>(a, s) : a.d == 128 ? launch<__half, 128>(a, s) : launch<__half, 256>(a, s);
  return a.d == 64 ? launch<__nv_bfloat16, 64>(a, s) : a.d == 128 ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 256>(a, s);
}

}  // namespace upf
