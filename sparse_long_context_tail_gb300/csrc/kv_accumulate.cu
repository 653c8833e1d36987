// Attention weight that cache entries have drawn.
//
// For entry e of request r: w_out = decay w_in + sum over the rows (query i, q head h) that see e of
// exp(scale q.k_e - lse), with lse the row's from the attention.  Rows whose lse is -inf saw nothing.
//
// Only the keys' half of the records is read, and each entry's sum is added up in one order, so results repeat.  This file
// has the kernel for at most eight rows a kv head (decoding); more rows take kv_accumulate_tc.cu.
//
// What it takes: about 160 instructions per 16 entries and head of d = 128, 32 of them conversions, 32 scalings and 8
// products, at 2.3 to 2.7 a clock and SM.  Neither the issue slots, a third of which are idle, nor HBM, which would allow 40 % more,
// are at their limit: a tile's wait, products, exponentials and sums are one chain.  One new token of 16 requests of 4096 to
// 131072 entries (8 heads, d = 128, 32 q heads): 60 us, 4.4 TB/s; one of 131072: 22.7 us; of 4096 (d = 64): 6.0 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv_accumulate.cuh"

namespace upf {

namespace {

using namespace acc;

// One CTA an SM.  The tiles (16 entries) that some row sees, of all requests in order, are dealt out to the CTAs in equal runs.
// Of each request in its run a CTA goes through the tiles in blocks, up to 24 kv heads at a time.  A warp has one head, whose rows
// (operand B of mma.sync) and constants stay in its registers, and every 24 / heads-th tile; entries on M, codes times scales
// as operand A straight from registers.  It leaves the tile's sums in shared memory, and after the
// block they are added up over the heads.  (With whole tiles to a warp, all heads of them, the last
// warps of an SM worked alone for a quarter of the time: a tile takes one warp of 24 about 6 us.)
// (With 32 warps 16 ragged requests took 58.7 us for 59.4, and 4096 entries 7.4 for 6.0.)
constexpr int kWarps = 24, kThreads = 32 * kWarps;
constexpr int kSumTiles = 384;          // tiles times heads of a block
constexpr int kBlockTiles = 192;        // most tiles of a block

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

__device__ __forceinline__ void copy_async16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// A lane's quarters of rows g and g + 8 of a record's keys.
template <int kDim>
struct Keys {
  uint32_t w[2][Shape<kDim>::kWords];
  uint16_t s[2][Shape<kDim>::kParts];    // scales of the quarter's one or two groups
};

// From the lane's first codes and scales in shared memory.
template <int kDim>
__device__ __forceinline__ void read_keys(Keys<kDim>& k, const uint8_t* codes, const uint8_t* scales) {
  using S = Shape<kDim>;
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int p = 0; p < S::kParts; ++p) {
      const uint8_t* const c = codes + p * (8 * S::kPart) + y * (4 * S::kPart);
      const uint8_t* const s = scales + p * 8 + y * (kDim / 2);
      if constexpr (S::kPart == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(c);
        k.w[y][4 * p] = x.x;
        k.w[y][4 * p + 1] = x.y;
        k.w[y][4 * p + 2] = x.z;
        k.w[y][4 * p + 3] = x.w;
        k.s[y][p] = *reinterpret_cast<const uint16_t*>(s);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(c);
        k.w[y][0] = x.x;
        k.w[y][1] = x.y;
        k.s[y][0] = *s;
      }
    }
}

// s[entry g, g + 8][rows 2 t4, 2 t4 + 1] += keys . rows, over eight dims of the lane (from zero at the first)
template <int kDim>
__device__ __forceinline__ void products(float (&s)[4], const Keys<kDim>& k, int w, const uint4& q) {
  using S = Shape<kDim>;
  const int p = w / S::kPartWords;
  uint32_t x0[4], x1[4];
  kv::e2m1x8_to_f16(k.w[0][w], x0);
  kv::e2m1x8_to_f16(k.w[1][w], x1);
  const __half2 h0 = as_half2(kv::e4m3x2_to_f16x2(k.s[0][p])), h1 = as_half2(kv::e4m3x2_to_f16x2(k.s[1][p]));
  const bool second = S::kPart == 128 && w % S::kPartWords >= 2;
  const __half2 s0 = second ? __high2half2(h0) : __low2half2(h0), s1 = second ? __high2half2(h1) : __low2half2(h1);
  const uint32_t a0[4] = {hmul2(x0[0], s0), hmul2(x1[0], s1), hmul2(x0[1], s0), hmul2(x1[1], s1)};
  const uint32_t a1[4] = {hmul2(x0[2], s0), hmul2(x1[2], s1), hmul2(x0[3], s0), hmul2(x1[3], s1)};
  const uint32_t b0[2] = {q.x, q.y}, b1[2] = {q.z, q.w};
  if (w == 0) mma_f16_zero(s, a0, b0);
  else mma_f16(s, a0, b0);
  mma_f16(s, a1, b1);
}

// Eight rows of a kv head as operand B, and what turns their products into weights (of rows 2 t4, 2 t4 + 1).
template <int kDim>
struct Rows {
  uint4 q[Shape<kDim>::kWords];      // of two steps each
  float f[2], lse[2], lift[2];       // lse with a minus
  int i[2];                          // queries; -1: no such row
  bool far;                          // some row's weights are held at 1 (the same in all lanes)
};

// By a warp; lane (g, t4) has the t4-th quarters of row g's parts.
template <typename T, int kDim>
__device__ __forceinline__ void load_rows(const KvAccumulateArgs& a, Rows<kDim>& out, const Request& r, int h) {
  using S = Shape<kDim>;
  constexpr const T* kT = nullptr;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const bool real = g < r.q_len * a.gamma;
  const int i = real ? g / a.gamma : 0, head = a.qhead[h * a.gamma + (real ? g - i * a.gamma : 0)];
  const int64_t at = r.q0 + i;
  const T* const src = static_cast<const T*>(a.q) + at * a.q_stride + head * kDim;
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < S::kParts; ++p)
#pragma unroll
    for (int v = 0; v < S::kPartWords; ++v) {
      const uint4 y = real ? __ldg(reinterpret_cast<const uint4*>(src + p * 128 + t4 * (S::kPart / 4)) + v) : make_uint4(0, 0, 0, 0);
      out.q[p * S::kPartWords + v] = y;
      top = kv::max_abs2(kv::max_abs2(top, kv::max_abs2(y.x, y.y, kT), kT), kv::max_abs2(y.z, y.w, kT), kT);
    }
  const float lse = real ? __ldg(a.lse + at * a.Hq + head) : -INFINITY;
  const float2 tops = kv::pair_to_float2(top, kT);
  uint32_t amax = max(__float_as_uint(fabsf(tops.x)), __float_as_uint(fabsf(tops.y)));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  const RowConstants c = row_constants(a, real, amax, lse);
  if (c.bad && t4 == 0) set_status(a.status, UPF_ERR_NONFINITE);
  auto half = [&](uint32_t w) {
    const float2 y = kv::pair_to_float2(w, kT);
    return c.on ? pack_f16(y.x * c.down, y.y * c.down) : 0u;
  };
#pragma unroll
  for (int w = 0; w < S::kWords; ++w) out.q[w] = make_uint4(half(out.q[w].x), half(out.q[w].y), half(out.q[w].z), half(out.q[w].w));
  // a row that is not there has the weight 0
  const float f = c.on ? c.f : 0.f, minus = c.on ? -c.hi : -INFINITY, lift = c.on ? c.lift : 0.f;
  out.far = __any_sync(0xFFFFFFFFu, is_far(minus));
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int from = (2 * t4 + b) * 4;
    out.f[b] = __shfl_sync(0xFFFFFFFFu, f, from);
    out.lse[b] = __shfl_sync(0xFFFFFFFFu, minus, from);
    out.lift[b] = __shfl_sync(0xFFFFFFFFu, lift, from);
    out.i[b] = __shfl_sync(0xFFFFFFFFu, real ? i : -1, from);    // one that does not count sees NaNs, too
  }
}

// A warp's ring: kAhead tiles' keys (codes, then scales), filled by asynchronous copies.
template <int kDim>
struct Ring {
  static constexpr int kCodes = 8 * kDim, kTile = kCodes + kDim;   // bytes of 16 entries' codes of a head, and with their scales
  // Enough for the latency, and no more: 8, 4 and 3 take 28.8, 60.1 and 48.1 us where these take 26.8, 59.4 and 46.9 (32 heads of
  // d = 64, 16 requests of d = 128, 24 of d = 256).
  static constexpr int kAhead = kDim == 64 ? 4 : kDim == 128 ? 3 : 2;
  static_assert(kAhead * kWarps <= kBlockTiles, "tiles are copied a block ahead at most, where their records are known");
  static constexpr int kBytes = kAhead * kTile;
  // Of 128 bytes of scales a lane copies four; of 64 two lanes copy the same ones.
  __device__ static constexpr int kScaleAt(int lane) { return (kDim == 64 ? lane & 15 : lane) * 4; }
  static constexpr int kSmem = kWarps * kBytes + 2 * kSumTiles * 16 * 4;
};

// A request's tiles that some row sees: [0, sink_t) and [lo_t, ..).
struct Tiles {
  int sink_t, lo_t, count;
  __device__ __forceinline__ int entry(int t) const { return (t < sink_t ? t : t - sink_t + lo_t) * 16; }
};
__device__ __forceinline__ Tiles tiles_of(const KvAccumulateArgs& a, const Request& x) {
  const View v = view_of(a, x);
  Tiles t;
  t.lo_t = v.w0 / 16;
  t.sink_t = min((v.sinks + 15) / 16, t.lo_t);
  t.count = x.q_len ? t.sink_t + (x.n + 15) / 16 - t.lo_t : 0;
  return t;
}

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, 1) kv_accumulate_kernel(const KvAccumulateArgs a) {
  using S = Shape<kDim>;
  using R = Ring<kDim>;
  extern __shared__ __align__(16) uint8_t smem[];
  // from a shuffle, so that what depends on the warp alone is known to be the same in all lanes
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), g = lane >> 2, t4 = lane & 3;
  const uint8_t* const ring = smem + warp * R::kBytes;
  float* const sums = reinterpret_cast<float*>(smem + kWarps * R::kBytes);           // [2][tile * heads + head][16]
  __shared__ Starts<kThreads> starts;
  __shared__ unsigned long long table[4 * kBlockTiles];      // records of the tiles of four blocks; bit 0: its page is bad
  pdl_wait();
  auto count = [&](const Request& x) { return tiles_of(a, x).count; };
  const Deal deal = deal_out<kThreads, false>(a, starts, nullptr, count);
  fade_unseen<kThreads, false>(a, [&](const Request& x, int& from, int& to) {
    const Tiles t = tiles_of(a, x);
    from = t.sink_t * 16;
    to = t.lo_t * 16;
  });
  const long long share = (deal.total + gridDim.x - 1) / gridDim.x;
  long long u = blockIdx.x * share, first;
  const long long end = min(u + share, deal.total);
  int r, top;
  Request x;
  if (u >= end || !find_request<kThreads, false>(a, starts, nullptr, deal, u, r, x, first, top, count)) return;
  for (;;) {
    const Tiles tiles = tiles_of(a, x);
    const View view = view_of(a, x);
    const int begin = int(u - first), n = int(min(end - first, (long long)tiles.count)) - begin;   // the run's tiles of this request
    // those that every row sees whole: [whole, whole + wholes), along the entries one run
    const int last_e = (view.base + 1) / 16 * 16, first_e = a.window ? max(0, view.base + x.q_len - a.window + 15) / 16 * 16 : 0;
    const int whole = first_e / 16 - tiles.lo_t + tiles.sink_t - begin, all_wholes = max(0, (last_e - first_e) / 16);
    // as many heads at a time as there are warps (16 at a time: 64 heads 55 us for 51)
    for (int h0 = 0; h0 < a.H; h0 += kWarps) {
      const int hn = min(kWarps, a.H - h0), lanes = kWarps / hn;          // heads; warps of a head
      const int block = min(kBlockTiles, kSumTiles / hn) / lanes * lanes;   // tiles of a block
      const int around = 4 * block;                                      // of the table
      // Those of tiles [from, to).  Where there is none (a bad page) the cache's first record is copied,
      // and not looked at.
      auto note = [&](int j, const uint8_t* rec) {
        table[j % around] = reinterpret_cast<unsigned long long>((rec ? rec : a.data) + (int64_t)h0 * S::kRecord) | !rec;
      };
      auto look_up = [&](int from, int to) {
        for (int j = from + threadIdx.x; j < min(n, to); j += kThreads) note(j, record_at<kDim>(a, r, x, view, tiles.entry(begin + j)));
      };
      // the first three blocks' pages (a thread has one at most) are on their way while the rows are made ready
      static_assert(3 * kBlockTiles <= kThreads, "a page a thread");
      const int e_first = tiles.entry(begin + threadIdx.x);
      const bool looks = threadIdx.x < min(n, 3 * block) && !unseen(x, view, e_first);
      const int page = looks ? page_at(a, r, e_first) : -1;
      const int mine = warp / hn, h = warp - mine * hn;       // this warp's first tile and its head; warps past the last one of a head: none
      Rows<kDim> y;
      load_rows<T, kDim>(a, y, x, h0 + h);
      const int wholes = y.far ? 0 : all_wholes;     // the loop that looks at each entry holds weights at 1, too
      if (threadIdx.x < min(n, 3 * block)) note(threadIdx.x, looks ? record_in<kDim>(a, page, e_first) : nullptr);
      __syncthreads();
      // ---- the copies, kAhead tiles before the products
      int copy_j = mine < lanes ? mine : n, copy_at = mine, copy_slot = 0;               // tile, its places in the table and in the ring
      const uint32_t ring0 = ptx::smem_u32(ring) + lane * 16, ring_scale = ptx::smem_u32(ring) + R::kCodes + R::kScaleAt(lane);
      const int64_t offset = h * S::kRecord + lane * 16, to_scale = 16 * kDim + R::kScaleAt(lane) - lane * 16;
      auto copy_tile = [&] {
        if (copy_j < n) {
          const uint8_t* const src = reinterpret_cast<const uint8_t*>(table[copy_at] & ~1ull) + offset;
#pragma unroll
          for (int k = 0; k < R::kCodes; k += 512) copy_async16(ring0 + copy_slot + k, src + k);
#pragma unroll
          for (int k = 0; k < kDim; k += 128) copy_async4(ring_scale + copy_slot + k, src + to_scale + k);
          copy_slot = copy_slot + R::kTile == R::kBytes ? 0 : copy_slot + R::kTile;
          copy_j += lanes;
          copy_at = copy_at + lanes >= around ? copy_at + lanes - around : copy_at + lanes;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int i = 0; i < R::kAhead; ++i) copy_tile();
      // where the lane's keys and scales are in the ring
      const uint8_t* const keys = ring + g * (S::kPart / 2) + t4 * (S::kPart / 8);
      const uint8_t* const scales = ring + R::kCodes + g * (kDim / 16) + t4 * (S::kPart / 64);
      int j = mine < lanes ? mine : n, slot = 0;
      for (int j0 = 0, buffer = 0; j0 < n; j0 += block, buffer ^= kSumTiles * 16) {
        const int j1 = min(n, j0 + block);
        // where the lane's sum of the tile goes
        float* out = sums + buffer + ((j - j0) * hn + h) * 16 + g + 8 * (t4 & 1);
        auto work = [&](auto masked, int to) {
#pragma unroll 1
          for (; j < to; j += lanes, out += lanes * hn * 16) {
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kAhead - 1) : "memory");
            __syncwarp();
            Keys<kDim> k;
            read_keys<kDim>(k, keys + slot, scales + slot);
            float s[4];
#pragma unroll
            for (int w = 0; w < S::kWords; ++w) products<kDim>(s, k, w, y.q[w]);
            slot = slot + R::kTile == R::kBytes ? 0 : slot + R::kTile;
            __syncwarp();      // these keys are in registers
            copy_tile();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              s[c] = __fmaf_rn(s[c], y.f[c & 1], y.lse[c & 1]);
              if constexpr (decltype(masked)::value) s[c] = held(s[c], y.lse[c & 1]);
              s[c] = ptx::ex2_approx(s[c]);
            }
            if constexpr (decltype(masked)::value) {
              const int e = tiles.entry(begin + j);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (!sees(a, view, y.i[c & 1], e + g + 8 * (c >> 1))) s[c] = 0.f;
            }
            // over the rows: the four lanes of an entry have two each, and entries g and g + 8
            const float v0 = __fmaf_rn(s[1], y.lift[1], s[0] * y.lift[0]), v1 = __fmaf_rn(s[3], y.lift[1], s[2] * y.lift[0]);
            float v = (t4 & 1 ? v1 : v0) + __shfl_xor_sync(0xFFFFFFFFu, t4 & 1 ? v0 : v1, 1);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
            *out = v;          // lanes t4 and t4 + 2 have the same
          }
        };
        work(std::true_type(), min(j1, whole));
        work(std::false_type(), min(j1, whole + wholes));
        work(std::true_type(), j1);
        // what the entry had, of the first entry that this thread adds up, while the other warps finish
        auto had = [&](int i) { return a.w_in[r * a.w_stride + tiles.entry(begin + j0 + (i >> 4)) + (i & 15)]; };
        float old = 0.f;
        if (h0 == 0 && a.w_in && threadIdx.x < (j1 - j0) * 16 &&
            tiles.entry(begin + j0 + (threadIdx.x >> 4)) + (threadIdx.x & 15) < x.n)
          old = had(threadIdx.x);
        __syncthreads();
        // ---- over the heads, while other warps are in the next block
        look_up(j0 + 3 * block, j0 + 4 * block);
        for (int i = threadIdx.x; i < (j1 - j0) * 16; i += kThreads) {
          const int t = j0 + (i >> 4), e = tiles.entry(begin + t) + (i & 15);
          if (e >= x.n) continue;
          float v = 0.f;
          if (!(table[t % around] & 1))      // an entry of a bad page is not seen
            for (int k = 0; k < hn; ++k) v += sums[buffer + ((i >> 4) * hn + k) * 16 + (i & 15)];
          const int64_t to = r * a.w_stride + e;
          a.w_out[to] = h0 ? a.w_out[to] + v : a.w_in ? __fmaf_rn(a.decay, i == threadIdx.x ? old : had(i), v) : v;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();   // the table and the sums are the next heads' or request's
    }
    u = first + begin + n;
    if (u >= end) break;
    first += tiles.count;
    for (++r; r < a.R; ++r) {
      x = load_request<false>(a, r, top);
      const int mine = count(x);
      if (u < first + mine) break;
      first += mine;
    }
    if (r >= a.R) break;
  }
}

template <typename T, int kDim>
cudaError_t launch(const KvAccumulateArgs& a, cudaStream_t s) {
  constexpr int kSmem = Ring<kDim>::kSmem;
  // once per device and process: this launches nothing
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (a.device & 63);
  if (a.device > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_accumulate_kernel<T, kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const long long tiles = (long long)a.R * ((((int64_t)a.max_pages << a.page_shift) + 15) / 16);   // at most
  return launch_kernel(kv_accumulate_kernel<T, kDim>, dim3(unsigned(std::min<long long>(kPlanSMs, tiles))), kThreads, kSmem, s, true, a);
}

template <int kDim>
cudaError_t launch_dim(const KvAccumulateArgs& a, bool f16, cudaStream_t s) {
  return f16 ? launch<__half, kDim>(a, s) : launch<__nv_bfloat16, kDim>(a, s);
}

// One new token of 131072 entries of 8 heads, 8 rows a head: 23.0 us here, 28.7 there; 12 rows would be two passes here, 29 us there.
// 16 ragged requests of 4 rows: 60 and 81 us.
bool few_rows(int gamma, int max_q) { return gamma * max_q <= 8; }

}  // namespace

size_t kv_accumulate_workspace_bytes(int H, int gamma, int max_q, int num_q, int R, int d) {
  return few_rows(gamma, max_q) ? 256 : kv_accumulate_tc_workspace_bytes(H, gamma, num_q, R, d);
}

cudaError_t launch_kv_accumulate(const KvAccumulateArgs& a, bool f16, cudaStream_t s) {
  if (!few_rows(a.gamma, a.max_q)) return launch_kv_accumulate_tc(a, f16, s);
  return a.d == 64 ? launch_dim<64>(a, f16, s) : a.d == 128 ? launch_dim<128>(a, f16, s) : launch_dim<256>(a, f16, s);
}

}  // namespace upf
