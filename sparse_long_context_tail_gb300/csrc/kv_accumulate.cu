// Attention weight that cache entries have drawn.
//
// For entry e of request r: w_out = decay w_in + sum over the rows (query i, q head h) that see e of
// exp(scale q.k_e - lse), with lse the row's from the attention.  Rows whose lse is -inf saw nothing.
//
// Only the keys' half of the records is read.  A warp takes a unit of kTiles runs of 16 entries (a
// record of every kv head each) through all kv heads, so that an entry's sum stays in its registers
// and comes in one order; rows on N of mma.sync (eight at a time), entries on M, codes times scales
// as operand A straight from the loads.
#include <cfloat>

#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.9259629911266174e-8f;   // their sum is log2 e to 2^-49

struct Request {
  int q0, q_len, n;     // first row, rows, entries; rows 0: nothing to do
};

__device__ __forceinline__ Request load_request(const KvAccumulateArgs& a, int r) {
  Request x{r, 1, a.kv_len[r]};
  bool ok = x.n >= 0 && x.n <= ((int64_t)a.max_pages << a.page_shift) && x.n <= a.w_cols;
  if (a.cu_q) {
    x.q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    ok = ok && x.q0 >= 0 && q1 >= x.q0 && q1 <= a.num_q && q1 - x.q0 <= a.max_q;
    x.q_len = q1 - x.q0;
  }
  if (!ok) {
    set_status(a.status, UPF_ERR_INVALID_ARG);
    x.q0 = x.q_len = x.n = 0;
  }
  return x;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A row's logit factor 2^exp * mantissa of the scale, within fp32.
__device__ __forceinline__ float factor_of(const KvAccumulateArgs& a, int exp) {
  if (exp > 127) return FLT_MAX;
  return fminf(a.scale_mant * __uint_as_float(uint32_t(max(exp, -126) + 127) << 23), FLT_MAX);
}

template <int kDim>
struct Shape {
  static constexpr int kPart = kDim >= 128 ? 128 : kDim;
  static constexpr int kParts = kDim / kPart;
  static constexpr int kPartWords = kPart / 32;            // words of codes of a lane's quarter row of a part
  static constexpr int kWords = kDim / 32;
  static constexpr int kSteps = kDim / 16;
  static constexpr int kRecord = kv::record_bytes(kDim);
};

// A lane's quarters of rows g and g + 8 of a record's keys.
template <int kDim>
struct Keys {
  uint32_t w[2][Shape<kDim>::kWords];
  uint16_t s[2][Shape<kDim>::kParts];    // scales of the quarter's one or two groups
};

template <int kDim>
__device__ __forceinline__ void load_keys(Keys<kDim>& k, const uint8_t* rec, int g, int t4) {
  using S = Shape<kDim>;
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int p = 0; p < S::kParts; ++p) {
      const int row = g + 8 * y;
      const uint8_t* const src = rec + p * (8 * S::kPart) + row * (S::kPart / 2) + t4 * (S::kPart / 8);
      const uint8_t* const sc = rec + 16 * kDim + row * (kDim / 16) + p * 8;
      if constexpr (S::kPart == 128) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
        k.w[y][4 * p] = x.x;
        k.w[y][4 * p + 1] = x.y;
        k.w[y][4 * p + 2] = x.z;
        k.w[y][4 * p + 3] = x.w;
        k.s[y][p] = __ldg(reinterpret_cast<const uint16_t*>(sc + 2 * t4));
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
        k.w[y][0] = x.x;
        k.w[y][1] = x.y;
        k.s[y][0] = __ldg(sc + t4);
      }
    }
}

// Eight rows of a kv head as operand B, and what turns their products into weights.
template <int kDim>
struct Rows {
  uint32_t q[Shape<kDim>::kSteps][2];    // divided by the power of two of the row's largest element
  float f[2], lse[2], lift[2];           // of rows 2 t4, 2 t4 + 1: weight = 2^(s f - lse) lift
  int i[2];                              // their queries; -1: no such row
};

template <typename T, int kDim>
__device__ __forceinline__ void load_rows(const KvAccumulateArgs& a, Rows<kDim>& x, const Request& r, int h, int row0, int g,
                                          int t4) {
  using S = Shape<kDim>;
  constexpr const T* kT = nullptr;
  const int rows = r.q_len * a.gamma, rho = row0 + g;
  const bool real = rho < rows;
  const int i = real ? rho / a.gamma : 0, head = a.qhead[h * a.gamma + (real ? rho - i * a.gamma : 0)];
  const int64_t at = r.q0 + i;
  const T* const src = static_cast<const T*>(a.q) + at * a.q_stride + head * kDim;
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < S::kParts; ++p)
#pragma unroll
    for (int v = 0; v < S::kPart / 32; ++v) {
      const uint4 y = real ? __ldg(reinterpret_cast<const uint4*>(src + p * 128 + t4 * (S::kPart / 4)) + v) : make_uint4(0, 0, 0, 0);
      const int s = p * 8 + 2 * v;
      x.q[s][0] = y.x;
      x.q[s][1] = y.y;
      x.q[s + 1][0] = y.z;
      x.q[s + 1][1] = y.w;
      top = kv::max_abs2(kv::max_abs2(top, kv::max_abs2(y.x, y.y, kT), kT), kv::max_abs2(y.z, y.w, kT), kT);
    }
  const float lse = real ? __ldg(a.lse + at * a.Hq + head) : -INFINITY;
  const float2 tops = kv::pair_to_float2(top, kT);
  // a NaN or an infinity anywhere in the row: bits at and above those of infinity
  uint32_t amax = max(__float_as_uint(fabsf(tops.x)), __float_as_uint(fabsf(tops.y)));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  const bool bad = real && (amax >= 0x7F800000u || !(lse < INFINITY));
  if (bad && t4 == 0) set_status(a.status, UPF_ERR_NONFINITE);
  const bool on = real && !bad && lse > -INFINITY;
  int e = int(amax >> 23) - 127;
  e = !on || amax == 0 ? 0 : max(-126, min(e, 126));
  const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
  for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float2 y = kv::pair_to_float2(x.q[s][b], kT);
      x.q[s][b] = on ? pack_f16(y.x * down, y.y * down) : 0u;
    }
  // the logarithm's product with log2 e in two parts: the rounding of one would be that of every weight of the row
  const float hi = lse * kLog2e, lo = __fmaf_rn(lse, kLog2e, -hi) + lse * kLog2eLow, lift = ptx::ex2_approx(-lo);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int from = (2 * t4 + b) * 4;
    x.f[b] = factor_of(a, a.scale_exp + __shfl_sync(0xFFFFFFFFu, e, from));
    x.lse[b] = __shfl_sync(0xFFFFFFFFu, hi, from);
    x.lift[b] = __shfl_sync(0xFFFFFFFFu, lift, from);
    x.i[b] = __shfl_sync(0xFFFFFFFFu, on ? i : -1, from);
  }
  __syncwarp();   // the matrix instructions take whole warps
}

// s[entry g, g + 8][rows 2 t4, 2 t4 + 1] = keys . rows
template <int kDim>
__device__ __forceinline__ void products(float (&s)[4], const Keys<kDim>& k, const Rows<kDim>& x) {
  using S = Shape<kDim>;
  s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
  for (int w = 0; w < S::kWords; ++w) {
    const int p = w / S::kPartWords;
    uint32_t x0[4], x1[4];
    kv::e2m1x8_to_f16(k.w[0][w], x0);
    kv::e2m1x8_to_f16(k.w[1][w], x1);
    const uint32_t c0 = kv::e4m3x2_to_f16x2(k.s[0][p]), c1 = kv::e4m3x2_to_f16x2(k.s[1][p]);
    const __half2 h0 = *reinterpret_cast<const __half2*>(&c0), h1 = *reinterpret_cast<const __half2*>(&c1);
    const bool second = S::kPart == 128 && w % S::kPartWords >= 2;
    const __half2 s0 = second ? __high2half2(h0) : __low2half2(h0), s1 = second ? __high2half2(h1) : __low2half2(h1);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const uint32_t af[4] = {hmul2(x0[2 * st], s0), hmul2(x1[2 * st], s1), hmul2(x0[2 * st + 1], s0), hmul2(x1[2 * st + 1], s1)};
      mma_f16(s, af, x.q[2 * w + st]);
    }
  }
}

template <typename T, int kDim, int kTiles>
__global__ void __launch_bounds__(kThreads) kv_accumulate_kernel(const KvAccumulateArgs a) {
  using S = Shape<kDim>;
  constexpr int kUnit = 16 * kTiles;
  __shared__ long long starts[kThreads + 1];   // units before each thread's requests
  __shared__ long long warp_sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int per = (a.R + kThreads - 1) / kThreads;
  long long units = 0;
  for (int j = 0; j < per; ++j) {
    const int r = threadIdx.x * per + j;
    if (r >= a.R) break;
    const Request x = load_request(a, r);
    if (x.q_len) units += (x.n + kUnit - 1) / kUnit;
  }
  long long sum = units;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) sum += warp_sums[w];
  starts[threadIdx.x + 1] = sum;
  if (threadIdx.x == 0) starts[0] = 0;
  __syncthreads();
  const long long total = starts[kThreads];

  for (long long u = (long long)blockIdx.x * kWarps + warp; u < total; u += (long long)gridDim.x * kWarps) {
    // the unit's request: the thread whose run of requests holds it, then along that run
    int lo = 0, hi = kThreads;      // starts[lo] <= u < starts[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= u) lo = mid;
      else hi = mid;
    }
    long long first = starts[lo];
    int r = lo * per;
    Request x = load_request(a, r);
    for (;;) {
      const long long mine = x.q_len ? (x.n + kUnit - 1) / kUnit : 0;
      if (u < first + mine) break;
      first += mine;
      if (++r >= a.R) return;   // the lengths have changed under the call
      x = load_request(a, r);
    }
    const int e0 = int(u - first) * kUnit;
    const int base = x.n - x.q_len;                                  // position of query 0
    const int64_t w_lo = a.window ? max((int64_t)0, (int64_t)base - a.window + 1) : 0;   // first entry inside some row's window
    const int w0 = int(w_lo), sinks = min(a.sinks, w0);

    // the records of head 0, one tile a lane
    const uint8_t* record = nullptr;
    if (lane < kTiles) {
      const int e = e0 + 16 * lane;
      if (e < x.n && (e + 15 >= w0 || e < sinks)) {
        const int page = a.page_table[(int64_t)r * a.page_stride + (e >> a.page_shift)];
        const int64_t b = ((int64_t)page << (a.page_shift - 4)) + ((e & ((1 << a.page_shift) - 1)) >> 4);
        if (page >= 0 && b < (a.num_slots >> 4)) record = a.data + b * a.H * S::kRecord;
        else set_status(a.status, UPF_ERR_INVALID_ARG);
      }
    }
    const uint8_t* rec[kTiles];
    // entries that every row sees: none of the tiles' need a look then
    const bool whole = e0 + kUnit <= base + 1 && (a.window == 0 || e0 > base + x.q_len - 1 - a.window);
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
      rec[i] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(record), i));
    float acc[kTiles][2] = {};
    const int rows = x.q_len * a.gamma;
    for (int h = 0; h < a.H; ++h) {
      Keys<kDim> k[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        if (rec[i]) load_keys<kDim>(k[i], rec[i] + (int64_t)h * S::kRecord, g, t4);
      for (int row0 = 0; row0 < rows; row0 += 8) {
        Rows<kDim> y;
        load_rows<T, kDim>(a, y, x, h, row0, g, t4);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          if (!rec[i]) continue;
          float s[4];
          products<kDim>(s, k[i], y);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int b = c & 1, e = e0 + 16 * i + g + 8 * (c >> 1);
            bool sees = y.i[b] >= 0;
            if (!whole) {
              const int p = base + y.i[b];
              sees = sees && e <= p && (a.window == 0 || p - e < a.window || e < a.sinks);
            }
            const float w = ptx::ex2_approx(__fmaf_rn(s[c], y.f[b], -y.lse[b]));
            acc[i][c >> 1] = sees ? __fmaf_rn(w, y.lift[b], acc[i][c >> 1]) : acc[i][c >> 1];
          }
        }
      }
    }
    // the four lanes of an entry have two rows of each eight
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float v = acc[i][y];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        const int e = e0 + 16 * i + g + 8 * y;
        if (t4 != 0 || e >= x.n) continue;
        const int64_t at = r * a.w_stride + e;
        a.w_out[at] = a.w_in ? __fmaf_rn(a.decay, a.w_in[at], v) : v;
      }
  }
}

template <typename T, int kDim>
cudaError_t launch(const KvAccumulateArgs& a, cudaStream_t s) {
  constexpr int kTiles = kDim == 256 ? 2 : 4;
  const long long most = (long long)a.R * ((((int64_t)a.max_pages << a.page_shift) + 15) / 16);   // tiles at most
  const long long full = 2 * kPlanSMs;
  if (most <= full * kWarps)
    return launch_kernel(kv_accumulate_kernel<T, kDim, 1>, dim3(unsigned((most + kWarps - 1) / kWarps)), kThreads, 0, s, false, a);
  return launch_kernel(kv_accumulate_kernel<T, kDim, kTiles>, dim3(unsigned(full)), kThreads, 0, s, false, a);
}

template <int kDim>
cudaError_t launch_dim(const KvAccumulateArgs& a, bool f16, cudaStream_t s) {
  return f16 ? launch<__half, kDim>(a, s) : launch<__nv_bfloat16, kDim>(a, s);
}

}  // namespace

size_t kv_accumulate_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_kv_accumulate(const KvAccumulateArgs& a, bool f16, cudaStream_t s) {
  return a.d == 64 ? launch_dim<64>(a, f16, s) : a.d == 128 ? launch_dim<128>(a, f16, s) : launch_dim<256>(a, f16, s);
}

}  // namespace upf
