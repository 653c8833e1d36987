// What the kernels of the accumulated attention weights share: requests and what their rows see of them,
// how work is dealt out over the requests, and what turns a row's products into weights.
#pragma once

#include <cfloat>

#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {
namespace acc {

struct Request {
  int q0, q_len, n;     // first row, rows, entries; no rows: nothing to do
};

// Request r, and whether it makes sense by itself.
__device__ __forceinline__ bool look_at(const KvAccumulateArgs& a, int r, Request& x) {
  x = Request{r, 1, a.kv_len[r]};
  bool ok = x.n >= 0 && x.n <= ((int64_t)a.max_pages << a.page_shift) && x.n <= a.w_cols;
  if (a.cu_q) {
    x.q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    ok = ok && x.q0 >= 0 && q1 >= x.q0 && q1 <= a.num_q && q1 - x.q0 <= a.max_q;
    x.q_len = q1 - x.q0;
  }
  return ok;
}
// Where the rows end of requests up to this one, of which `top` were those of the ones before it.
__device__ __forceinline__ int end_of(const Request& x, bool ok, int top) { return ok && x.q_len > 0 ? max(top, x.q0 + x.q_len) : top; }

// Request x after look_at(): with no rows if it is to be skipped.  kRowsOnce: also a request whose rows begin before `top`, which
// is moved on (cu_q is not ascending then): the many-row kernel's rows have places in the workspace by their numbers, and
// those of requests that go back may be others' places.
template <bool kRowsOnce>
__device__ __forceinline__ void admit(const KvAccumulateArgs& a, Request& x, bool ok, int& top) {
  if (kRowsOnce && a.cu_q) {
    const int before = top;
    top = end_of(x, ok, top);
    ok = ok && (x.q_len == 0 || x.q0 >= before);
  }
  if (!ok) {
    set_status(a.status, UPF_ERR_INVALID_ARG);
    x.q0 = x.q_len = x.n = 0;
  }
}
template <bool kRowsOnce>
__device__ __forceinline__ Request load_request(const KvAccumulateArgs& a, int r, int& top) {
  Request x;
  const bool ok = look_at(a, r, x);
  admit<kRowsOnce>(a, x, ok, top);
  return x;
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

// What of a request's entries its rows see.
struct View {
  int base;        // position of query 0
  int w0, sinks;   // first entry inside some row's window; first entries that stay visible before it
};
__device__ __forceinline__ View view_of(const KvAccumulateArgs& a, const Request& x) {
  View v;
  v.base = x.n - x.q_len;
  v.w0 = a.window ? int(max((int64_t)0, (int64_t)v.base - a.window + 1)) : 0;
  v.sinks = min(a.sinks, v.w0);
  return v;
}

// Keys of head 0 of the 16 entries from e on, or null if no row sees one of them or their page is bad.
__device__ __forceinline__ bool unseen(const Request& x, const View& v, int e) { return e >= x.n || (e + 15 < v.w0 && e >= v.sinks); }
__device__ __forceinline__ int page_at(const KvAccumulateArgs& a, int r, int e) {
  return a.page_table[(int64_t)r * a.page_stride + (e >> a.page_shift)];
}
template <int kDim>
__device__ __forceinline__ const uint8_t* record_in(const KvAccumulateArgs& a, int page, int e) {
  const int64_t b = ((int64_t)page << (a.page_shift - 4)) + ((e & ((1 << a.page_shift) - 1)) >> 4);
  if (page >= 0 && b < (a.num_slots >> 4)) return a.data + b * a.H * Shape<kDim>::kRecord;
  set_status(a.status, UPF_ERR_INVALID_ARG);
  return nullptr;
}
template <int kDim>
__device__ __forceinline__ const uint8_t* record_at(const KvAccumulateArgs& a, int r, const Request& x, const View& v, int e) {
  return unseen(x, v, e) ? nullptr : record_in<kDim>(a, page_at(a, r, e), e);
}

// Does query i of the request (-1: none) see entry e?
__device__ __forceinline__ bool sees(const KvAccumulateArgs& a, const View& v, int i, int e) {
  const int p = v.base + i;
  return i >= 0 && e <= p && (a.window == 0 || p - e < a.window || e < a.sinks);
}

// Does every row see all entries [e0, e1)?
__device__ __forceinline__ bool all_seen(const KvAccumulateArgs& a, const Request& x, const View& v, int e0, int e1) {
  return e1 <= v.base + 1 && (a.window == 0 || e0 > v.base + x.q_len - 1 - a.window);
}

// ------------------------------------------------------------- dealing out --
// Units of all requests in order, count(request) of each; thread i has looked at requests [i * per, (i + 1) * per).

struct Deal {
  long long total;
  int per;
};
template <int kThreads>
struct Starts {
  long long starts[kThreads + 1];        // units before each thread's requests
  long long warp_sums[kThreads / 32];
  int warp_tops[kThreads / 32];
};

// `tops` [kThreads], in shared memory: where the rows of the requests before each thread's end (kRowsOnce).
template <int kThreads, bool kRowsOnce, typename Count>
__device__ __forceinline__ Deal deal_out(const KvAccumulateArgs& a, Starts<kThreads>& s, int* tops, Count&& count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Deal d;
  d.per = (a.R + kThreads - 1) / kThreads;
  int top = 0;
  Request x{};
  bool ok = false;
  const bool kept = kRowsOnce && a.cu_q && a.R > 1 && d.per == 1;      // this thread's request is looked at once
  if (kRowsOnce && a.cu_q && a.R > 1) {
    for (int j = 0; j < d.per; ++j) {
      const int r = threadIdx.x * d.per + j;
      if (r < a.R) {
        ok = look_at(a, r, x);
        top = end_of(x, ok, top);
      }
    }
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, top, k);
      if (lane >= k) top = max(top, y);
    }
    if (lane == 31) s.warp_tops[warp] = top;
    top = __shfl_up_sync(0xFFFFFFFFu, top, 1);
    if (lane == 0) top = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) top = max(top, s.warp_tops[w]);
  }
  if (kRowsOnce) tops[threadIdx.x] = top;
  long long sum = 0;
  for (int j = 0; j < d.per; ++j) {
    const int r = threadIdx.x * d.per + j;
    if (r < a.R) {
      if (!kept) ok = look_at(a, r, x);
      admit<kRowsOnce>(a, x, ok, top);
      sum += count(x);
    }
  }
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, k);
    if (lane >= k) sum += y;
  }
  if (lane == 31) s.warp_sums[warp] = sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) sum += s.warp_sums[w];
  s.starts[threadIdx.x + 1] = sum;
  if (threadIdx.x == 0) s.starts[0] = 0;
  __syncthreads();
  d.total = s.starts[kThreads];
  return d;
}

// The request that unit u belongs to, the units before it, and where the rows up to it end; false if the lengths have changed under
// the call.
template <int kThreads, bool kRowsOnce, typename Count>
__device__ __forceinline__ bool find_request(const KvAccumulateArgs& a, const Starts<kThreads>& s, const int* tops, const Deal& d,
                                             long long u, int& r, Request& x, long long& first, int& top, Count&& count) {
  // the thread whose run of requests holds it, then along that run
  int lo = 0, hi = kThreads;      // starts[lo] <= u < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.starts[mid] <= u) lo = mid;
    else hi = mid;
  }
  first = s.starts[lo];
  top = kRowsOnce ? tops[lo] : 0;
  for (r = lo * d.per; r < a.R; ++r) {
    x = load_request<kRowsOnce>(a, r, top);
    const int mine = count(x);
    if (u < first + mine) return true;
    first += mine;
  }
  return false;
}

// Entries behind the window, where no unit is, fade too: [from, to) of each request, which range() gives.
template <int kThreads, bool kRowsOnce, typename Range>
__device__ __forceinline__ void fade_unseen(const KvAccumulateArgs& a, Range&& range) {
  if (!a.window || (a.w_in == a.w_out && a.decay == 1.f)) return;
  for (int r = 0, top = 0; r < a.R; ++r) {
    const Request x = load_request<kRowsOnce>(a, r, top);
    if (!x.q_len) continue;
    int from, to;
    range(x, from, to);
    for (int64_t e = from + (int64_t)blockIdx.x * kThreads + threadIdx.x; e < to; e += (int64_t)gridDim.x * kThreads) {
      const int64_t at = r * a.w_stride + e;
      a.w_out[at] = a.w_in ? a.decay * a.w_in[at] : 0.f;
    }
  }
}

// ------------------------------------------------------------------- rows --

__device__ __forceinline__ __half2 as_half2(uint32_t a) { return *reinterpret_cast<const __half2*>(&a); }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(as_half2(a), b);
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

// A weight is 2^(s f - hi) lift, with s the product of the key and of the row divided by a power of two
// (times `down`).  hi and what its rounding leaves (in `lift`) are lse * log2 e: the rounding of one number would be
// that of every weight of the row.  (So in the kernel for few rows.  The one for many rows has one number for both, -(hi + low),
// a word less a row to read for each entry: its weights are off by 2^-24 |lse| more, which an fp32 lse is off by itself.)
//
// From |hi| = kFar on the rounding of lse alone is half a power of two and more, so there lift is 1, and
// a weight, which the row's other weights leave 1 at most, is held at 1: an exponent that is off by
// thousands would make it infinite.  (At 1e10 `low` is -247, and lift as a factor of its own infinite: 0 times it a NaN.)
constexpr float kFar = 0x1p23f;

struct RowConstants {
  bool on, bad, zero;      // does it count; is it not finite; is it all zeros
  int e;                   // the power of two
  float down, f, hi, low, lift;
};

// Is a row with hi (or -hi) one whose weights are held at 1?
__device__ __forceinline__ bool is_far(float hi) { return fabsf(hi) >= kFar && fabsf(hi) < INFINITY; }
// The exponent of a weight of such a row (a NaN stays one), or of any other.
__device__ __forceinline__ float held(float x, float hi) { return fabsf(hi) >= kFar && x > 0.f ? 0.f : x; }

// `amax`: bits of the row's largest magnitude in fp32 (at and above those of infinity if it has a NaN or an infinity).
__device__ __forceinline__ RowConstants row_constants(const KvAccumulateArgs& a, bool real, uint32_t amax, float lse) {
  constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.9259629911266174e-8f;   // their sum is log2 e to 2^-49
  RowConstants c;
  c.hi = lse * kLog2e;
  c.bad = real && (amax >= 0x7F800000u || (lse != -INFINITY && !(fabsf(c.hi) < INFINITY)));
  c.on = real && !c.bad && lse > -INFINITY;
  c.zero = amax == 0;
  c.e = !c.on || c.zero ? 0 : max(-126, min(int(amax >> 23) - 127, 126));
  c.down = __uint_as_float(uint32_t(127 - c.e) << 23);
  c.f = factor_of(a, a.scale_exp + c.e);
  c.low = __fmaf_rn(lse, kLog2e, -c.hi) + lse * kLog2eLow;
  if (is_far(c.hi)) {
    const float both = c.hi + c.low;
    if (fabsf(both) < INFINITY) c.hi = both;
    c.low = 0.f;
  }
  c.lift = ptx::ex2_approx(-c.low);
  return c;
}

}  // namespace acc

cudaError_t launch_kv_accumulate_tc(const KvAccumulateArgs& a, bool f16, cudaStream_t s);
size_t kv_accumulate_tc_workspace_bytes(int H, int gamma, int num_q, int R, int d);

}  // namespace upf
