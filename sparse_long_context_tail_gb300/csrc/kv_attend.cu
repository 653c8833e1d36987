// Attention of new tokens over the 4-bit cache.
//
// For row (query i of request r, q head h), at position p = kv_len - q_len + i:
//   visible entries e: e <= p, and without a window or with p - e < window or
//   e < sinks;  out = sum_e softmax_e(scale q.k_e) v_e, lse = ln sum_e exp(scale q.k_e).
// Nothing visible: out = 0, lse = -inf.
#include <cfloat>

#include "kv_layout.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Request {
  int q0, q_len, n;   // first row, rows, cache entries
};

// What the device tables say about request r; a table that makes no sense gives
// a request without rows or without entries, and an error in the status word.
__device__ __forceinline__ Request load_request(const KvAttendArgs& a, int r) {
  Request x{r, 1, 0};
  bool ok = true;
  if (a.cu_q) {
    x.q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    x.q_len = q1 - x.q0;
    if (x.q0 < 0 || q1 < x.q0 || q1 > a.num_q || x.q_len > a.max_q) {
      ok = false;
      x.q0 = x.q_len = 0;
    }
  }
  x.n = a.kv_len[r];
  if (x.n < 0 || x.n > (int64_t)a.max_pages << a.page_shift) {
    ok = false;
    x.n = 0;
  }
  if (!ok) set_status(a.status, UPF_ERR_INVALID_ARG);
  return x;
}

// One CTA per row; its warps take the entries in turn, the lanes share the dims.
template <typename T, int kDim>
__global__ void __launch_bounds__(256) kv_attend_row_kernel(const KvAttendArgs a) {
  constexpr int kPer = kDim / 32;
  __shared__ float sm[8], sl[8], so[8][kDim];
  const int r = blockIdx.x, i = blockIdx.y, h = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Request x = load_request(a, r);
  if (i >= x.q_len) return;
  const int g = a.kv_of_q[h];
  const int64_t row = x.q0 + i;
  const int p = x.n - x.q_len + i;
  float q[kPer], o[kPer];
  const T* qp = static_cast<const T*>(a.q) + row * a.q_stride + (int64_t)h * kDim;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    q[j] = float(qp[lane * kPer + j]);
    o[j] = 0.f;
  }
  float m = -FLT_MAX, l = 0.f;
  for (int e = warp; e <= p; e += 8) {
    if (a.window && p - e >= a.window && e >= a.sinks) continue;
    const int page = a.page_table[(int64_t)r * a.page_stride + (e >> a.page_shift)];
    const int64_t slot = ((int64_t)page << a.page_shift) + (e & ((1 << a.page_shift) - 1));
    if (page < 0 || slot >= a.num_slots) {
      set_status(a.status, UPF_ERR_INVALID_ARG);
      continue;
    }
    const uint8_t* rec = a.data + ((slot >> 4) * a.H + g) * kv::record_bytes(kDim);
    const int er = int(slot & 15), grp = lane * kPer / 16;
    float kx[kPer], vx[kPer], dot = 0.f;
    const float ks = kv::half2_bits_to_float2(kv::e4m3x2_to_f16x2(rec[kv::k_scale(kDim, er, grp)])).x;
    const float vs = kv::half2_bits_to_float2(kv::e4m3x2_to_f16x2(rec[kv::v_scale(kDim, er, grp)])).x;
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
      const int in = (lane * kPer + j) % 16;   // dim inside the group
      const uint8_t kb = rec[kv::k_codes(kDim, er, grp) + in / 2];
      const int vo = kDim == 64 ? (in / 8) * kv::v_chunk_stride(64) + (in % 8) / 2 : in / 2;
      const uint8_t vb = rec[kv::v_codes(kDim, er, grp) + vo];
      uint32_t hk[4], hv[4];
      kv::e2m1x8_to_f16(kb, hk);
      kv::e2m1x8_to_f16(vb, hv);
      const float2 k2 = kv::half2_bits_to_float2(hk[0]), v2 = kv::half2_bits_to_float2(hv[0]);
      kx[j] = k2.x * ks;
      kx[j + 1] = k2.y * ks;
      vx[j] = v2.x * vs;
      vx[j + 1] = v2.y * vs;
      dot += q[j] * kx[j] + q[j + 1] * kx[j + 1];
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, s);
    const float y = dot * a.scale_log2;
    const float m2 = fmaxf(m, y), c = exp2f(m - m2), w = exp2f(y - m2);
    l = l * c + w;
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = o[j] * c + w * vx[j];
    m = m2;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) so[warp][lane * kPer + j] = o[j];
  __syncthreads();
  float mx = -FLT_MAX, lx = 0.f;
  for (int w = 0; w < 8; ++w) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < 8; ++w) lx += sl[w] * exp2f(sm[w] - mx);
  for (int j = threadIdx.x; j < kDim; j += blockDim.x) {
    float acc = 0.f;
    for (int w = 0; w < 8; ++w) acc += so[w][j] * exp2f(sm[w] - mx);
    const uint32_t b = kv::float2_to_pair(lx > 0.f ? acc / lx * a.v_mul : (lx == 0.f ? 0.f : lx), 0.f,
                                          static_cast<const T*>(nullptr));
    reinterpret_cast<uint16_t*>(a.out)[row * a.out_stride + (int64_t)h * kDim + j] = uint16_t(b);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[row * a.Hq + h] = lx > 0.f ? (mx + log2f(lx)) * kLn2 : (lx == 0.f ? -INFINITY : lx);
}

}  // namespace

size_t kv_attend_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_kv_attend(const KvAttendArgs& a, bool f16, cudaStream_t s) {
  const dim3 grid(a.R, a.max_q, a.Hq);
#define UPF_ROW(D)                                                                          \
  (f16 ? launch_kernel(kv_attend_row_kernel<__half, D>, grid, 256, 0, s, false, a)          \
       : launch_kernel(kv_attend_row_kernel<__nv_bfloat16, D>, grid, 256, 0, s, false, a))
  return a.d == 64 ? UPF_ROW(64) : a.d == 128 ? UPF_ROW(128) : UPF_ROW(256);
#undef UPF_ROW
}

}  // namespace upf
