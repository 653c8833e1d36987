// Rotary positions of queries and keys.
//
// Pair i of a head at position p turns by p f_i radians.  With
// turns_i = 2^64 f_i / (2 pi) as an integer, p * turns_i modulo 2^64 is the fraction of
// a turn, whatever the position's size and sign: one 64-bit product in place of an angle whose
// reduction would need more than fp32 (at p = 10^5 an fp32 angle is off by 2^-8).  Its upper 32 bits
// are taken, 2^-32 of a turn, under the rounding of the fp32 sine and cosine.
//
// Bound by HBM: every element is read and written once (131072 tokens of 32 + 8 heads of d = 128: 392 us, 6.8 TB/s;
// 20011 rows of d = 256 out of a wider row: 58 us of 54).  Eight tokens: 2.6 us, the launch and two loads one after the other.  A thread takes the same
// 16 dims (eight pairs) of a token in several heads, so that sines and cosines are worked out once
// for all of them and 2 kHeads 16-byte loads are in flight.
#include "kv_layout.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;     // heads of a thread whose loads are in flight together

// Cosine and sine of the angle of `pos`, times m; sign -1 turns back.
__device__ __forceinline__ float2 turn_of(uint64_t turns, int64_t pos, float m, float sign) {
  const uint64_t x = uint64_t(pos) * turns + 0x80000000ull;
  const float half_turns = float(int32_t(x >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * m, s * (m * sign));
}

template <typename T>
__device__ __forceinline__ void rotate8(uint4& x, uint4& y, const float2 (&cs)[8], bool interleaved) {
  constexpr const T* kT = nullptr;
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (interleaved) {   // word i: pair i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = kv::pair_to_float2(w[i], kT);
      w[i] = kv::float2_to_pair(v.x * cs[i].x - v.y * cs[i].y, v.y * cs[i].x + v.x * cs[i].y, kT);
    }
  } else {             // words i, 4 + i: the first and second elements of pairs 2i, 2i + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = kv::pair_to_float2(w[i], kT), b = kv::pair_to_float2(w[4 + i], kT);
      const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
      w[i] = kv::float2_to_pair(a.x * c0.x - b.x * c0.y, a.y * c1.x - b.y * c1.y, kT);
      w[4 + i] = kv::float2_to_pair(b.x * c0.x + a.x * c0.y, b.y * c1.x + a.y * c1.y, kT);
    }
  }
  x = make_uint4(w[0], w[1], w[2], w[3]);
  y = make_uint4(w[4], w[5], w[6], w[7]);
}

// rotary_dim a multiple of 16: a thread per token, run of 16 dims and group of heads.
// Runs past the rotary dims are copied (none where the outputs are the inputs).
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  const uint32_t per = a.runs * a.groups;
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, t = i / per;
  if (t >= a.T) return;
  if (a.count && t >= *a.count) return;
  const uint32_t rest = uint32_t(i - t * per), group = rest / a.runs, run = rest - group * a.runs;
  const bool turn = run < a.rotary / 16;
  // the thread's two vectors of eight elements within a head
  int first = run * 16, second = first + 8;
  if (turn && !a.interleaved) {
    first = run * 8;
    second = first + a.rotary / 2;
  }
  float2 cs[8];
  if (turn) {
    const int64_t pos = a.positions[t];
    const ulonglong2* const turns = reinterpret_cast<const ulonglong2*>(a.turns + run * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const ulonglong2 f = __ldg(turns + j);
      cs[2 * j] = turn_of(f.x, pos, a.magnitude, a.sign);
      cs[2 * j + 1] = turn_of(f.y, pos, a.magnitude, a.sign);
    }
  }
  const int heads = a.q.heads + a.k.heads, h1 = min(heads, int(group + 1) * a.heads_each);
  for (int h0 = group * a.heads_each; h0 < h1; h0 += kHeads) {
    uint4 x[kHeads], y[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      if (h >= h1) break;
      const RopeRows& r = h < a.q.heads ? a.q : a.k;
      const T* const src = static_cast<const T*>(r.in) + t * r.in_stride + (h < a.q.heads ? h : h - a.q.heads) * a.d;
      x[j] = *reinterpret_cast<const uint4*>(src + first);
      y[j] = *reinterpret_cast<const uint4*>(src + second);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      if (h >= h1) break;
      const RopeRows& r = h < a.q.heads ? a.q : a.k;
      T* const dst = static_cast<T*>(r.out) + t * r.out_stride + (h < a.q.heads ? h : h - a.q.heads) * a.d;
      if (turn) rotate8<T>(x[j], y[j], cs, a.interleaved);
      *reinterpret_cast<uint4*>(dst + first) = x[j];
      *reinterpret_cast<uint4*>(dst + second) = y[j];
    }
  }
}

// Any even rotary_dim: a thread per token and two dims, all heads.  Element by element, a table load and a sine a pair:
// 131072 tokens of 32 + 8 heads of d = 128, 24 dims of them turned, 717 us; 48 dims by the kernel above 396.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const RopeArgs a) {
  constexpr const T* kT = nullptr;
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, t = i / a.runs;
  if (t >= a.T) return;
  if (a.count && t >= *a.count) return;
  const int p = int(i - t * a.runs);
  const bool turn = p < a.rotary / 2;
  const bool halves = turn && !a.interleaved;
  const int first = halves ? p : 2 * p, second = halves ? p + a.rotary / 2 : first + 1;
  const float2 cs = turn ? turn_of(a.turns[p], a.positions[t], a.magnitude, a.sign) : make_float2(0.f, 0.f);
  for (int h = 0; h < a.q.heads + a.k.heads; ++h) {
    const RopeRows& r = h < a.q.heads ? a.q : a.k;
    const int at = (h < a.q.heads ? h : h - a.q.heads) * a.d;
    const uint16_t* const src = static_cast<const uint16_t*>(r.in) + t * r.in_stride + at;
    uint16_t* const dst = static_cast<uint16_t*>(r.out) + t * r.out_stride + at;
    uint32_t w = uint32_t(src[first]) | uint32_t(src[second]) << 16;
    if (turn) {
      const float2 v = kv::pair_to_float2(w, kT);
      w = kv::float2_to_pair(v.x * cs.x - v.y * cs.y, v.y * cs.x + v.x * cs.y, kT);
    }
    dst[first] = uint16_t(w);
    dst[second] = uint16_t(w >> 16);
  }
}

template <typename T>
cudaError_t launch(RopeArgs a, cudaStream_t s) {
  const bool in_place = (!a.q.heads || a.q.in == a.q.out) && (!a.k.heads || a.k.in == a.k.out);
  const int dims = in_place ? a.rotary : a.d;
  if (a.rotary % 16) {
    a.runs = dims / 2;
    const int64_t blocks = ((int64_t)a.T * a.runs + kThreads - 1) / kThreads;
    return launch_kernel(rope_any_kernel<T>, dim3(unsigned(blocks)), kThreads, 0, s, true, a);
  }
  a.runs = dims / 16;
  // All heads by one thread, so that its sines serve all of them, unless that leaves SMs without
  // threads: then as few heads as kHeads each (8 tokens: 5.3 and 2.6 us; 20011 rows of d = 256: 58.5 and 60.5).
  const int heads = a.q.heads + a.k.heads;
  const int64_t full = (int64_t)kPlanSMs * 1024, mine = (int64_t)a.T * a.runs;
  int groups = int((full + mine - 1) / mine);
  const int most = (heads + kHeads - 1) / kHeads;
  if (groups > most) groups = most;
  a.heads_each = (most + groups - 1) / groups * kHeads;
  a.groups = (heads + a.heads_each - 1) / a.heads_each;
  const int64_t blocks = (mine * a.groups + kThreads - 1) / kThreads;
  return launch_kernel(rope_kernel<T>, dim3(unsigned(blocks)), kThreads, 0, s, true, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool f16, cudaStream_t s) {
  return f16 ? launch<__half>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace upf
