// Writing tokens' keys and values into the 4-bit cache and reading them back.
//
// Both move 2.56 bytes per element and do next to nothing with them, so they are
// bound by HBM.  A warp takes four tokens.  Writing, a lane takes a whole group (16
// dims, two 16-byte loads of the same sector), so that its largest magnitude, its
// scale and their reciprocals are worked out once and without an exchange; the
// values' codes of four tokens whose slots follow one another fill whole sectors.
// Reading, a lane takes eight dims, so that a warp's 16-byte stores fill whole
// 128-byte lines: with a group a lane they half filled each sector twice.  Measured
// (8 heads, d = 128): 131072 entries read in 105 us, 0.97 of the copy rate, against 123
// with a group a lane; 32768 tokens written in 31 us (0.82 of it) with a group a lane,
// against 38 with eight dims a lane, which works every scale out twice.
//
// A slot given twice in one call takes the later token's values, as if the
// tokens were written in order: without a rule the two tokens' groups could mix.
// Short calls look for a later token with the same slot; longer ones claim
// their slots first (owner[slot] = the latest token), in one launch of a cluster
// of CTAs whose cost goes with the tokens, not with the size of the cache, and
// which the loads of the writing launch do not wait for.  Measured, looking against
// claiming, us: 8 heads of d = 128: 64 tokens 2.4 and 3.9, 1024 tokens 3.3 and 5.5, 2048 tokens
// 4.6 and 6.3, 4096 tokens 7.9 and 7.7; one head of d = 64, where the looks are all there is:
// 64 tokens 2.2 and 3.9, 1024 tokens 7.0 and 5.2, 4096 tokens 11.2 and 5.5.  1024 tokens
// (UPF_KV_FEW_TOKENS) lie between the two crossings.
#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

constexpr int kQuad = 4;              // tokens of a warp
constexpr int kRuns = 2;              // runs of 64 dims that a reading warp has in flight
constexpr int kClaimCtas = 8, kClaimThreads = 1024;

__device__ __forceinline__ int token_count(const int32_t* count, int T) {
  return count ? min(max(*count, 0), T) : T;
}

// Group `i` of token t, counted along the kv heads: keys and values.
struct Group {
  uint32_t k[8], v[8];
};

template <typename T>
__device__ __forceinline__ void load_words(const T* src, uint32_t (&w)[8], bool on) {
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  if (on) {
    x = reinterpret_cast<const uint4*>(src)[0];
    y = reinterpret_cast<const uint4*>(src)[1];
  }
  w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
}

template <typename T>
__device__ __forceinline__ Group load_group(const KvWriteArgs& a, int64_t t, int i, bool on) {
  Group x;
  load_words(static_cast<const T*>(a.k) + t * a.k_stride + i * 16, x.k, on);
  load_words(static_cast<const T*>(a.v) + t * a.v_stride + i * 16, x.v, on);
  return x;
}

struct Packed {
  uint2 k, v;
  uint8_t ks, vs;
};

template <typename T>
__device__ __forceinline__ Packed pack_group(const KvWriteArgs& a, const Group& x) {
  Packed p;
  p.k = kv::quantise16<T>(x.k, a.k_mul, &p.ks);
  p.v = kv::quantise16<T>(x.v, a.v_mul, &p.vs);
  return p;
}

template <int kDim>
__device__ __forceinline__ void store_group(const KvWriteArgs& a, int64_t slot, int i, const Packed& p) {
  const int h = i / (kDim / 16), grp = i % (kDim / 16), row = int(slot & 15);
  uint8_t* const rec = a.data + ((slot >> 4) * a.H + h) * kv::record_bytes(kDim);
  *reinterpret_cast<uint2*>(rec + kv::k_codes(kDim, row, 2 * grp)) = p.k;
  if constexpr (kDim == 64) {   // two chunks
    *reinterpret_cast<uint32_t*>(rec + kv::v_codes(kDim, row, 2 * grp)) = p.v.x;
    *reinterpret_cast<uint32_t*>(rec + kv::v_codes(kDim, row, 2 * grp + 1)) = p.v.y;
  } else {
    *reinterpret_cast<uint2*>(rec + kv::v_codes(kDim, row, 2 * grp)) = p.v;
  }
  rec[kv::k_scale(kDim, row, grp)] = p.ks;
  rec[kv::v_scale(kDim, row, grp)] = p.vs;
}

// One CTA per four tokens, one warp per eight groups.
template <typename T, int kDim>
__global__ void __launch_bounds__(512) kv_write_few_kernel(const KvWriteArgs a) {
  __shared__ int again;   // tokens of the four whose slot comes again
  if (threadIdx.x == 0) again = 0;
  __syncthreads();
  const int n = token_count(a.count, a.T), t0 = blockIdx.x * kQuad;
  if (t0 >= n) return;
  int64_t slots[kQuad];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kQuad; ++i) slots[i] = t0 + i < n ? a.slots[t0 + i] : -1;
  for (int u = t0 + 1 + threadIdx.x; u < n; u += blockDim.x) {
    const int64_t s = a.slots[u];
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
      if (u > t0 + i && s == slots[i]) mine |= 1 << i;
  }
  if (mine) atomicOr(&again, mine);
  __syncthreads();
  const int lane = threadIdx.x & 31, tok = lane >> 3;
  const int64_t slot = tok == 0 ? slots[0] : tok == 1 ? slots[1] : tok == 2 ? slots[2] : slots[3];
  if (slot >= a.num_slots && threadIdx.x < 32) set_status(a.status, UPF_ERR_INVALID_ARG);
  const bool on = slot >= 0 && slot < a.num_slots && !((again >> tok) & 1);
  const int groups = a.H * (kDim / 16);
  for (int w = threadIdx.x >> 5; w * 8 < groups; w += blockDim.x >> 5) {
    const int i = w * 8 + (lane & 7);
    const bool mine = on && i < groups;
    const Packed p = pack_group<T>(a, load_group<T>(a, t0 + tok, i, mine));
    if (mine) store_group<kDim>(a, slot, i, p);
  }
}

// owner[slot] = the last token with that slot, for every slot named: one cluster.
// Four tokens a thread at a time, so that a call of 32768 waits for memory twice.
__global__ void __cluster_dims__(kClaimCtas, 1, 1) __launch_bounds__(kClaimThreads) kv_claim_kernel(const KvWriteArgs a) {
  pdl_trigger();   // the writing launch may load its tokens
  constexpr int kAll = kClaimCtas * kClaimThreads, kEach = 4;
  const int n = token_count(a.count, a.T), first = blockIdx.x * kClaimThreads + threadIdx.x;
  int64_t slots[kEach];
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) slots[i] = t0 + i * kAll < n ? a.slots[t0 + i * kAll] : -1;
  };
  for (int t0 = first; t0 < n; t0 += kEach * kAll) {
    load(t0);
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (slots[i] >= 0 && slots[i] < a.num_slots) a.owner[slots[i]] = -1;
  }
  __threadfence();
  ptx::cluster_sync();
  for (int t0 = first; t0 < n; t0 += kEach * kAll) {
    if (n > kEach * kAll) load(t0);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (slots[i] >= a.num_slots) set_status(a.status, UPF_ERR_INVALID_ARG);
      else if (slots[i] >= 0) atomicMax(a.owner + slots[i], t0 + i * kAll);
    }
  }
}

// One warp per four tokens and eight groups (along the kv heads).
template <typename T, int kDim>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteArgs a) {
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * 8 + (threadIdx.x >> 5);   // under 2^32 (checked by the caller)
  const uint32_t groups = a.H * (kDim / 16), per = (groups + 7) / 8, quad = w / per, i = (w - quad * per) * 8 + (lane & 7);
  const int64_t t = (int64_t)quad * kQuad + (lane >> 3);
  const bool in = t < token_count(a.count, a.T) && i < groups;
  const int64_t slot = in ? a.slots[t] : -1;
  const bool on = slot >= 0 && slot < a.num_slots;
  const Packed p = pack_group<T>(a, load_group<T>(a, t, i, on));
  pdl_wait();   // the claims
  if (on && __ldcg(a.owner + slot) == t) store_group<kDim>(a, slot, i, p);
}

template <typename T, int kDim>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadArgs a) {
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const uint32_t runs = a.H * (kDim / 64), per = (runs + kRuns - 1) / kRuns, quad = w / per, j0 = (w - quad * per) * kRuns;
  const int64_t t = (int64_t)quad * kQuad + (lane >> 3);
  if (t >= token_count(a.count, a.T)) return;
  const int64_t slot = a.slots[t];
  const int row = int(slot & 15);
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (j0 == 0) set_status(a.status, UPF_ERR_INVALID_ARG);
    return;
  }
  const uint8_t* const base = a.data + (slot >> 4) * a.H * kv::record_bytes(kDim);
  struct {
    uint32_t k, v;
    uint8_t ks, vs;
  } p[kRuns];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    if (j0 + i >= runs) break;
    const uint8_t* const rec = base + (j0 + i) / (kDim / 64) * kv::record_bytes(kDim);
    const int oct = (j0 + i) % (kDim / 64) * 8 + (lane & 7);
    if (a.k) {
      p[i].k = *reinterpret_cast<const uint32_t*>(rec + kv::k_codes(kDim, row, oct));
      p[i].ks = rec[kv::k_scale(kDim, row, oct / 2)];
    }
    if (a.v) {
      p[i].v = *reinterpret_cast<const uint32_t*>(rec + kv::v_codes(kDim, row, oct));
      p[i].vs = rec[kv::v_scale(kDim, row, oct / 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    if (j0 + i >= runs) break;
    const int64_t at = (int64_t)(j0 + i) * 64 + (lane & 7) * 8;
    if (a.k) __stcs(reinterpret_cast<uint4*>(static_cast<T*>(a.k) + t * a.k_stride + at), kv::dequantise8<T>(p[i].k, p[i].ks, a.k_mul));
    if (a.v) __stcs(reinterpret_cast<uint4*>(static_cast<T*>(a.v) + t * a.v_stride + at), kv::dequantise8<T>(p[i].v, p[i].vs, a.v_mul));
  }
}

// Blocks of eight warps for four tokens and one `per`-th of a row each.
dim3 warp_blocks(int T, int per) { return dim3(unsigned(((int64_t)((T + kQuad - 1) / kQuad) * per + 7) / 8)); }

template <typename T, int kDim>
cudaError_t write(const KvWriteArgs& a, cudaStream_t s) {
  if (!a.owner) {
    const int warps = (a.H * (kDim / 16) + 7) / 8;
    return launch_kernel(kv_write_few_kernel<T, kDim>, (a.T + kQuad - 1) / kQuad, 32 * (warps < 16 ? warps : 16), 0, s, false, a);
  }
  const cudaError_t e = launch_kernel(kv_claim_kernel, kClaimCtas, kClaimThreads, 0, s, false, a);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv_write_kernel<T, kDim>, warp_blocks(a.T, (a.H * (kDim / 16) + 7) / 8), 256, 0, s, true, a);
}

template <typename T, int kDim>
cudaError_t read(const KvReadArgs& a, cudaStream_t s) {
  return launch_kernel(kv_read_kernel<T, kDim>, warp_blocks(a.T, (a.H * (kDim / 64) + kRuns - 1) / kRuns), 256, 0, s, false, a);
}

}  // namespace

#define UPF_BY_DIM(call, T) (a.d == 64 ? call<T, 64>(a, s) : a.d == 128 ? call<T, 128>(a, s) : call<T, 256>(a, s))

cudaError_t launch_kv_write(const KvWriteArgs& a, bool f16, cudaStream_t s) {
  return f16 ? UPF_BY_DIM(write, __half) : UPF_BY_DIM(write, __nv_bfloat16);
}

cudaError_t launch_kv_read(const KvReadArgs& a, bool f16, cudaStream_t s) {
  return f16 ? UPF_BY_DIM(read, __half) : UPF_BY_DIM(read, __nv_bfloat16);
}

#undef UPF_BY_DIM

}  // namespace upf
