// Writing tokens' keys and values into the 4-bit cache and reading them back.
//
// One thread handles one group (16 dims: 32 bytes of input, 9 bytes of cache),
// so the group's largest magnitude and its 16 roundings need no exchange between
// threads.
//
// A slot given twice in one call takes the later token's values, as if the
// tokens were written in order: without a rule the two tokens' groups could mix.
// Short calls look for a later token with the same slot; longer ones claim
// their slots first (owner[slot] = the latest token), in two small launches
// whose cost goes with the tokens, not with the size of the cache.
#include "kv_layout.cuh"
#include "upf_internal.cuh"

namespace upf {

namespace {

__device__ __forceinline__ int token_count(const int32_t* count, int T) {
  return count ? min(max(*count, 0), T) : T;
}

template <typename T>
__device__ __forceinline__ void write_group(const KvWriteArgs& a, int64_t slot, const T* src, int h, int grp, bool values) {
  uint32_t w[8];
  const uint4 lo = *reinterpret_cast<const uint4*>(src), hi = *reinterpret_cast<const uint4*>(src + 8);
  w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
  w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
  uint8_t scale;
  const uint2 codes = kv::quantise16<T>(w, values ? a.v_mul : a.k_mul, &scale);
  uint8_t* rec = a.data + ((slot >> 4) * a.H + h) * kv::record_bytes(a.d);
  const int row = int(slot & 15);
  if (!values) {
    *reinterpret_cast<uint2*>(rec + kv::k_codes(a.d, row, grp)) = codes;
    rec[kv::k_scale(a.d, row, grp)] = scale;
  } else {
    uint8_t* p = rec + kv::v_codes(a.d, row, grp);
    if (a.d == 64) {
      *reinterpret_cast<uint32_t*>(p) = codes.x;
      *reinterpret_cast<uint32_t*>(p + kv::v_chunk_stride(64)) = codes.y;
    } else {
      *reinterpret_cast<uint2*>(p) = codes;
    }
    rec[kv::v_scale(a.d, row, grp)] = scale;
  }
}

// One CTA per token.
template <typename T>
__global__ void __launch_bounds__(256) kv_write_few_kernel(const KvWriteArgs a) {
  const int n = token_count(a.count, a.T), t = blockIdx.x;
  if (t >= n) return;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0) set_status(a.status, UPF_ERR_INVALID_ARG);
    return;
  }
  int again = 0;
  for (int u = t + 1 + threadIdx.x; u < n; u += blockDim.x) again |= a.slots[u] == slot;
  if (__syncthreads_or(again)) return;
  const int groups = a.H * (a.d / 16);
  for (int i = threadIdx.x; i < 2 * groups; i += blockDim.x) {
    const bool values = i >= groups;
    const int j = values ? i - groups : i;
    const T* src = static_cast<const T*>(values ? a.v : a.k) + (int64_t)t * (values ? a.v_stride : a.k_stride) + j * 16;
    write_group<T>(a, slot, src, j / (a.d / 16), j % (a.d / 16), values);
  }
}

__global__ void __launch_bounds__(256) kv_owner_clear_kernel(const KvWriteArgs a) {
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= token_count(a.count, a.T)) return;
  const int64_t slot = a.slots[t];
  if (slot >= 0 && slot < a.num_slots) a.owner[slot] = -1;
}

__global__ void __launch_bounds__(256) kv_owner_claim_kernel(const KvWriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= token_count(a.count, a.T)) return;
  const int64_t slot = a.slots[t];
  if (slot >= a.num_slots) set_status(a.status, UPF_ERR_INVALID_ARG);
  else if (slot >= 0) atomicMax(a.owner + slot, t);
}

// One thread per (token, kv head, group), keys and values.
template <typename T>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int groups = a.H * (a.d / 16);
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t t = i / groups;
  const int j = int(i % groups);
  if (t >= token_count(a.count, a.T)) return;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots || a.owner[slot] != t) return;
  write_group<T>(a, slot, static_cast<const T*>(a.k) + t * a.k_stride + j * 16, j / (a.d / 16), j % (a.d / 16), false);
  write_group<T>(a, slot, static_cast<const T*>(a.v) + t * a.v_stride + j * 16, j / (a.d / 16), j % (a.d / 16), true);
}

template <typename T>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadArgs a) {
  const int groups = a.H * (a.d / 16);
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t t = i / groups;
  const int j = int(i % groups);
  if (t >= token_count(a.count, a.T)) return;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (j == 0) set_status(a.status, UPF_ERR_INVALID_ARG);
    return;
  }
  const int h = j / (a.d / 16), grp = j % (a.d / 16), row = int(slot & 15);
  const uint8_t* rec = a.data + ((slot >> 4) * a.H + h) * kv::record_bytes(a.d);
  uint32_t w[8];
  if (a.k) {
    const uint2 codes = *reinterpret_cast<const uint2*>(rec + kv::k_codes(a.d, row, grp));
    kv::dequantise16<T>(codes, rec[kv::k_scale(a.d, row, grp)], a.k_mul, w);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.k) + t * a.k_stride + j * 16);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  if (a.v) {
    const uint8_t* p = rec + kv::v_codes(a.d, row, grp);
    uint2 codes;
    if (a.d == 64) {
      codes.x = *reinterpret_cast<const uint32_t*>(p);
      codes.y = *reinterpret_cast<const uint32_t*>(p + kv::v_chunk_stride(64));
    } else {
      codes = *reinterpret_cast<const uint2*>(p);
    }
    kv::dequantise16<T>(codes, rec[kv::v_scale(a.d, row, grp)], a.v_mul, w);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.v) + t * a.v_stride + j * 16);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, bool f16, cudaStream_t s) {
  cudaError_t e;
  if (!a.owner) {
    const int groups = 2 * a.H * (a.d / 16);
    const int threads = groups >= 256 ? 256 : (groups + 31) / 32 * 32;
    return f16 ? launch_kernel(kv_write_few_kernel<__half>, a.T, threads, 0, s, false, a)
               : launch_kernel(kv_write_few_kernel<__nv_bfloat16>, a.T, threads, 0, s, false, a);
  }
  const int tb = (a.T + 255) / 256;
  if ((e = launch_kernel(kv_owner_clear_kernel, tb, 256, 0, s, false, a)) != cudaSuccess) return e;
  if ((e = launch_kernel(kv_owner_claim_kernel, tb, 256, 0, s, true, a)) != cudaSuccess) return e;
  const int64_t blocks = ((int64_t)a.T * a.H * (a.d / 16) + 255) / 256;
  return f16 ? launch_kernel(kv_write_kernel<__half>, dim3(unsigned(blocks)), 256, 0, s, true, a)
             : launch_kernel(kv_write_kernel<__nv_bfloat16>, dim3(unsigned(blocks)), 256, 0, s, true, a);
}

cudaError_t launch_kv_read(const KvReadArgs& a, bool f16, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.T * a.H * (a.d / 16) + 255) / 256;
  return f16 ? launch_kernel(kv_read_kernel<__half>, dim3(unsigned(blocks)), 256, 0, s, false, a)
             : launch_kernel(kv_read_kernel<__nv_bfloat16>, dim3(unsigned(blocks)), 256, 0, s, false, a);
}

}  // namespace upf
