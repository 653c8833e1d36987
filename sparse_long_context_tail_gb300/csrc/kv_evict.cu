// Eviction of cache entries by accumulated attention weight.
//
// Two launches.  The first finds each request's kept entries: the first `sinks`, the last
// `recent`, and of those between the heaviest, as many as the budget leaves; weights are not
// negative, so their bit patterns are ordered as they are, and the least kept weight is
// found digit by digit (11, 10 and 10 bits) from histograms, one cluster of CTAs a request.
// Of entries as heavy as it the first ones are kept.  Each CTA then lists the kept ones of its
// run of entries, in order.
//
// The second moves them together.  Entry j of the result was entry s_j >= j, so chunks of
// places written in ascending order never overwrite what a later chunk has yet to read.  To run
// them at the same time, a CTA reads its whole chunk (64 entries of one kv head) into shared memory, says so, and
// writes once the chunks have been read whose entries lie in its places: the entries in 64 places go to
// 64 places in a row at most, which two chunks hold.  Chunks are taken by ticket, so those that
// a CTA waits for have been taken before by CTAs that wait for nothing to read them.
#include <algorithm>
#include <type_traits>

#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {

struct KvEvictPlan {
  int32_t n, left;    // entries before and after
  int32_t move;       // 1: some are to be moved or copied
  int32_t pad;
};

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kChunk = 64;            // places of a moving CTA
constexpr int kMoveThreads = 128;

__host__ __device__ constexpr int64_t chunks_of(int64_t places) { return (places + kChunk - 1) / kChunk; }

// The slot of entry e of a table row, or -1 if its page is bad.
__device__ __forceinline__ int64_t slot_of(const int32_t* row, int e, int shift, int64_t num_slots) {
  const int page = row[e >> shift];
  const int64_t slot = ((int64_t)page << shift) + (e & ((1 << shift) - 1));
  return page >= 0 && slot < num_slots ? slot : -1;
}

__device__ __forceinline__ int32_t ld_cluster(const int32_t* mine, uint32_t rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::mapa_shared(ptx::smem_u32(mine), rank)) : "memory");
  return v;
}

// Sum over the CTA's threads, for all of them.
__device__ __forceinline__ int block_sum(int v, int* scratch) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) all += scratch[w];
  return all;
}

// Sum over the threads before this one; `all`: over all.
__device__ __forceinline__ int block_scan(int v, int* scratch, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  const int s = scratch[lane];
  int t = s;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, t, d);
    if (lane >= d) t += y;
  }
  all = __shfl_sync(0xFFFFFFFFu, t, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, t - s, warp);
  return before + x - v;
}
static_assert(kSelWarps == 32, "a warp scans the warps' sums");

__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(const KvEvictArgs a, const uint32_t ctas) {
  __shared__ int32_t hist[kBins];
  __shared__ int32_t scratch[32], said[4], counts[2];
  const uint32_t rank = blockIdx.x % ctas;   // in the request's cluster
  const int r = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31;
  const int n = a.kv_len[r];
  const float* const w = a.w + r * a.w_stride;
  const int32_t* const row = a.table + r * a.table_stride;
  const int32_t* const row_out = a.table_out ? a.table_out + r * a.table_out_stride : row;
  if (tid < 4) said[tid] = 0;
  if (r == 0 && rank == 0 && tid == 0) *a.ticket = 0;
  __syncthreads();

  // ---- is there anything to do, and can it be done?
  const int page = 1 << a.page_shift;
  bool fine = n >= 0 && n <= ((int64_t)a.max_pages << a.page_shift) && n <= a.w_cols;
  const bool cut = fine && n > a.trigger;
  const int left = cut ? a.budget : n;
  const bool move = cut || a.table_out || a.w_out != a.w;
  if (fine && move) {
    fine = left <= a.w_out_cols && (!a.table_out || left <= ((int64_t)a.max_pages_out << a.page_shift));
    int bad = 0;
    if (fine && (cut || a.table_out)) {
      for (int p = rank * kSelThreads + tid; p < (n + page - 1) / page; p += ctas * kSelThreads)
        bad |= slot_of(row, p << a.page_shift, a.page_shift, a.num_slots) < 0;
      if (a.table_out)
        for (int p = rank * kSelThreads + tid; p < (left + page - 1) / page; p += ctas * kSelThreads)
          bad |= slot_of(row_out, p << a.page_shift, a.page_shift, a.num_slots) < 0;
    }
    if (cut)
      for (int e = rank * kSelThreads + tid; e < n; e += ctas * kSelThreads) {
        const float x = w[e];
        if (!(x >= 0.f && x < INFINITY)) bad |= 2;
      }
    if (bad) atomicOr(&said[0], bad);
  }
  if (ctas > 1) ptx::cluster_sync();
  else __syncthreads();
  int bad = 0;
  for (uint32_t c = 0; c < ctas; ++c) bad |= ctas > 1 ? ld_cluster(&said[0], c) : said[0];
  if (!fine || bad) {
    if (tid == 0 && rank == 0) set_status(a.status, !fine || (bad & 1) ? UPF_ERR_INVALID_ARG : UPF_ERR_NONFINITE);
    fine = false;
  }
  if (ctas > 1) ptx::cluster_sync();   // every CTA has read the others' words
  if (!fine || !cut) {
    const int now = fine ? left : a.table_out ? 0 : n;
    if (rank == 0 && tid == 0) {
      a.plan[r] = KvEvictPlan{n, now, fine && move ? 1 : 0, 0};
      a.len_out[r] = now;
    }
    for (int j = rank * kSelThreads + tid; j < a.budget; j += ctas * kSelThreads)
      if (a.kept) a.kept[r * a.kept_stride + j] = fine && j < left ? j : -1;
    if (fine && move) {
      for (int j = rank * kSelThreads + tid; j < left; j += ctas * kSelThreads) {
        a.list[(int64_t)r * a.cap + j] = j;
        a.list_w[(int64_t)r * a.cap + j] = w[j];
      }
    }
  } else {
    // ---- the least kept weight among entries [sinks, sinks + middle)
    const int middle = n - a.sinks - a.recent, want = a.budget - a.sinks - a.recent;
    const float* const m = w + a.sinks;
    const int each = (middle + ctas - 1) / ctas, from = min(middle, int(rank) * each), to = min(middle, from + each);
    // bits of a weight; -0 is 0
    auto key_of = [&](int i) { return __float_as_uint(m[i]) & 0x7FFFFFFFu; };
    uint32_t least = 0;      // its bits, as far as they are known
    int need = want;         // how many of the entries that agree with them are kept
    if (want > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0, bits = pass == 0 ? 11 : 10, bins = 1 << bits;
        for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i0 = from; i0 < to; i0 += kSelThreads) {
          const int i = i0 + tid;
          const uint32_t key = i < to ? key_of(i) : 0;
          const bool on = i < to && (pass == 0 || (key >> (shift + bits)) == (least >> (shift + bits)));
          // weights of a request share few digits: one addition for all lanes with the same one
          const int digit = on ? int(key >> shift & (bins - 1)) : -1;
          const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
          if (on && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
        }
        if (ctas > 1) ptx::cluster_sync();
        else __syncthreads();
        // thread t: the bins bins - 1 - 2 t and, below it, bins - 2 - 2 t (from the heaviest on)
        int c[2] = {0, 0};
        const int top = bins - 1 - 2 * tid;
        if (top > 0)
          for (uint32_t k = 0; k < ctas; ++k) {
            c[0] += ctas > 1 ? ld_cluster(&hist[top], k) : hist[top];
            c[1] += ctas > 1 ? ld_cluster(&hist[top - 1], k) : hist[top - 1];
          }
        int all;
        const int before = block_scan(c[0] + c[1], scratch, all);
        if (top > 0 && before < need && before + c[0] + c[1] >= need) {
          const bool second = before + c[0] < need;
          said[1] = second ? top - 1 : top;
          said[2] = need - before - (second ? c[0] : 0);
        }
        if (ctas > 1) ptx::cluster_sync();   // no CTA reads these bins any more
        else __syncthreads();
        least |= uint32_t(said[1]) << shift;
        need = said[2];
        __syncthreads();
      }
    } else {
      least = 0x7FFFFFFFu;   // above every weight
    }
    // ---- entries above it and as heavy before this CTA's run
    int above = 0, equal = 0;
    for (int i = from + tid; i < to; i += kSelThreads) {
      const uint32_t key = key_of(i);
      above += key > least;
      equal += key == least;
    }
    above = block_sum(above, scratch);
    equal = block_sum(equal, scratch);
    if (tid == 0) {
      counts[0] = above;
      counts[1] = equal;
    }
    above = equal = 0;
    if (ctas > 1) {
      ptx::cluster_sync();
      for (uint32_t c = 0; c < rank; ++c) {
        above += ld_cluster(&counts[0], c);
        equal += ld_cluster(&counts[1], c);
      }
      ptx::cluster_sync();   // no CTA leaves while others read its words
    }
    // ---- the list
    int32_t* const list = a.list + (int64_t)r * a.cap;
    float* const list_w = a.list_w + (int64_t)r * a.cap;
    auto put = [&](int j, int e) {
      list[j] = e;
      list_w[j] = w[e];
      if (a.kept) a.kept[r * a.kept_stride + j] = e;
    };
    for (int i0 = from; i0 < to; i0 += kSelThreads) {
      const int i = i0 + tid;
      const uint32_t key = i < to ? key_of(i) : 0;
      const bool more = i < to && key > least, same = i < to && key == least;
      int all;
      const int before = block_scan(int(more) << 16 | int(same), scratch, all);
      const int rank_same = equal + (before & 0xFFFF);
      if (more || (same && rank_same < need)) put(a.sinks + above + (before >> 16) + min(rank_same, need), a.sinks + i);
      above += all >> 16;
      equal += all & 0xFFFF;
    }
    for (int j = rank * kSelThreads + tid; j < a.sinks + a.recent; j += ctas * kSelThreads)
      put(j < a.sinks ? j : j + want, j < a.sinks ? j : j - a.sinks + n - a.recent);
    if (rank == 0 && tid == 0) {
      a.plan[r] = KvEvictPlan{n, left, 1, 0};
      a.len_out[r] = left;
    }
  }
  // the second launch's marks
  const int64_t marks = a.H * chunks_of(a.cap);
  for (int64_t i = rank * kSelThreads + tid; i < marks; i += ctas * kSelThreads) a.read[r * marks + i] = 0;
}

// First place of list[0 .. n) (ascending) whose entry is at or above e, by a warp.
__device__ __forceinline__ int first_at(const int32_t* list, int n, int e) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;        // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int below = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && __ldg(list + at) < e));   // of the probes
    if (below == 0) return lo;
    lo += (below - 1) * step + 1;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

__device__ __forceinline__ int32_t load_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(int32_t* p, int32_t v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <int kDim>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const KvEvictArgs a, const int64_t units) {
  constexpr int kRecord = kv::record_bytes(kDim), kD = kv::part_dims(kDim), kParts = kDim / kD, kC = kD / 16;
  constexpr int kRecords = kChunk / 16;
  __shared__ __align__(128) uint8_t rec[kRecords * kRecord];
  __shared__ int64_t from[kChunk];       // slots of the entries
  __shared__ int32_t said[4];
  const int tid = threadIdx.x;
  const int64_t per_head = chunks_of(a.cap);
  if (tid == 0) said[0] = atomicAdd(a.ticket, 1);
  __syncthreads();
  // ticket -> chunk first, so that tickets of one request and head ascend with the chunk
  const int64_t u = said[0];
  if (u >= units) return;
  const int per = a.R * a.H, c = int(u / per), rh = int(u - (int64_t)c * per), r = rh / a.H, h = rh - r * a.H;
  const KvEvictPlan plan = a.plan[r];
  if (!plan.move) return;
  const int j0 = c * kChunk, places = min(kChunk, plan.left - j0);
  const int32_t* const list = a.list + (int64_t)r * a.cap;
  // ---- weights: this chunk's, and this chunk's share of the places that fall free
  if (h == 0) {
    float* const w = a.w_out + r * a.w_out_stride;
    if (tid < places) w[j0 + tid] = a.list_w[(int64_t)r * a.cap + j0 + tid];
    const int end = min(plan.n, a.w_out_cols), chunks = max(1, int(chunks_of(plan.left)));
    if (c < chunks)
      for (int64_t e = plan.left + (int64_t)c * kMoveThreads + tid; e < end; e += (int64_t)chunks * kMoveThreads) w[e] = 0.f;
  }
  if (places <= 0) return;
  int32_t* const mark = a.read + ((int64_t)r * a.H + h) * per_head;
  const bool in_place = !a.table_out || a.table_out == a.table;
  // ---- nothing to do where all entries stay where they are
  const bool stays = in_place && __ldg(list + j0 + places - 1) == j0 + places - 1;
  if (stays) {   // then list[j] = j up to here
    if (tid == 0) store_release(mark + c, 1);
    return;
  }
  if (tid < 64) {   // which of the entries kept are in this chunk's places now
    const int at = first_at(list, plan.left, tid < 32 ? j0 : j0 + kChunk);
    if ((tid & 31) == 0) said[2 + tid / 32] = at;
  }
  const int32_t* const row = a.table + r * a.table_stride;
  const int32_t* const row_out = a.table_out ? a.table_out + r * a.table_out_stride : row;
  if (tid < places) from[tid] = slot_of(row, __ldg(list + j0 + tid), a.page_shift, a.num_slots);
  __syncthreads();
  auto record_of = [&](int64_t slot) { return a.data + ((slot >> 4) * a.H + h) * (int64_t)kRecord; };
  // ---- the record that the request ends in keeps its other rows
  const int whole = (places + 15) / 16;
  if (places & 15) {
    const int64_t slot = slot_of(row_out, j0 + (whole - 1) * 16, a.page_shift, a.num_slots);
    const uint4* const src = reinterpret_cast<const uint4*>(record_of(slot));
    for (int i = tid; i < kRecord / 16; i += kMoveThreads) reinterpret_cast<uint4*>(rec + (whole - 1) * kRecord)[i] = src[i];
    __syncthreads();
  }
  // ---- read: rows side by side are likely to come from rows side by side
  constexpr int kKeyVecs = kD / 32;    // 16-byte vectors of a row's keys in a part
  for (int i = tid; i < places * kParts * kKeyVecs; i += kMoveThreads) {
    const int j = i / (kParts * kKeyVecs), v = i % (kParts * kKeyVecs), p = v / kKeyVecs, x = v % kKeyVecs;
    const int at = p * 8 * kD + x * 16, row_b = kD / 2;
    *reinterpret_cast<uint4*>(rec + (j >> 4) * kRecord + at + (j & 15) * row_b) =
        *reinterpret_cast<const uint4*>(record_of(from[j]) + at + int(from[j] & 15) * row_b);
  }
  using Piece = typename std::conditional<kC == 8, uint2, uint32_t>::type;   // a row's codes of a chunk of the values
  for (int i = tid; i < kChunk * kParts * 8; i += kMoveThreads) {
    const int j = i % kChunk, x = i / kChunk, p = x / 8, y = x % 8;
    if (j >= places) continue;
    auto at = [&](int s) { return 8 * kDim + p * 8 * kD + (s >> 3) * 4 * kD + y * 8 * kC + (s & 7) * kC; };
    *reinterpret_cast<Piece*>(rec + (j >> 4) * kRecord + at(j & 15)) =
        *reinterpret_cast<const Piece*>(record_of(from[j]) + at(int(from[j] & 15)));
  }
  constexpr int kGroups = kDim / 16;
  for (int i = tid; i < places * (kGroups / 4); i += kMoveThreads) {
    const int j = i / (kGroups / 4), x = i % (kGroups / 4) * 4;
    *reinterpret_cast<uint32_t*>(rec + (j >> 4) * kRecord + kv::k_scale(kDim, j & 15, x)) =
        *reinterpret_cast<const uint32_t*>(record_of(from[j]) + kv::k_scale(kDim, int(from[j] & 15), x));
  }
  for (int i = tid; i < kChunk * kGroups; i += kMoveThreads) {
    const int j = i % kChunk, x = i / kChunk;
    if (j >= places) continue;
    rec[(j >> 4) * kRecord + kv::v_scale(kDim, j & 15, x)] = record_of(from[j])[kv::v_scale(kDim, int(from[j] & 15), x)];
  }
  // ---- say so, and wait until the entries in these places have been read
  __syncthreads();
  if (tid == 0) {
    store_release(mark + c, 1);
    const int lo = said[2], hi = said[3];
    bool ok = true;
    const long long t0 = clock64();
    for (int k = lo / kChunk; lo < hi && k <= (hi - 1) / kChunk && k < c && ok; ++k)
      while (ok && load_acquire(mark + k) == 0) ok = clock64() - t0 < a.wait_limit;
    if (!ok) set_status(a.status, UPF_ERR_TIMEOUT);
    said[1] = ok;
  }
  __syncthreads();
  if (!said[1]) return;
  for (int k = 0; k < whole; ++k) {
    const int64_t slot = slot_of(row_out, j0 + k * 16, a.page_shift, a.num_slots);
    uint4* const dst = reinterpret_cast<uint4*>(record_of(slot));
    for (int i = tid; i < kRecord / 16; i += kMoveThreads) dst[i] = reinterpret_cast<const uint4*>(rec + k * kRecord)[i];
  }
}

// CTAs of a request's cluster.
int cluster_of(const KvEvictArgs& a) {
  const int64_t most = std::min<int64_t>((int64_t)a.max_pages << a.page_shift, a.w_cols);
  int c = 1;
  while (c < kMaxCluster && most > (int64_t)c * 8192) c *= 2;
  return c;
}

}  // namespace

size_t kv_evict_workspace(KvEvictArgs& a, void* ws) {
  const int64_t places = std::min<int64_t>((int64_t)a.max_pages << a.page_shift, a.trigger);
  a.cap = int(places);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void* const p = static_cast<char*>(ws) + (ws ? off : 0);
    off = (off + bytes + 255) & ~size_t(255);
    return p;
  };
  a.plan = static_cast<KvEvictPlan*>(take(sizeof(KvEvictPlan) * a.R));
  a.ticket = static_cast<int32_t*>(take(sizeof(int32_t)));
  a.list = static_cast<int32_t*>(take(sizeof(int32_t) * a.R * a.cap));
  a.list_w = static_cast<float*>(take(sizeof(float) * a.R * a.cap));
  a.read = static_cast<int32_t*>(take(sizeof(int32_t) * a.R * a.H * chunks_of(a.cap)));
  return off;
}

cudaError_t launch_kv_evict(const KvEvictArgs& a, cudaStream_t s) {
  const int ctas = cluster_of(a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas) * unsigned(a.R));
  cfg.blockDim = kSelThreads;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_select_kernel, a, uint32_t(ctas));
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.R * a.H * chunks_of(a.cap);
  const dim3 grid = dim3(unsigned(units));
  return a.d == 64    ? launch_kernel(kv_evict_move_kernel<64>, grid, kMoveThreads, 0, s, false, a, units)
         : a.d == 128 ? launch_kernel(kv_evict_move_kernel<128>, grid, kMoveThreads, 0, s, false, a, units)
                      : launch_kernel(kv_evict_move_kernel<256>, grid, kMoveThreads, 0, s, false, a, units);
}

}  // namespace upf
