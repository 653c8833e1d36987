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

// Sum over the threads before this one.
__device__ __forceinline__ int block_scan(int v, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  const int s = scratch[lane];
  int t = s;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, t, d);
    if (lane >= d) t += y;
  }
  return __shfl_sync(0xFFFFFFFFu, t - s, warp) + x - v;
}
static_assert(kSelWarps == 32, "a warp scans the warps' sums");

// A cluster of `ctas` CTAs a request.  A warp has a run of entries of its own, 32 at a time, the first
// kHeld times in registers through all passes (131072 entries of a request; of more, the rest is read again).
__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(const KvEvictArgs a, const uint32_t ctas) {
  constexpr int kHeld = 16, kPasses = 3;
  __shared__ int32_t hist[kPasses][kBins];
  __shared__ int32_t scratch[kPasses][32], found[kPasses][2], bad_here, counts[2], warp_counts[kSelWarps][2];
  const uint32_t rank = blockIdx.x % ctas;   // in the request's cluster
  const int r = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = rank * kSelThreads + tid, stride = ctas * kSelThreads;   // of the cluster's threads
  auto sync = [&] {
    if (ctas > 1) ptx::cluster_sync();
    else __syncthreads();
  };
  auto of_cta = [&](const int32_t* mine, uint32_t c) { return ctas > 1 ? ld_cluster(mine, c) : *mine; };
  const int n = a.kv_len[r];
  const float* const w = a.w + r * a.w_stride;
  const int32_t* const row = a.table + r * a.table_stride;
  for (int i = tid; i < kPasses * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  if (tid == 0) bad_here = 0;
  pdl_trigger();
  // the second launch's ticket and marks
  if (r == 0 && first == 0) *a.ticket = 0;
  const int64_t marks = a.H * chunks_of(a.cap);
  for (int64_t i = first; i < marks; i += stride) a.read[r * marks + i] = 0;

  // ---- is there anything to do, and can it be done?
  bool fine = n >= 0 && n <= ((int64_t)a.max_pages << a.page_shift) && n <= a.w_cols;
  const bool cut = fine && n > a.trigger;
  const int left = cut ? a.budget : n;
  const bool move = cut || a.table_out || a.w_out != a.w;
  if (move) fine = fine && left <= a.w_out_cols && (!a.table_out || left <= ((int64_t)a.max_pages_out << a.page_shift));

  // ---- the weights between the ends
  const int middle = n - a.sinks - a.recent, want = a.budget - a.sinks - a.recent;
  const float* const m = w + a.sinks;
  const int runs = cut ? (middle + 32 * kSelWarps * int(ctas) - 1) / (32 * kSelWarps * int(ctas)) : 0;   // of 32 entries, a warp
  const int from = (rank * kSelWarps + warp) * runs * 32 + lane;    // under 2^30 + 2^15
  uint32_t held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = k < runs && from + 32 * k < middle ? __float_as_uint(m[from + 32 * k]) : 0u;
  // f(k, bits): entry from + 32 k of the middle, where there is one (`there`)
  auto each = [&](auto&& f) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (k < runs) f(k, held[k], from + 32 * k < middle);
    for (int k = kHeld; k < runs; ++k) {
      const bool there = from + 32 * k < middle;
      f(k, there ? __float_as_uint(m[from + 32 * k]) : 0u, there);
    }
  };
  // Of a weight's bits: the order of weights.  -0 is 0.
  constexpr uint32_t kMagnitude = 0x7FFFFFFFu, kInfinity = 0x7F800000u;
  auto is_bad = [&](uint32_t bits) { return (bits & kMagnitude) >= kInfinity || bits > 0x80000000u; };
  // One to the bin of each entry whose upper bits are those of `least`.
  auto count = [&](int pass, uint32_t least) {
    const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0, bits = pass == 0 ? 11 : 10;
    each([&](int, uint32_t raw, bool there) {
      const uint32_t key = raw & kMagnitude;
      const bool on = there && (pass == 0 || (key >> (shift + bits)) == (least >> (shift + bits)));
      const int digit = on ? int(key >> shift & ((1u << bits) - 1)) : -1;
      // equal digits of a warp wait for one another: those of zeros, and of warps with one digit, go together
      const uint32_t zeros = __ballot_sync(0xFFFFFFFFu, on && key == 0);
      if (__all_sync(0xFFFFFFFFu, digit == __shfl_sync(0xFFFFFFFFu, digit, 0))) {
        if (lane == 0 && on) atomicAdd(&hist[pass][digit], 32);
      } else {
        if (lane == 0 && zeros) atomicAdd(&hist[pass][0], __popc(zeros));
        if (on && key != 0) atomicAdd(&hist[pass][digit], 1);
      }
    });
  };
  __syncthreads();
  if (fine) {
    const int page = 1 << a.page_shift;
    int bad = 0;
    if (cut || a.table_out)
      for (int p = first; p < (n + page - 1) / page; p += stride) bad |= slot_of(row, p << a.page_shift, a.page_shift, a.num_slots) < 0;
    if (a.table_out)
      for (int p = first; p < (left + page - 1) / page; p += stride)
        bad |= slot_of(a.table_out + r * a.table_out_stride, p << a.page_shift, a.page_shift, a.num_slots) < 0;
    if (cut) {
      for (int e = first; e < a.sinks + a.recent; e += stride)
        if (is_bad(__float_as_uint(w[e < a.sinks ? e : e + middle]))) bad |= 2;
      each([&](int, uint32_t raw, bool) {
        if (is_bad(raw)) bad |= 2;
      });
      if (want > 0) count(0, 0);
    }
    if (bad) atomicOr(&bad_here, bad);
  }
  sync();
  int bad = 0;
  for (uint32_t c = 0; c < ctas; ++c) bad |= of_cta(&bad_here, c);
  if (!fine || bad) {
    if (first == 0) set_status(a.status, !fine || (bad & 1) ? UPF_ERR_INVALID_ARG : UPF_ERR_NONFINITE);
    fine = false;
  }
  int32_t* const list = a.list + (int64_t)r * a.cap;
  float* const list_w = a.list_w + (int64_t)r * a.cap;
  int32_t* const kept = a.kept ? a.kept + r * a.kept_stride : nullptr;
  if (!fine || !cut) {
    const int now = fine ? left : a.table_out ? 0 : n;
    if (first == 0) {
      a.plan[r] = KvEvictPlan{n, now, fine && move ? 1 : 0, 0};
      a.len_out[r] = now;
    }
    for (int j = first; kept && j < a.budget; j += stride) kept[j] = fine && j < left ? j : -1;
    for (int j = first; fine && move && j < left; j += stride) {
      list[j] = j;
      list_w[j] = w[j];
    }
    sync();   // no CTA leaves while others read its words
    return;
  }
  // ---- the least kept weight
  uint32_t least = kMagnitude;   // its bits, as far as they are known; none to be kept: above every weight
  int need = 0;                  // how many of the entries as heavy as it are kept
  if (want > 0) {
    least = 0;
    need = want;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0, bins = pass == 0 ? 2048 : 1024;
      if (pass > 0) {
        count(pass, least);
        sync();
      }
      // thread t: bin bins - 1 - 2 t and the one below it (from the heaviest on)
      const int top = bins - 1 - 2 * tid;
      int c[2] = {0, 0};
      if (top > 0)
        for (uint32_t k = 0; k < ctas; ++k) {
          c[0] += of_cta(&hist[pass][top], k);
          c[1] += of_cta(&hist[pass][top - 1], k);
        }
      const int before = block_scan(c[0] + c[1], scratch[pass]);
      if (top > 0 && before < need && before + c[0] + c[1] >= need) {
        const bool second = before + c[0] < need;
        found[pass][0] = second ? top - 1 : top;
        found[pass][1] = need - before - (second ? c[0] : 0);
      }
      __syncthreads();
      least |= uint32_t(found[pass][0]) << shift;
      need = found[pass][1];
    }
  }
  // ---- entries above it and as heavy: before this warp, before this CTA
  int above = 0, equal = 0;
  each([&](int, uint32_t raw, bool there) {
    const uint32_t key = raw & kMagnitude;
    above += __popc(__ballot_sync(0xFFFFFFFFu, there && key > least));
    equal += __popc(__ballot_sync(0xFFFFFFFFu, there && key == least));
  });
  if (lane == 0) {
    warp_counts[warp][0] = above;
    warp_counts[warp][1] = equal;
  }
  __syncthreads();
  {
    const int x = warp_counts[lane][0], y = warp_counts[lane][1];
    above = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? x : 0);
    equal = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? y : 0);
    if (warp == 0) {
      const int all_x = __reduce_add_sync(0xFFFFFFFFu, x), all_y = __reduce_add_sync(0xFFFFFFFFu, y);
      if (lane == 0) {
        counts[0] = all_x;
        counts[1] = all_y;
      }
    }
  }
  if (ctas > 1) {
    ptx::cluster_sync();
    for (uint32_t c = 0; c < rank; ++c) {
      above += ld_cluster(&counts[0], c);
      equal += ld_cluster(&counts[1], c);
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");   // this CTA has read the others' words
  }
  // ---- the list
  auto put = [&](int j, int e, float x) {
    list[j] = e;
    list_w[j] = x;
    if (kept) kept[j] = e;
  };
  const uint32_t before_lane = (1u << lane) - 1;
  each([&](int k, uint32_t raw, bool there) {
    const uint32_t key = raw & kMagnitude;
    const uint32_t more = __ballot_sync(0xFFFFFFFFu, there && key > least), same = __ballot_sync(0xFFFFFFFFu, there && key == least);
    const int rank_same = equal + __popc(same & before_lane);
    if (there && (key > least || (key == least && rank_same < need)))
      put(a.sinks + above + __popc(more & before_lane) + min(rank_same, need), a.sinks + from + 32 * k, __uint_as_float(raw));
    above += __popc(more);
    equal += __popc(same);
  });
  for (int j = first; j < a.sinks + a.recent; j += stride) {
    const int e = j < a.sinks ? j : j + middle;
    put(j < a.sinks ? j : j + want, e, w[e]);
  }
  if (first == 0) {
    a.plan[r] = KvEvictPlan{n, left, 1, 0};
    a.len_out[r] = left;
  }
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");   // no CTA leaves while others read its words
}

// First place of list[0 .. n) (ascending) whose entry is at or above e, by a warp.
__device__ __forceinline__ int first_at(const int32_t* list, int n, int e) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;        // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int below = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && list[at] < e));   // of the probes
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

__device__ __forceinline__ void copy_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}

template <int kDim>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const KvEvictArgs a, const int64_t units) {
  constexpr int kRecord = kv::record_bytes(kDim), kD = kv::part_dims(kDim), kParts = kDim / kD, kC = kD / 16;
  constexpr int kRecords = kChunk / 16, kGroups = kDim / 16;
  __shared__ __align__(128) uint8_t rec[kRecords * kRecord];
  __shared__ const uint8_t* base[kChunk];   // records of the entries
  __shared__ uint8_t old_row[kChunk];       // and their rows in them
  __shared__ uint8_t* place[kRecords];      // records of the places
  __shared__ int32_t said[4];
  const int tid = threadIdx.x;
  const int64_t per_head = chunks_of(a.cap);
  pdl_wait();
  if (tid == 0) said[0] = atomicAdd(a.ticket, 1);
  __syncthreads();
  // ticket -> chunk first, so that tickets of one request and head ascend with the chunk
  const uint32_t u = said[0], per = a.R * a.H;
  if (u >= units) return;
  const int c = int(u / per), rh = int(u - c * per), r = rh / a.H, h = rh - r * a.H;
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
  // ---- nothing to do where all entries stay where they are: then list[j] = j up to here
  const bool in_place = !a.table_out || a.table_out == a.table;
  if (in_place && list[j0 + places - 1] == j0 + places - 1) {
    if (tid == 0) store_release(mark + c, 1);
    return;
  }
  auto record_of = [&](int64_t slot) { return a.data + ((slot >> 4) * a.H + h) * (int64_t)kRecord; };
  const int whole = (places + 15) / 16;
  if (tid < places) {
    const int64_t slot = slot_of(a.table + r * a.table_stride, list[j0 + tid], a.page_shift, a.num_slots);
    base[tid] = record_of(slot);
    old_row[tid] = uint8_t(slot & 15);
  }
  if (tid >= 64 && tid < 64 + whole)
    place[tid - 64] = record_of(slot_of(a.table_out ? a.table_out + r * a.table_out_stride : a.table + r * a.table_stride,
                                        j0 + (tid - 64) * 16, a.page_shift, a.num_slots));
  __syncthreads();
  // ---- read.  V scales are bytes, through registers; the rest goes to shared memory by itself
  constexpr int kBytes = kChunk * kGroups / kMoveThreads;
  const int j = tid % kChunk;                  // a thread has one entry's scales
  const uint8_t* const mine = base[j < places ? j : 0];
  const int mine_row = old_row[j < places ? j : 0];
  uint8_t scale[kBytes];
#pragma unroll
  for (int i = 0; i < kBytes; ++i) scale[i] = mine[kv::v_scale(kDim, mine_row, tid / kChunk + i * (kMoveThreads / kChunk))];
  // the record that the request ends in keeps its other rows
  if (places & 15) {
    for (int i = tid; i < kRecord / 16; i += kMoveThreads)
      reinterpret_cast<uint4*>(rec + (whole - 1) * kRecord)[i] = reinterpret_cast<const uint4*>(place[whole - 1])[i];
    __syncthreads();
  }
  constexpr int kKeyVecs = kD / 32;    // 16-byte vectors of a row's keys in a part
#pragma unroll
  for (int i0 = 0; i0 < kChunk * kParts * kKeyVecs; i0 += kMoveThreads) {
    const int i = i0 + tid, j = i / (kParts * kKeyVecs), v = i % (kParts * kKeyVecs), p = v / kKeyVecs, x = v % kKeyVecs;
    const int at = p * 8 * kD + x * 16;
    if (j < places) copy_async16(rec + (j >> 4) * kRecord + at + (j & 15) * (kD / 2), base[j] + at + old_row[j] * (kD / 2));
  }
  if (j < places) {   // rows side by side are likely to come from rows side by side
#pragma unroll
    for (int i = 0; i < kChunk * kParts * 8 / kMoveThreads; ++i) {
      const int x = tid / kChunk + i * (kMoveThreads / kChunk), p = x / 8, y = x % 8;
      auto at = [&](int s) { return 8 * kDim + p * 8 * kD + (s >> 3) * 4 * kD + y * 8 * kC + (s & 7) * kC; };
      uint8_t* const dst = rec + (j >> 4) * kRecord + at(j & 15);
      if constexpr (kC == 8) copy_async8(dst, mine + at(mine_row));
      else copy_async4(dst, mine + at(mine_row));
    }
  }
#pragma unroll
  for (int i0 = 0; i0 < kChunk * kGroups / 4; i0 += kMoveThreads) {
    const int i = i0 + tid, j = i / (kGroups / 4), x = i % (kGroups / 4) * 4;
    if (j < places && i < kChunk * kGroups / 4)
      copy_async4(rec + (j >> 4) * kRecord + kv::k_scale(kDim, j & 15, x), base[j] + kv::k_scale(kDim, old_row[j], x));
  }
  // which of the kept entries lie in this chunk's places
  if (tid < 64) {
    const int at = first_at(list, plan.left, tid < 32 ? j0 : j0 + kChunk);
    if ((tid & 31) == 0) said[2 + tid / 32] = at;
  }
  if (j < places) {
#pragma unroll
    for (int i = 0; i < kBytes; ++i)
      rec[(j >> 4) * kRecord + kv::v_scale(kDim, j & 15, tid / kChunk + i * (kMoveThreads / kChunk))] = scale[i];
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
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
  for (int k = 0; k < whole; ++k)
    for (int i = tid; i < kRecord / 16; i += kMoveThreads)
      reinterpret_cast<uint4*>(place[k])[i] = reinterpret_cast<const uint4*>(rec + k * kRecord)[i];
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
  return a.d == 64    ? launch_kernel(kv_evict_move_kernel<64>, grid, kMoveThreads, 0, s, true, a, units)
         : a.d == 128 ? launch_kernel(kv_evict_move_kernel<128>, grid, kMoveThreads, 0, s, true, a, units)
                      : launch_kernel(kv_evict_move_kernel<256>, grid, kMoveThreads, 0, s, true, a, units);
}

}  // namespace upf
