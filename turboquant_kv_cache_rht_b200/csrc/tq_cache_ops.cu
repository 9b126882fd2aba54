// Moving slots of a cache: compaction of the kept slots of every row, and
// copies of rows.  Bytes only; both are bound by memory.
#include "tq_internal.cuh"

#include <algorithm>
#include <climits>

namespace tq {
namespace {

// One column of an array's slots: `width` bytes at byte `offset` of each slot.
struct Column {
  uint8_t* base;
  int slot_bytes, offset, width;
};
constexpr int kMaxColumns = 24;
struct Columns {
  Column c[kMaxColumns];
  int n;
};

// What a compaction reads of a row, and whether it may touch it.
struct RowPlan {
  int first, count, room;  // first slot, slots kept, slots from `first` on
  bool sound;
};
__device__ __forceinline__ RowPlan plan_row(const CacheView& cv, int b, const int32_t* counts, int max_count,
                                            const int32_t* start) {
  const int len = min(max(cv.seq_lens[b], 0), cv.capacity), first = start ? start[b] : 0, count = counts[b];
  return RowPlan{first, count, len - first,
                 first >= 0 && first <= len && count >= 0 && count <= max_count && count <= len - first};
}

// The last of a row's `blocks` blocks publishes its length (every block read it
// before taking its ticket), unless one of them met a bad list.
__device__ __forceinline__ void publish_row(const CacheView& cv, int b, int blocks, int new_len, bool good) {
  const int bad = __syncthreads_or(!good);
  if (threadIdx.x == 0) {
    constexpr int kBad = 1 << 30;  // in append_sync: a block of this row met a bad list
    if (bad) {
      atomicOr(cv.status, (int)kFlagIndex);
      atomicOr(&cv.append_sync[b], kBad);
    }
    __threadfence();
    const int ticket = atomicAdd(&cv.append_sync[b], 1);
    if ((ticket & (kBad - 1)) == blocks - 1) {
      if (!(ticket & kBad)) cv.seq_lens[b] = new_len;
      cv.append_sync[b] = 0;
    }
  }
}

constexpr int kCompactThreads = 1024, kCompactPer = 4;

// Moves kept entries down, in order: load(slot) gives an entry's bytes, store(slot,
// bytes) writes them.  Entry i comes from slot index[i] >= i, so a chunk's stores only
// touch slots that this chunk or an earlier one has read: they follow the barrier
// after its loads, while the next chunk's loads (from slots past these stores) and the
// indices of the one after are already under way: a chunk costs one memory latency.
// CHECKS: the list's order too (one block of a (row, head) does).
template <typename W, bool CHECKS, typename Load, typename Store>
__device__ __forceinline__ bool move_entries(const int32_t* __restrict__ idx, int count, int limit, Load load,
                                             Store store) {
  constexpr int CHUNK = kCompactThreads * kCompactPer, NP = CHECKS ? kCompactPer : 1;
  const int tid = threadIdx.x;
  bool good = true;
  auto indices = [&](int c0, int (&s)[kCompactPer], int (&before)[NP]) {
#pragma unroll
    for (int j = 0; j < kCompactPer; ++j) {
      const int i = c0 + j * kCompactThreads + tid;
      s[j] = i < count ? idx[i] : INT_MAX;  // (past the list: not a slot)
      if constexpr (CHECKS) before[j] = i < count && i > 0 ? idx[i - 1] : -1;
    }
  };
  auto loads = [&](int c0, const int (&s)[kCompactPer], const int (&before)[NP], W (&v)[kCompactPer]) {
#pragma unroll
    for (int j = 0; j < kCompactPer; ++j) {
      const bool in = s[j] >= 0 && s[j] < limit;
      if (c0 + j * kCompactThreads + tid < count) {
        good = good && in;
        if constexpr (CHECKS) good = good && s[j] > before[j];
      }
      if (in) v[j] = load(s[j]);
    }
  };
  int s0[kCompactPer], s1[kCompactPer], p0[NP], p1[NP];
  W v0[kCompactPer], v1[kCompactPer];
  indices(0, s0, p0);
  indices(CHUNK, s1, p1);
  loads(0, s0, p0, v0);
  for (int c0 = 0; c0 < count; c0 += CHUNK) {
    loads(c0 + CHUNK, s1, p1, v1);
    int s2[kCompactPer], p2[NP];
    indices(c0 + 2 * CHUNK, s2, p2);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCompactPer; ++j) {
      if (s0[j] >= 0 && s0[j] < limit) store(c0 + j * kCompactThreads + tid, v0[j]);
      s0[j] = s1[j];
      s1[j] = s2[j];
      if constexpr (CHECKS) p1[j] = p2[j];
      v0[j] = v1[j];
    }
  }
  return good;
}

template <typename W>
__device__ __forceinline__ bool move_column(uint8_t* col, int slot_bytes, const int32_t* idx, int count, int limit,
                                            bool checks) {
  auto load = [&](int s) { return *reinterpret_cast<const W*>(col + (long)s * slot_bytes); };
  auto store = [&](int i, const W& x) { *reinterpret_cast<W*>(col + (long)i * slot_bytes) = x; };
  return checks ? move_entries<W, true>(idx, count, limit, load, store)
                : move_entries<W, false>(idx, count, limit, load, store);
}

// The 2-byte columns of a row together (norms): up to three.
struct Halves {
  uint16_t x[3];
};

// Grid: (the 2-byte columns as one, if there are any, then the others; kv_heads;
// batch).  (A block for each 2-byte column took as long as one of 16 bytes, and made
// more blocks than the SMs hold.)
__global__ void __launch_bounds__(kCompactThreads, 1)
    compact_kernel(const __grid_constant__ Columns cols, const __grid_constant__ CacheView cv, int halves,
                   const int32_t* __restrict__ index, long stride_b, long stride_h,
                   const int32_t* __restrict__ counts, int max_count, const int32_t* __restrict__ start) {
  const int h = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  const RowPlan r = plan_row(cv, b, counts, max_count, start);
  bool good = r.sound;
  if (r.sound) {
    const int32_t* idx = index + b * stride_b + h * stride_h;
    const long slot0 = ((long)b * cv.kv_heads + h) * cv.capacity + r.first;
    if (halves > 0 && blockIdx.x == 0) {
      uint16_t* col[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) col[k] = reinterpret_cast<uint16_t*>(cols.c[k < halves ? k : 0].base) + slot0;
      good = move_entries<Halves, true>(
          idx, r.count, r.room,
          [&](int s) {
            Halves x;
#pragma unroll
            for (int k = 0; k < 3; ++k) x.x[k] = k < halves ? col[k][s] : (uint16_t)0;
            return x;
          },
          [&](int i, const Halves& x) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
              if (k < halves) col[k][i] = x.x[k];
          });
    } else {
      const Column& c = cols.c[blockIdx.x + (halves > 0 ? halves - 1 : 0)];
      uint8_t* col = c.base + slot0 * c.slot_bytes + c.offset;
      const bool checks = blockIdx.x == 0;
      if (c.width == 16) good = move_column<uint4>(col, c.slot_bytes, idx, r.count, r.room, checks);
      else if (c.width == 8) good = move_column<uint2>(col, c.slot_bytes, idx, r.count, r.room, checks);
      else good = move_column<uint32_t>(col, c.slot_bytes, idx, r.count, r.room, checks);
    }
  }
  publish_row(cv, b, gridDim.x * gridDim.y, r.first + r.count, good);
  pdl_trigger();
}

constexpr int kSmallThreads = 256, kSmallPer = 8;

// Short lists: one block moves every column of a (row, head) in one chunk.
// Grid: (1, kv_heads, batch).
__global__ void __launch_bounds__(kSmallThreads)
    compact_small_kernel(const __grid_constant__ Columns cols, const __grid_constant__ CacheView cv,
                         const int32_t* __restrict__ index, long stride_b, long stride_h,
                         const int32_t* __restrict__ counts, int max_count, const int32_t* __restrict__ start) {
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  __shared__ Column sc[kMaxColumns];  // (columns differ between lanes)
  if (tid < cols.n) sc[tid] = cols.c[tid];
  __syncthreads();
  pdl_wait();
  pdl_trigger();  // this grid is resident at once: the next may set up
  const RowPlan r = plan_row(cv, b, counts, max_count, start);
  bool good = r.sound;
  if (r.sound) {
    const int32_t* idx = index + b * stride_b + h * stride_h;
    const long slot0 = ((long)b * cv.kv_heads + h) * cv.capacity + r.first;
    uint4 v[kSmallPer];
    uint8_t* to[kSmallPer];
#pragma unroll
    for (int j = 0; j < kSmallPer; ++j) {
      const int u = j * kSmallThreads + tid, i = u / cols.n;
      to[j] = nullptr;
      if (i >= r.count) continue;
      const Column& c = sc[u - i * cols.n];
      const int s = idx[i], before = i > 0 ? idx[i - 1] : -1;
      if (s < 0 || s >= r.room || s <= before) good = false;
      if (s < 0 || s >= r.room) continue;
      const uint8_t* from = c.base + (slot0 + s) * c.slot_bytes + c.offset;
      to[j] = c.base + (slot0 + i) * c.slot_bytes + c.offset;
      if (c.width == 16) v[j] = *reinterpret_cast<const uint4*>(from);
      else if (c.width == 8) {
        const uint2 x = *reinterpret_cast<const uint2*>(from);
        v[j] = make_uint4(x.x, x.y, 0u, 0u);
      } else if (c.width == 4) v[j].x = *reinterpret_cast<const uint32_t*>(from);
      else v[j].x = *reinterpret_cast<const uint16_t*>(from);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSmallPer; ++j) {
      if (!to[j]) continue;
      const int u = j * kSmallThreads + tid, width = sc[u % cols.n].width;
      if (width == 16) *reinterpret_cast<uint4*>(to[j]) = v[j];
      else if (width == 8) *reinterpret_cast<uint2*>(to[j]) = make_uint2(v[j].x, v[j].y);
      else if (width == 4) *reinterpret_cast<uint32_t*>(to[j]) = v[j].x;
      else *reinterpret_cast<uint16_t*>(to[j]) = (uint16_t)v[j].x;
    }
  }
  publish_row(cv, b, gridDim.y, r.first + r.count, good);
}

constexpr int kCopyThreads = 256, kCopyPer = 8;          // 16-byte words per thread, all loaded before the first store
constexpr int kCopyPiece = kCopyThreads * kCopyPer * 16;  // bytes of an array that a block moves

// First block of each array along the grid's x (the sizes of max_len tokens).
struct CopyPieces {
  int first[7];
};

// Grid: (pieces of every array, kv_heads, pairs).
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ SlotArrays da, const __grid_constant__ CacheView dst,
                const __grid_constant__ SlotArrays sa, const __grid_constant__ CacheView src,
                const __grid_constant__ CopyPieces pieces, const int32_t* __restrict__ dst_rows,
                const int32_t* __restrict__ src_rows, const int32_t* __restrict__ lengths, int n, int max_len) {
  const int tid = threadIdx.x, h = blockIdx.y, i = blockIdx.z;
  const bool reports = tid == 0 && h == 0 && blockIdx.x == 0;
  int a = 0;
#pragma unroll
  for (int k = 1; k < 6; ++k)
    if (k < sa.n && (int)blockIdx.x >= pieces.first[k]) a = k;
  const int bytes = sa.bytes[a];
  const long at = (long)(blockIdx.x - pieces.first[a]) * kCopyPiece;
  pdl_wait();
  const int to = dst_rows[i], from = src_rows[i];
  const bool one_cache = da.p[0] == sa.p[0];
  if (to < 0 || to >= dst.batch || from < 0 || from >= src.batch) {
    if (reports) atomicOr(dst.status, (int)kFlagIndex);
    return;
  }
  if (one_cache && to == from) return;
  bool clash = false;  // with an earlier pair's dst row, or (one cache) with any pair's src row
  for (int j = tid; j < n; j += kCopyThreads)
    clash = clash || (j < i && dst_rows[j] == to) || (one_cache && src_rows[j] == to);
  if (__syncthreads_or(clash)) {
    if (reports) atomicOr(dst.status, (int)kFlagIndex);
    return;
  }
  const int stored = min(max(src.seq_lens[from], 0), src.capacity);
  int len = lengths ? min(max(lengths[i], 0), stored) : stored;
  if (len > max_len) {
    len = max_len;
    if (reports) atomicOr(dst.status, (int)kFlagMaxCtx);
  }
  if (len > dst.capacity) {
    if (reports) atomicOr(dst.status, (int)kFlagCapacity);
    return;
  }
  if (reports) dst.seq_lens[to] = len;
  const long total = (long)len * bytes;  // of this array, row and head: contiguous
  if (at >= total) return;
  const uint8_t* s = sa.p[a] + ((long)from * src.kv_heads + h) * src.capacity * bytes + at;
  uint8_t* d = da.p[a] + ((long)to * dst.kv_heads + h) * dst.capacity * bytes + at;
  const int m = (int)min((long)kCopyPiece, total - at), words = m >> 4;
  uint4 v[kCopyPer];
#pragma unroll
  for (int j = 0; j < kCopyPer; ++j)
    if (j * kCopyThreads + tid < words) v[j] = __ldcs(reinterpret_cast<const uint4*>(s) + j * kCopyThreads + tid);
#pragma unroll
  for (int j = 0; j < kCopyPer; ++j)
    if (j * kCopyThreads + tid < words) __stcs(reinterpret_cast<uint4*>(d) + j * kCopyThreads + tid, v[j]);
  const int tail = (words << 4) + 2 * tid;  // a row's last bytes: up to seven 2-byte ones
  if (tail < m) *reinterpret_cast<uint16_t*>(d + tail) = *reinterpret_cast<const uint16_t*>(s + tail);
}

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel kern, dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_cache_compact(const SlotArrays& arrays, const CacheView& cv, const int32_t* index,
                                 long stride_b, long stride_h, const int32_t* counts, int max_count,
                                 const int32_t* start, cudaStream_t stream) {
  Columns cols = {};  // the 2-byte ones first
  int halves = 0;
  for (int pass = 0; pass < 2; ++pass)
    for (int a = 0; a < arrays.n; ++a) {
      const int bytes = arrays.bytes[a];
      const int width = bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : bytes % 4 == 0 ? 4 : 2;
      if ((width == 2) != (pass == 0)) continue;
      for (int o = 0; o < bytes; o += width) cols.c[cols.n++] = Column{arrays.p[a], bytes, o, width};
      halves += width == 2 ? 1 : 0;  // (an array of 2-byte slots: norms)
    }
  // A list whose pieces one block holds at once takes a block per (row, head): 64
  // drafts of 32 rows and 8 heads cut to 6 in 4 us instead of the 10 that a block
  // per column takes to start and to meet; long lists need the columns' blocks.
  if ((long)max_count * cols.n <= kSmallThreads * kSmallPer)
    return launch(compact_small_kernel, dim3(1, cv.kv_heads, cv.batch), kSmallThreads, stream, cols, cv, index,
                  stride_b, stride_h, counts, max_count, start);
  const int blocks = cols.n - (halves > 0 ? halves - 1 : 0);
  return launch(compact_kernel, dim3(blocks, cv.kv_heads, cv.batch), kCompactThreads, stream, cols, cv, halves, index,
                stride_b, stride_h, counts, max_count, start);
}

cudaError_t launch_cache_copy(const SlotArrays& da, const CacheView& dst, const SlotArrays& sa,
                              const CacheView& src, const int32_t* dst_rows, const int32_t* src_rows,
                              const int32_t* lengths, int n, int max_len, cudaStream_t stream) {
  CopyPieces pieces = {};
  long blocks = 0;
  for (int a = 0; a < sa.n; ++a) {
    pieces.first[a] = (int)blocks;
    const long bytes = (long)std::min(max_len, src.capacity) * sa.bytes[a];
    blocks += std::max(1L, (bytes + kCopyPiece - 1) / kCopyPiece);
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
  }
  return launch(copy_kernel, dim3((unsigned)blocks, dst.kv_heads, n), kCopyThreads, stream, da, dst, sa, src, pieces,
                dst_rows, src_rows, lengths, n, max_len);
}

}  // namespace tq
