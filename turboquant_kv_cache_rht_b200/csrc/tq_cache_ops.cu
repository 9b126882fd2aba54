// Moving slots of a cache: compaction of the kept slots of every row, and
// copies of rows.  Bytes only; both are bound by memory.
#include "tq_internal.cuh"

#include <algorithm>

namespace tq {
namespace {

constexpr int kMoveThreads = 256;

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

// Moves a column's kept entries down, in order.  Entry i comes from slot
// index[i] >= i, so a chunk's stores only touch slots that this chunk or an
// earlier one has read: they follow the barrier after its loads.
template <typename W>
__device__ __forceinline__ bool move_column(uint8_t* col, int slot_bytes, const int32_t* __restrict__ idx,
                                            int count, int limit) {
  constexpr int PER = 8;
  const int tid = threadIdx.x;
  bool good = true;
  for (int c0 = 0; c0 < count; c0 += kMoveThreads * PER) {
    W v[PER];
    bool on[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = c0 + j * kMoveThreads + tid;
      on[j] = i < count;
      if (on[j]) {
        const int s = idx[i], before = i > 0 ? idx[i - 1] : -1;
        on[j] = s >= 0 && s < limit;
        good = good && on[j] && s > before;
        if (on[j]) v[j] = *reinterpret_cast<const W*>(col + (long)s * slot_bytes);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = c0 + j * kMoveThreads + tid;
      if (on[j]) *reinterpret_cast<W*>(col + (long)i * slot_bytes) = v[j];
    }
  }
  return good;
}

// Grid: (columns, kv_heads, batch).  The last block of a row publishes its
// length (every block read it before taking its ticket).
__global__ void __launch_bounds__(kMoveThreads)
    compact_kernel(const __grid_constant__ Columns cols, const __grid_constant__ CacheView cv,
                   const int32_t* __restrict__ index, long stride_b, long stride_h,
                   const int32_t* __restrict__ counts, int max_count, const int32_t* __restrict__ start) {
  const int h = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  const int len = min(max(cv.seq_lens[b], 0), cv.capacity);
  const int first = start ? start[b] : 0, count = counts[b];
  const bool sound = first >= 0 && first <= len && count >= 0 && count <= max_count && count <= len - first;
  bool good = sound;
  if (sound) {
    const Column& c = cols.c[blockIdx.x];
    uint8_t* col = c.base + (((long)b * cv.kv_heads + h) * cv.capacity + first) * c.slot_bytes + c.offset;
    const int32_t* idx = index + b * stride_b + h * stride_h;
    if (c.width == 16) good = move_column<uint4>(col, c.slot_bytes, idx, count, len - first);
    else if (c.width == 8) good = move_column<uint2>(col, c.slot_bytes, idx, count, len - first);
    else if (c.width == 4) good = move_column<uint32_t>(col, c.slot_bytes, idx, count, len - first);
    else good = move_column<uint16_t>(col, c.slot_bytes, idx, count, len - first);
  }
  const int bad = __syncthreads_or(!good);
  if (threadIdx.x == 0) {
    constexpr int kBad = 1 << 30;  // in append_sync: a block of this row met a bad list
    if (bad) {
      atomicOr(cv.status, (int)kFlagIndex);
      atomicOr(&cv.append_sync[b], kBad);
    }
    __threadfence();
    const int ticket = atomicAdd(&cv.append_sync[b], 1);
    if ((ticket & (kBad - 1)) == (int)(gridDim.x * gridDim.y) - 1) {
      if (!(ticket & kBad)) cv.seq_lens[b] = first + count;
      cv.append_sync[b] = 0;
    }
  }
  pdl_trigger();
}

constexpr int kCopyPieces = 4;  // 16-byte pieces per thread

// Grid: (chunks of `tokens` slots, kv_heads, pairs).
__global__ void __launch_bounds__(kMoveThreads)
    copy_kernel(const __grid_constant__ SlotArrays da, const __grid_constant__ CacheView dst,
                const __grid_constant__ SlotArrays sa, const __grid_constant__ CacheView src,
                const int32_t* __restrict__ dst_rows, const int32_t* __restrict__ src_rows,
                const int32_t* __restrict__ lengths, int n, int max_len, int tokens) {
  const int tid = threadIdx.x, h = blockIdx.y, i = blockIdx.z;
  const bool reports = tid == 0 && h == 0 && blockIdx.x == 0;
  pdl_wait();
  const int to = dst_rows[i], from = src_rows[i];
  const bool one_cache = da.p[0] == sa.p[0];
  if (to < 0 || to >= dst.batch || from < 0 || from >= src.batch) {
    if (reports) atomicOr(dst.status, (int)kFlagIndex);
    return;
  }
  if (one_cache && to == from) return;
  bool clash = false;  // with an earlier pair's dst row, or (one cache) with any pair's src row
  for (int j = tid; j < n; j += kMoveThreads)
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
  const int t0 = blockIdx.x * tokens, m = min(tokens, len - t0);
  if (m <= 0) return;
  // the chunk's bytes of every array, 16 at a time (a chunk starts on a multiple
  // of 16 slots), laid end to end; then the bytes past the last whole piece
  const long s0 = ((long)from * src.kv_heads + h) * src.capacity + t0;
  const long d0 = ((long)to * dst.kv_heads + h) * dst.capacity + t0;
  int total = 0;
#pragma unroll
  for (int a = 0; a < 6; ++a) total += a < sa.n ? (m * sa.bytes[a]) >> 4 : 0;
  for (int u0 = 0; u0 < total; u0 += kMoveThreads * kCopyPieces) {
    uint4 v[kCopyPieces];
    uint8_t* to_p[kCopyPieces];
#pragma unroll
    for (int j = 0; j < kCopyPieces; ++j) {
      int u = u0 + j * kMoveThreads + tid;
      to_p[j] = nullptr;
#pragma unroll
      for (int a = 0; a < 6; ++a) {
        if (a >= sa.n) break;
        const int k = (m * sa.bytes[a]) >> 4;
        if (u >= 0 && u < k) {
          v[j] = *reinterpret_cast<const uint4*>(sa.p[a] + s0 * sa.bytes[a] + 16l * u);
          to_p[j] = da.p[a] + d0 * da.bytes[a] + 16l * u;
        }
        u -= k;
      }
    }
#pragma unroll
    for (int j = 0; j < kCopyPieces; ++j)
      if (to_p[j]) *reinterpret_cast<uint4*>(to_p[j]) = v[j];
  }
  for (int a = 0; a < sa.n; ++a) {
    const int bytes = m * sa.bytes[a], at = (bytes & ~15) + 2 * tid;
    if (at < bytes)
      *reinterpret_cast<uint16_t*>(da.p[a] + d0 * da.bytes[a] + at) =
          *reinterpret_cast<const uint16_t*>(sa.p[a] + s0 * sa.bytes[a] + at);
  }
}

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel kern, dim3 grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMoveThreads);
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
  Columns cols = {};
  for (int a = 0; a < arrays.n; ++a) {
    const int bytes = arrays.bytes[a];
    const int width = bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : bytes % 4 == 0 ? 4 : 2;
    for (int o = 0; o < bytes; o += width) cols.c[cols.n++] = Column{arrays.p[a], bytes, o, width};
  }
  return launch(compact_kernel, dim3(cols.n, cv.kv_heads, cv.batch), stream, cols, cv, index, stride_b,
                stride_h, counts, max_count, start);
}

cudaError_t launch_cache_copy(const SlotArrays& da, const CacheView& dst, const SlotArrays& sa,
                              const CacheView& src, const int32_t* dst_rows, const int32_t* src_rows,
                              const int32_t* lengths, int n, int max_len, cudaStream_t stream) {
  int slot = 0;
  for (int a = 0; a < sa.n; ++a) slot += sa.bytes[a];
  const int tokens = std::max(16, kMoveThreads * kCopyPieces * 16 / slot / 16 * 16);
  const int chunks = std::max(1, (std::min(max_len, src.capacity) + tokens - 1) / tokens);
  return launch(copy_kernel, dim3(chunks, dst.kv_heads, n), stream, da, dst, sa, src, dst_rows, src_rows,
                lengths, n, max_len, tokens);
}

}  // namespace tq
