// Tokens sorted by expert: the sort of the assignments, and the rows copied into its order. (The way back is in
// unpermute.cu.)
//
// The sort is a stable counting sort of the T k assignments (token, then slot) by expert: an assignment's rank is the
// number of earlier ones to its expert, its row the expert's offset plus that (under a placement: round robin over the
// expert's replicas). Whole numbers only, so the order of the atomics does not show. An index outside [0, E) is no
// assignment; ranks at and past the capacity have no row.
//   count_kernel  assignments of each block to each expert
//   rank_kernel   a block's ranks: the counts of the blocks before it, of the warps before a warp, and within a warp
//                 the lanes before a lane that hold the same expert; the offsets are made again by every block
// A batch of one block takes the second kernel alone, which then counts its own.
//
// Rows are copied as words, token by token: the row is read once and written to each of its places.
//
// One GB300: the sort of T k assignments is bound by latency, a few dependent steps a block: 256 x 8 to 256 experts 5.8
// us, one launch; 4096 x 8 6.6 us, 16384 x 8 8.7, 65536 x 8 14.2 (with 1024 experts 16384 x 8 13.4 us: the blocks'
// counts). A block adds up the others' counts itself instead of a third launch; reading them one after the other with
// atomics took 11.8 us for 16384 x 8. The copies are bound by HBM: 16384 rows to eight places each, 7168 bytes and
// scales 164 us (6.6 TB/s, a copy's rate is 6.78), 14336 bytes 315 us (6.7), 65536 rows of 128 bytes 13.5 us (5.6); odd
// 16-bit rows of 1003 59 us (5.0: 64 bytes an access). Slower: bulk copies out of shared memory, a place each (186 us
// instead of 171 for the rows of 7168 bytes); odd rows by the 16-byte words of their places, shifted (65536 x 511 bf16
// with the sort 196 us instead of 135: the parts of words at a row's ends; only rows of kilobytes gain, 215 to 195 for
// 8192 x 7167).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {
namespace pm {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct SortArgs {
  const int32_t* idx;
  const float* weight;  // or nullptr
  int32_t* hist;        // [blocks][E]
  int32_t* counts;
  int32_t* offsets;
  int32_t* inv_pos;
  int32_t* row_token;
  float* row_weight;  // or nullptr
  int64_t n;          // T k
  int64_t per_block;  // a multiple of kThreads
  int E, k, cap, blocks;
  int n_slots, max_replicas;  // 0: one slot an expert
  const int32_t* slot_expert;
  const int32_t* slot_replica;
  const int32_t* replicas;
  const int32_t* replica_slot;
};

__global__ void __launch_bounds__(kThreads) count_kernel(const SortArgs a) {
  extern __shared__ int32_t hist[];
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t lo = blockIdx.x * a.per_block, hi = min(a.n, lo + a.per_block);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int e = a.idx[i];
    if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// exclusive prefix of v over the block's threads, and the total
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before + incl - v;
}

// Shared memory: per warp a count of each expert, then the ranks before the warp's [kWarps][E]; for each expert the
// ranks before this round's [E] and the assignments in all [E]; the offset of each group [max(E, n_slots)].
// EACH: assignments of a lane in a round.
template <int EACH>
__global__ void __launch_bounds__(kThreads) rank_kernel(const SortArgs a) {
  extern __shared__ __align__(16) int32_t sh[];
  __shared__ int warp_sums[kWarps];
  const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* cnt = sh;
  int32_t* base = cnt + kWarps * E;
  int32_t* all = base + E;
  int32_t* offset = all + E;
  const int64_t lo = blockIdx.x * a.per_block, hi = min(a.n, lo + a.per_block);
  int held = 0;
  const int bits = 32 - __clz(E);  // of 0 .. E
  for (int64_t c0 = lo; c0 < hi; c0 += EACH * kThreads) {
    const int64_t at = c0 + warp * 32 * EACH + lane;
    int mine[EACH], rank[EACH];
    float weight[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int64_t i = at + 32 * j;
      mine[j] = i < hi ? a.idx[i] : -1;
      weight[j] = a.row_weight && i < hi ? a.weight[i] : 0.f;
    }
    if (c0 > lo) __syncthreads();
    for (int e = threadIdx.x; e < kWarps / 4 * E; e += kThreads) reinterpret_cast<int4*>(cnt)[e] = make_int4(0, 0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EACH; ++j)
      if (mine[j] < 0 || mine[j] >= E) mine[j] = -1;
    const bool some = c0 + warp * 32 * EACH < hi;  // of the whole warp
    uint32_t same[EACH];  // the lanes that hold the same expert, bit by bit of its number
#pragma unroll
    for (int j = 0; j < EACH; ++j) same[j] = 0xffffffffu;
    for (int b = 0; some && b < bits; ++b)
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const bool set = (unsigned)(mine[j] < 0 ? E : mine[j]) >> b & 1u;
        const uint32_t with = __ballot_sync(0xffffffffu, set);
        same[j] &= set ? with : ~with;
      }
#pragma unroll
    for (int j = 0; j < EACH; ++j) {  // the first lane of an expert counts for all of its lanes
      if (!some) break;
      const int e = mine[j];
      const uint32_t peers = same[j], before = peers & ((1u << lane) - 1u);
      int32_t* c = cnt + warp * E + max(e, 0);
      const int had = *c;
      __syncwarp();
      if (e >= 0 && !before) *c = had + __popc(peers);
      __syncwarp();
      rank[j] = had + __popc(before);
    }
    if (c0 == lo && a.blocks > 1) {  // the other blocks' counts: kThreads / E of them at a time, or one
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int e = threadIdx.x; e < 2 * E; e += kThreads) base[e] = 0;
      __syncthreads();
      const int side = max(1, kThreads / E);
      for (int e = threadIdx.x % (side * E); e < side * E; e += kThreads) {
        if (threadIdx.x >= side * E) break;
        int total = 0, earlier = 0;
        const int32_t* h = a.hist + e % E;
#pragma unroll 16
        for (int b = e / E; b < a.blocks; b += side) {
          const int c = h[(int64_t)b * E];
          total += c;
          if (b < (int)blockIdx.x) earlier += c;
        }
        if (total) atomicAdd(&all[e % E], total);
        if (earlier) atomicAdd(&base[e % E], earlier);
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
      int n = c0 == lo && a.blocks == 1 ? 0 : base[e], c[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) c[w] = cnt[w * E + e];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        cnt[w * E + e] = n;
        n += c[w];
      }
      base[e] = n;
      if (a.blocks == 1) all[e] = n;  // of all once this is the last round, which it is: a batch of one block has one
    }
    if (c0 == lo) {
      __syncthreads();
      const int groups = a.n_slots ? a.n_slots : E;
      for (int g0 = 0; g0 < groups; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        int c = 0;
        if (g < groups) {
          if (a.n_slots) {  // rows of replica i of an expert with r of them: ranks i, i + r, .. below what it keeps
            const int e = a.slot_expert[g], i = a.slot_replica[g], r = a.replicas[e], kept = min(all[e], a.cap);
            c = kept > i ? (kept - i + r - 1) / r : 0;
          } else {
            c = min(all[g], a.cap);
          }
        }
        int total;
        const int first = held + block_prefix(c, warp_sums, total);
        if (g < groups) {
          offset[g] = first;
          if (blockIdx.x == 0) {
            a.counts[g] = c;
            a.offsets[g] = first;
          }
        }
        held += total;
      }
      if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[groups] = held;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int64_t i = at + 32 * j;
      if (i >= hi) continue;
      const int e = mine[j];
      int row = -1;
      if (e >= 0) {
        const int r = rank[j] + cnt[warp * E + e];
        if (r < a.cap) {
          if (a.n_slots) {
            const int n = a.replicas[e];
            row = offset[a.replica_slot[(int64_t)e * a.max_replicas + r % n]] + r / n;
          } else {
            row = offset[e] + r;
          }
          a.row_token[row] = (int)i / a.k;
          if (a.row_weight) a.row_weight[row] = weight[j];
        }
      }
      a.inv_pos[i] = row;
    }
  }
  for (int64_t r = max(lo, (int64_t)held) + threadIdx.x; r < hi; r += kThreads) {  // rows that hold nothing
    a.row_token[r] = -1;
    if (a.row_weight) a.row_weight[r] = 0.f;
  }
}

// ------------------------------------------------------------------------------------------
// rows into the sorted order
// ------------------------------------------------------------------------------------------
struct CopyPlane {
  const void* src;  // [T], ld words from row to row
  void* dst;        // [T k], contiguous
  int64_t ld;
  int words;          // of a row
  int piece, pieces;  // words of a warp's work, a multiple of 32, and those works of a row
};

// Words of a lane in a piece, at most: 16 where there are enough pieces for every SM, else 4 (16384 rows of 7168 bytes to
// eight places each: 165 us with the whole row in a piece, 169 with 8, 172 with 4). A kernel for each of 1, 2, 4 and 6
// words, since each word that a kernel has room for is an instruction for every place: 65536 rows of 129 codes of 8 bits,
// with scales and sort, 59.8 us, with room for 16 words 90; of 159 numbers of 16 bits, 5 words, 44.4 and 47.2 (wide
// words, 16384 x 1536 bf16, 70.5 and 69.1). From 7 words on the room costs nothing (16384 x 2304, 9 words: a kernel for 9
// 105.5 us, for 16 103.5; x 3000, 12 words: 136.2 and 136.6; 65536 x 255, 8 words of 16 bits: 70.7 and 68.9).
constexpr int kDeep = 16;

template <class Word, int DEPTH>
__device__ __forceinline__ void copy_item(const CopyPlane& p, const int32_t* inv_pos, int64_t T, int k, int64_t held,
                                          int64_t item, int lane) {
  const int64_t t = item / p.pieces;
  const int first = (int)(item - t * p.pieces) * p.piece, end = min(p.words, first + p.piece), c0 = first + lane;
  Word v[DEPTH];
  if (t >= T) {  // a row that holds nothing
    Word* dst = static_cast<Word*>(p.dst) + (held + (t - T)) * p.words;
#pragma unroll
    for (int u = 0; u < DEPTH; ++u)
      if (c0 + 32 * u < end) dst[c0 + 32 * u] = Word{};
    return;
  }
  const Word* src = static_cast<const Word*>(p.src) + t * p.ld;
#pragma unroll
  for (int u = 0; u < DEPTH; ++u)
    if (c0 + 32 * u < end) v[u] = src[c0 + 32 * u];
  const int mine = lane < k ? inv_pos[t * k + lane] : -1;
  for (int j = 0; j < k; ++j) {
    const int r = __shfl_sync(0xffffffffu, mine, j);
    if (r < 0 || r >= T * k) continue;
    Word* dst = static_cast<Word*>(p.dst) + (int64_t)r * p.words;
#pragma unroll
    for (int u = 0; u < DEPTH; ++u)
      if (c0 + 32 * u < end) dst[c0 + 32 * u] = v[u];
  }
}

// Rows of at most N LANES words: 32 / LANES of them a warp, a lane N words of each of its row's places, and one of the
// row's scales, of which there are at most LANES.
template <class Word, int LANES, int N>
__global__ void __launch_bounds__(256) permute_short_kernel(const CopyPlane p, const CopyPlane scales, const int32_t* inv_pos,
                                                            const int32_t* held_at, int64_t T, int k) {
  const int sub = threadIdx.x % LANES;
  const int64_t thread = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, threads = (int64_t)gridDim.x * blockDim.x;
  const int64_t held = min(max((int64_t)*held_at, (int64_t)0), T * k);
  const bool scaled = sub < scales.words;
  for (int64_t t = thread / LANES; t < T; t += threads / LANES) {
    const Word* const src = static_cast<const Word*>(p.src) + t * p.ld;
    Word v[N];
    uint32_t scale = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (sub + LANES * n < p.words) v[n] = src[sub + LANES * n];
    if (scaled) scale = static_cast<const uint32_t*>(scales.src)[t * scales.words + sub];
#pragma unroll 8
    for (int j = 0; j < k; ++j) {
      const int r = inv_pos[t * k + j];
      if (r < 0 || r >= T * k) continue;
      Word* const dst = static_cast<Word*>(p.dst) + (int64_t)r * p.words;
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (sub + LANES * n < p.words) dst[sub + LANES * n] = v[n];
      if (scaled) static_cast<uint32_t*>(scales.dst)[(int64_t)r * scales.words + sub] = scale;
    }
  }
  const int64_t bytes = (int64_t)p.words * sizeof(Word);
  rows::clear<sizeof(Word) < 4 ? sizeof(Word) : 4>(p.dst, held * bytes, T * k * bytes, thread, threads);
  if (scales.words) rows::clear<4>(scales.dst, 4 * held * scales.words, 4 * T * k * scales.words, thread, threads);
}

template <class Word, int DEPTH>
__global__ void __launch_bounds__(256) permute_kernel(const CopyPlane p, const CopyPlane scales, const int32_t* inv_pos,
                                                      const int32_t* held_at, int64_t T, int k) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int64_t held = min(max((int64_t)*held_at, (int64_t)0), T * k);
  const int64_t rows = T + (T * k - held);  // token rows, then those that hold nothing
  const int64_t items = rows * p.pieces, more = scales.words ? rows * scales.pieces : 0;
  for (int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < items + more; it += warps) {
    if (it < items)
      copy_item<Word, DEPTH>(p, inv_pos, T, k, held, it, lane);
    else
      copy_item<uint32_t, DEPTH>(scales, inv_pos, T, k, held, it - items, lane);
  }
}

// The word that rows of `bytes` bytes, `ld` bytes apart, are copied by: the widest that every row begins on.
template <class F>
cudaError_t with_word(int64_t bytes, int64_t ld, F&& f) {
  if (bytes % 16 == 0 && ld % 16 == 0) return f(uint4{});
  if (bytes % 4 == 0 && ld % 4 == 0) return f(uint32_t{});
  if (bytes % 2 == 0 && ld % 2 == 0) return f(uint16_t{});
  return f(uint8_t{});
}

// Assignments of a lane in a round of the sort. Two make twice the blocks, each of which reads every block's counts: two
// where those are few, and four where one block then takes all (two and four: 16 x 8 to 256 experts 3.0 and 3.6 us, 4096 x 8
// 6.6 and 9.2, 8192 x 8 7.2 and 8.1, 16384 x 8 12.0 and 8.7; to 64 experts 16384 x 8 7.3 and 8.7; to 1024 experts 2048 x 8
// 8.9 and 12.6, 8192 x 8 12.9 and 11.5).
constexpr int kMaxBlocks = 128;
int each(int64_t n, int E) {
  return n <= 2 * kThreads || (n > 4 * kThreads && n <= 2 * kThreads * kMaxBlocks && n * E <= 1 << 24) ? 2 : 4;
}
int64_t per_block(int64_t n, int E) {
  const int64_t items = (int64_t)each(n, E) * kThreads;
  return std::max<int64_t>(items, cdiv(cdiv(n, kMaxBlocks), items) * items);
}

}  // namespace pm

int sort_blocks(int64_t n, int E) { return (int)cdiv(n, pm::per_block(n, E)); }

// The blocks themselves become fewer where a lane takes four assignments instead of two (8192 x 8 to 256 experts 64,
// 8193 x 8 33), or another round.
int sort_most_blocks(int64_t n) {
  return n <= 4 * pm::kThreads ? 1 : (int)std::min<int64_t>(pm::kMaxBlocks, cdiv(n, 2 * pm::kThreads));
}

cudaError_t launch_sort_tokens(const SortDesc& d, int* launches, cudaStream_t stream) {
  pm::SortArgs a;
  a.idx = d.topk_idx;
  a.weight = d.topk_w;
  a.hist = d.scratch;
  a.counts = d.counts;
  a.offsets = d.offsets;
  a.inv_pos = d.inv_pos;
  a.row_token = d.row_token;
  a.row_weight = d.row_weight;
  a.n = (int64_t)d.T * d.k;
  a.per_block = pm::per_block(a.n, d.E);
  a.E = d.E;
  a.k = d.k;
  a.cap = d.capacity > 0 ? d.capacity : 0x7fffffff;
  a.blocks = sort_blocks(a.n, d.E);
  a.n_slots = d.n_slots;
  a.max_replicas = d.max_replicas;
  a.slot_expert = d.slot_expert;
  a.slot_replica = d.slot_replica;
  a.replicas = d.replicas;
  a.replica_slot = d.replica_slot;
  *launches = 0;
  if (d.T == 0) {
    const int groups = d.n_slots ? d.n_slots : d.E;
    cudaError_t e = cudaMemsetAsync(d.counts, 0, sizeof(int32_t) * groups, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(d.offsets, 0, sizeof(int32_t) * (groups + 1), stream);
    return e;
  }
  const size_t smem = sizeof(int32_t) * ((size_t)(pm::kWarps + 2) * d.E + std::max(d.E, d.n_slots));
  static PerDevice<bool> attr;  // up to 1024 experts and slots need more than the default
  bool set = false;
  cudaError_t e = per_device<bool>(
      attr,
      [](bool& v) {
        constexpr int kMost = (int)(sizeof(int32_t) * (pm::kWarps + 3) * 1024);
        cudaError_t r = cudaFuncSetAttribute(pm::rank_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(pm::rank_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        v = r == cudaSuccess;
        return r;
      },
      &set);
  if (e != cudaSuccess) return e;
  if (a.blocks > 1) {
    pm::count_kernel<<<a.blocks, pm::kThreads, sizeof(int32_t) * d.E, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early;  // beside the counts' end: it ranks its own assignments before it waits for them
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)a.blocks);
  cfg.blockDim = dim3(pm::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = a.blocks > 1 ? 1 : 0;
  ++*launches;
  return cudaLaunchKernelEx(&cfg, pm::each(a.n, d.E) == 2 ? pm::rank_kernel<2> : pm::rank_kernel<4>, a);
}

cudaError_t launch_permute(const PermuteDesc& d, cudaStream_t stream) {
  const int64_t bytes = (int64_t)d.cols * d.element_bytes, ld = d.T > 1 ? d.ldx * d.element_bytes : bytes;
  return pm::with_word(bytes, ld, [&](auto word) {
    using Word = decltype(word);
    pm::CopyPlane p, s{};
    p.src = d.x;
    p.dst = d.xd;
    p.ld = ld / (int64_t)sizeof(Word);
    p.words = (int)(bytes / (int64_t)sizeof(Word));
    const int64_t sms = num_sms();
    if (d.xd_scales) {
      s.src = d.x_scales;
      s.dst = d.xd_scales;
      s.ld = s.words = (int)cdiv(d.cols, 128);
    }
    // Rows of few words share a warp: 65536 rows of 8 words of 16 bytes 13.5 us, with a warp a row 22.9; with their sort
    // (14 us), 33 numbers of 16 bits 28.6 and 33.4 us, 33 codes of 8 bits and their scales 28.3 and 48.2 us.
    if (p.words <= 64) {
      const int lanes = p.words <= 4 ? 4 : p.words <= 8 ? 8 : 16;
      const unsigned blocks = (unsigned)std::min<int64_t>(cdiv((int64_t)d.T * lanes, 256), sms * 32);
      auto kernel = lanes == 4    ? pm::permute_short_kernel<Word, 4, 1>
                    : lanes == 8  ? pm::permute_short_kernel<Word, 8, 1>
                    : p.words <= 16 ? pm::permute_short_kernel<Word, 16, 1>
                    : p.words <= 32 ? pm::permute_short_kernel<Word, 16, 2>
                    : p.words <= 48 ? pm::permute_short_kernel<Word, 16, 3> : pm::permute_short_kernel<Word, 16, 4>;
      kernel<<<blocks, 256, 0, stream>>>(p, s, d.inv_pos, d.held, d.T, d.k);
      return cudaGetLastError();
    }
    // words of a lane in a piece, at most: a long row's in one piece where there are enough pieces for every SM
    const bool enough = d.T * cdiv(p.words, 32 * pm::kDeep) >= sms * 32;
    const int steps = (int)cdiv(p.words, 32), most = enough ? pm::kDeep : 4;
    const int step = (int)cdiv(steps, cdiv(steps, most));  // of a piece: even ones
    const auto cut = [&](pm::CopyPlane& q) {
      q.piece = 32 * step;
      q.pieces = (int)cdiv(q.words, q.piece);
    };
    cut(p);
    if (s.words) cut(s);
    const int64_t items = (int64_t)d.T * (p.pieces + (d.xd_scales ? s.pieces : 0));
    const unsigned blocks = (unsigned)std::min<int64_t>(cdiv(items, 8), sms * 16);
    const auto go = [&](auto kernel) {
      kernel<<<blocks, 256, 0, stream>>>(p, s, d.inv_pos, d.held, d.T, d.k);
      return cudaGetLastError();
    };
    if (step <= 1) return go(pm::permute_kernel<Word, 1>);
    if (step <= 2) return go(pm::permute_kernel<Word, 2>);
    if (step <= 4) return go(pm::permute_kernel<Word, 4>);
    if (step <= 6) return go(pm::permute_kernel<Word, 6>);
    return go(pm::permute_kernel<Word, pm::kDeep>);
  });
}

}  // namespace moe
