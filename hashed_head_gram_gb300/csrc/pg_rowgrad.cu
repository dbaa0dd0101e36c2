// Gradients of table lookups by sorted references: pg_embed_grad (the token embedding) and
// pg_lookup_grad (the hashed multi-head table, PageGram report 9.4, check 4).
//
// A reference is one read of a table row: (t) for the embedding, (t, order, head) for the
// hashed lookup, n of them. With their rows sorted (stably), the references of a row are
// neighbours and its gradient is one segmented sum:
//
//   1. rowgrad_sort_kernel: rows of the references (embedding: the canonical ID; hashed
//      lookup: the hashes of pg_hash.cuh), a stable radix sort of (row, reference) with
//      digits of up to 11 bits, and the numbers of the distinct rows. One cooperative launch; the
//      blocks meet at a grid barrier between the phases. Every block owns a contiguous share
//      of the references, so ranks follow from counts alone and no order depends on timing.
//      Everything it moves stays in L2; its time is latency and instructions: of 71 us for a
//      million reads (PageGram, three digits) 9 are the hashes, 14 the ranks, 10 the scattered
//      stores and 25 the barriers and what is read right after them.
//   2. rowgrad_sum_kernel: the sums, fp32, in ascending order of the references. The sorted
//      references are cut into tiles of a fixed size, whatever the rows' shares (one ID can take
//      a tenth of a batch): a group of lanes walks a tile, writes the rows that lie wholly in it
//      and leaves the sums of the others for
//   3. rowgrad_join_kernel, which adds the parts of a row that crosses tiles, in their order.
//
// The floor is the gradient read once and the output written once: 407 MB, 61 us for the million
// reads of 64 columns. The sums alone take 71 us (372 MB through DRAM while they run, 0.78 of the
// measured copy rate: random 128-byte reads, 16-byte loads 8 deep in 5 blocks of 128 threads an SM, where
// the signed bf16 to fp32 instance spills 28 bytes; 6 blocks spill more, 24 % slower; tiles of 16 references make the embedding's calls 6 and 13 % slower, of 64
// this one 8 %, the other calls within 4 %), and the sort comes before them: 155 us in all, so it is the
// whole distance to the floor. The embedding's sort runs on 32 SMs for 65,536 tokens while the other blocks zero the gradient.
#include "pg_async.cuh"
#include "pg_hash.cuh"
#include "pg_vec.h"

namespace pg {
namespace {

constexpr int kErrGradBarrier = 131072;  // device error bit: a block gave up at the grid barrier
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 8;                          // references a thread holds per tile
constexpr int kSortTile = kSortThreads * kSortItems;   // 8192
// Digits of 6 to 9 bits, where many blocks share a group, and of up to 11 in groups of few blocks:
// every block adds up its group's counts itself. (11 bits everywhere, with a shared scan of the
// counts and a second grid barrier a pass, sorted a million references no sooner in two passes
// than 7 bits do in three: 73 us each.)
constexpr int kMinDigitBits = 6;
constexpr int kManyBits = 9;
constexpr int kMaxDigitBits = 11;
constexpr uint32_t kFewBlocks = 16;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kMaxSortBlocks = 152;                    // one per SM
constexpr uint32_t kRefsPerBlock = 2048;               // at least, before another block joins
constexpr uint64_t kFillPerBlock = 256 << 10;          // bytes of zeros, before another block joins
constexpr int kIdBytes = 4 * (kSortTile + 8);          // a tile's canonical IDs, at one head a token
constexpr int kHashItems = 32;                         // (order, head) items of a table

struct SortCtrl {
  uint32_t barrier;  // arrivals at the grid barrier, all phases
  uint32_t done;     // blocks that finished the sort
  uint32_t count;    // segments (hashed lookup)
  uint32_t pad[61];
};

// Where the references' rows come from.
struct RefSource {
  const int32_t* tokens;
  const uint32_t* canon_map;
  int32_t* err;
  uint32_t vocab;
  uint32_t rows;     // embedding: table rows; rows itself is the key of padding
  uint32_t L;        // hashed lookup: sequence length
  uint64_t fm_L;     // its fastmod constant
  int32_t items;     // hashed lookup: references per token
  int32_t heads;     // of them in a group (items, where there is one group)
  uint32_t per;      // 2^32 / heads, rounded up: tile-local token numbers
  int32_t mode;
  int32_t words;     // hashed lookup: sign words of a reference (1, or an even number)
  ItemConst ic[kHashItems];
};

struct SortBuffers {
  SortCtrl* ctrl;
  uint32_t* hist;      // [blocks][digits]
  uint32_t* segs;      // [blocks] segments that start in a block's share
  uint2* pair[2];      // [n] (row, reference)
  uint64_t* sign;      // [n][words] sign words of the references (hashed lookup)
  float* parts;        // [tiles][2][r] sums of rows that cross a tile's start, its end
};

constexpr size_t kCtrlBytes = sizeof(SortCtrl);

inline size_t up32(size_t x) { return (x + 31) / 32 * 32; }

// References per tile of the sums: 32, and 8 while 32 would leave the GPU short of warps
// (lanes of 8 columns: 16 warps an SM).
constexpr int64_t kFewLanes = 152 * 16 * 32;

inline int tile_refs(int64_t n, int r) { return n * ((r + 7) / 8) / 32 >= kFewLanes ? 32 : 8; }

// Sign words kept for a reference of r columns.
inline int sign_words(int r) { return r <= 64 ? 1 : (r + 127) / 128 * 2; }

// Carves the buffers from `base`; returns the bytes they take (base may be null to size them).
size_t carve(uint8_t* base, int64_t n, int r, bool hashed, SortBuffers* b) {
  size_t at = 0;
  if (base) base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(base) + 31) & ~uintptr_t(31));
  auto take = [&](size_t bytes) {
    uint8_t* p = base ? base + at : nullptr;
    at += up32(bytes);
    return p;
  };
  const size_t un = static_cast<size_t>(n);
  b->ctrl = reinterpret_cast<SortCtrl*>(take(kCtrlBytes));
  b->hist = reinterpret_cast<uint32_t*>(take(sizeof(uint32_t) * kMaxDigits * kMaxSortBlocks));
  b->segs = reinterpret_cast<uint32_t*>(take(sizeof(uint32_t) * kMaxSortBlocks));
  for (int i = 0; i < 2; ++i) b->pair[i] = reinterpret_cast<uint2*>(take(8 * un));
  b->sign = hashed ? reinterpret_cast<uint64_t*>(take(8 * un * sign_words(r))) : nullptr;
  const size_t T = tile_refs(n, r);
  b->parts = reinterpret_cast<float*>(take((un + T - 1) / T * 2 * r * sizeof(float)));
  return at + 32;
}

// ------------------------------------------------------------------------------- the sort

// A later kernel of the same call may be scheduled from here on; it waits for this one's end
// (grid_dep_wait) before it reads anything.
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The G sorting blocks of the grid; false after a time limit of about one second. `phase` counts the
// barriers. A block that arrives after others have given up still completes the count and goes on:
// what they wrote before they arrived is all that it reads, and at its next barrier it gives up too. Its
// writes stay in range, and as `done` falls short of G the later kernels write nothing.
__device__ __forceinline__ bool grid_barrier(uint32_t G, uint32_t* counter, uint32_t* phase, int* s_ok, int* err_word) {
  *phase += 1;
  __syncthreads();
  if (G == 1) return true;
  if (threadIdx.x == 0) {
    // (the release covers what the block's threads wrote before __syncthreads)
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
    const uint32_t want = *phase * G;
    const uint64_t t0 = now_ns();
    uint32_t seen;
    bool ok = true;
    for (;;) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(counter) : "memory");
      if (seen >= want) break;
      if (now_ns() - t0 > kAsyncWaitNs) {
        ok = false;
        if (err_word) atomicOr(err_word, kErrGradBarrier);
        break;
      }
    }
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok != 0;
}

__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Exclusive scan of one value per thread over the block, and the total.
__device__ __forceinline__ uint32_t block_excl_scan(uint32_t v, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t inc = warp_incl_scan(v, lane);
  __syncthreads();
  if (lane == 31) s_warp[w] = inc;
  __syncthreads();
  if (w == 0) {
    const uint32_t x = s_warp[lane];
    const uint32_t xi = warp_incl_scan(x, lane);
    s_warp[lane] = xi - x;
    if (lane == 31) s_warp[kSortWarps] = xi;
  }
  __syncthreads();
  *total = s_warp[kSortWarps];
  return s_warp[w] + inc - v;
}
static_assert(kSortWarps == 32, "block_excl_scan: one lane a warp");

// What a block keeps of a tile of references between counting and scattering. A warp holds
// 32 * items consecutive references, lane l the l-th of each 32.
struct Held {
  uint32_t key[kSortItems], ref[kSortItems];
  uint32_t rank[kSortItems];  // among the warp's references of the same digit
};

__device__ __forceinline__ int tile_items(uint32_t left) {
  return static_cast<int>((min(left, static_cast<uint32_t>(kSortTile)) + kSortThreads - 1) / kSortThreads);
}

// Ranks a tile's references by the digit of `key`, stably, with per-warp counts in s_cnt
// [warps][digits], which become exclusive offsets over the warps; *total gets, in the first
// digits / 2 threads, the tile's counts of digits 2 tid (low half) and 2 tid + 1. Equal digits of a
// warp find one another by one ballot a bit (the match instruction takes a turn per distinct value).
template <int BITS>
__device__ __forceinline__ void rank_tile(Held& h, uint32_t first, uint32_t end, int items, int shift, uint16_t* s_cnt,
                                          uint32_t* s_part, uint32_t* total) {
  constexpr int kDigits = 1 << BITS, kPairs = kDigits / 2;
  constexpr int kParts = kSortThreads / kPairs < kSortWarps ? kSortThreads / kPairs : kSortWarps;
  constexpr int kWarpsPerPart = kSortWarps / kParts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();  // whoever used s_cnt is done
  uint4* clear = reinterpret_cast<uint4*>(s_cnt);
  for (int w = tid; w < kSortWarps * kDigits / 8; w += kSortThreads) clear[w] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  uint16_t* cnt = s_cnt + warp * kDigits;
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    if (j >= items) break;
    const bool in = first + j * 32 + lane < end;
    const uint32_t dig = (h.key[j] >> shift) & (kDigits - 1);
    uint32_t peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int q = 0; q < BITS; ++q) {
      const bool bit = dig & (1u << q);
      const uint32_t set = __ballot_sync(0xffffffffu, bit);
      peers &= bit ? set : ~set;
    }
    const uint32_t before = in ? cnt[dig] : 0u;
    h.rank[j] = before + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (in && lane == 31 - __clz(peers)) cnt[dig] = static_cast<uint16_t>(before + __popc(peers));
    __syncwarp();
  }
  __syncthreads();
  // Counts to offsets, two digits a word (at most 8192 in all, so the halves do not meet): thread
  // (part, pair) adds up its warps' words, then the parts before it, and walks its warps again.
  const int pair = tid % kPairs, part = tid / kPairs;
  uint32_t* word = reinterpret_cast<uint32_t*>(s_cnt) + pair;
  if (part < kParts) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kWarpsPerPart; ++w) sum += word[(part * kWarpsPerPart + w) * kPairs];
    s_part[part * kPairs + pair] = sum;
  }
  __syncthreads();
  uint32_t run = 0, all = 0;
  if (part < kParts) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const uint32_t c = s_part[k * kPairs + pair];
      if (k < part) run += c;
      all += c;
    }
#pragma unroll
    for (int w = 0; w < kWarpsPerPart; ++w) {
      const uint32_t c = word[(part * kWarpsPerPart + w) * kPairs];
      word[(part * kWarpsPerPart + w) * kPairs] = run;
      run += c;
    }
  }
  *total = all;  // (threads of part 0)
}

// The hashed lookup's references are numbered group by group: the rows of a group (one subtable,
// PageGram one order) lie in a range of their own, so each group is sorted by itself, by rows
// that count from its first: fewer digits, and counts of fewer blocks to add up. Reference j of
// a group is head j mod `heads` of token j / heads.

// Canonical IDs of the tokens that a group's references [.., end) and their n-grams read, tok0 the
// tile's first token; four reads of the token and then of the map in flight a thread.
__device__ __forceinline__ void stage_ids(const RefSource& src, uint32_t tok0, uint32_t end, uint32_t* s_id) {
  constexpr int kFly = 4;
  const int64_t first = static_cast<int64_t>(tok0) - 3;
  const int count = static_cast<int>((end - 1) / src.heads - first) + 1;
  for (int k0 = threadIdx.x; k0 < count; k0 += kFly * kSortThreads) {
    int32_t x[kFly];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int64_t at = first + k0 + f * kSortThreads;
      x[f] = k0 + f * kSortThreads < count && at >= 0 ? __ldg(src.tokens + at) : 0;
    }
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int64_t at = first + k0 + f * kSortThreads;
      if (x[f] < 0 || static_cast<uint32_t>(x[f]) >= src.vocab) {  // read as ID 0, and reported
        if (src.err) atomicMin(reinterpret_cast<unsigned int*>(src.err), static_cast<unsigned int>(at));
        x[f] = 0;
      }
      if (src.canon_map) x[f] = static_cast<int32_t>(__ldg(src.canon_map + x[f]));
    }
#pragma unroll
    for (int f = 0; f < kFly; ++f)
      if (k0 + f * kSortThreads < count) s_id[k0 + f * kSortThreads] = static_cast<uint32_t>(x[f]);
  }
}

// Row and sign hash of the reference `local` places after head 0 of token tok0 (local < 8192 +
// 32); *ref = its number by tokens (t * items + item), the row of its gradient.
template <bool PAGED>
__device__ __forceinline__ uint32_t hashed_key(const RefSource& src, const ItemConst* s_ic, const uint32_t* s_id,
                                               uint32_t item0, uint32_t tok0, uint32_t local, uint32_t* ref, uint64_t* hs) {
  const uint32_t s = __umulhi(local, src.per) + (src.heads == 1 ? local : 0u);
  const uint32_t item = item0 + local - s * src.heads;
  const uint32_t t = fastmod(tok0 + s, src.fm_L, src.L);
  *ref = (tok0 + s) * src.items + item;
  const ItemConst& it = s_ic[item];
  // (item_row_ids without the page hash where there are no pages: a third of its multiplications)
  uint64_t hp = 0, hh = 0, h2 = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= it.n) break;
    const uint64_t c = t >= static_cast<uint32_t>(j) ? s_id[s + 3 - j] : kPad;
    if (PAGED) hp ^= c * it.mp[j];
    hh ^= c * it.mh[j];
    h2 ^= c * it.ms[j];
  }
  *hs = h2;
  if (PAGED)
    return it.base + fastmod(fold32(hp), it.fm_main, it.div_main) * it.stride + fastmod(fold32(hh), it.fm_slot, it.slots);
  return it.base + fastmod(fold32(hh), it.fm_main, it.div_main);
}

// The sign words of reference `ref` (an even number of them beyond one: 16 bytes at a time).
__device__ __forceinline__ void store_signs(uint64_t* sign, uint32_t ref, int words, uint64_t hs) {
  if (words == 1) {
    sign[ref] = mix64(hs + kGolden);
    return;
  }
  ulonglong2* at = reinterpret_cast<ulonglong2*>(sign + static_cast<int64_t>(ref) * words);
  for (int q = 0; q < words; q += 2)
    at[q / 2] = make_ulonglong2(mix64(hs + kGolden * static_cast<uint64_t>(q + 1)),
                                mix64(hs + kGolden * static_cast<uint64_t>(q + 2)));
}

// Embedding: the position's row; padding gets the key `rows`.
__device__ __forceinline__ uint32_t embed_key(const RefSource& src, uint32_t i) {
  const uint32_t row = embed_row(src.tokens, src.canon_map, src.vocab, src.rows, i);
  if (row != kNoRow) return row;
  if (src.err) atomicMin(reinterpret_cast<unsigned int*>(src.err), i);
  return src.rows;
}

// Zeros over [p, p + bytes), p and bytes even: block `part` of `parts`.
__device__ __forceinline__ void fill_zeros(uint8_t* p, uint64_t bytes, uint32_t part, uint32_t parts) {
  uint8_t* first = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 31) & ~uintptr_t(31));
  uint8_t* end = p + bytes;
  uint8_t* last = reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(end) & ~uintptr_t(31));
  if (first > last) first = last = end;  // no whole 32 bytes
  const uint64_t pieces = static_cast<uint64_t>(last - first) / 32;
  const float zero[8] = {};
  for (uint64_t i = static_cast<uint64_t>(part) * kSortThreads + threadIdx.x; i < pieces;
       i += static_cast<uint64_t>(parts) * kSortThreads)
    store32(first + 32 * i, zero);
  if (part == 0) {
    for (uint8_t* q = p + 2 * threadIdx.x; q < first; q += 2 * kSortThreads) *reinterpret_cast<uint16_t*>(q) = 0;
    for (uint8_t* q = last + 2 * threadIdx.x; q < end; q += 2 * kSortThreads) *reinterpret_cast<uint16_t*>(q) = 0;
  }
}

// The first G blocks sort, `per_group` of them each of the groups of `size` references, a block
// `share` consecutive ones. Blocks past them, or the same ones afterwards where the grid has no
// others, zero the embedding's gradient (`fill`): writing all of it here, under a sort that uses
// few SMs and no bandwidth, is cheaper than knowing which rows will be written.
template <bool HASHED, int BITS>
__global__ void __launch_bounds__(kSortThreads, 1)
    rowgrad_sort_kernel(const __grid_constant__ RefSource src, const __grid_constant__ SortBuffers b, uint32_t n,
                        uint32_t size, uint32_t per_group, uint32_t share, int passes, uint32_t* __restrict__ rows_out,
                        int32_t* __restrict__ count_out, uint32_t G, uint8_t* fill, uint64_t fill_bytes,
                        int* err_word) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  uint16_t* s_cnt = reinterpret_cast<uint16_t*>(s_raw);                                 // [warps][digits]
  constexpr int kDigits = 1 << BITS, kPairs = kDigits / 2;
  __shared__ uint32_t s_base[kDigits], s_part[kSortThreads];
  __shared__ uint32_t s_warp[kSortWarps + 1];
  __shared__ uint32_t s_first;
  __shared__ int s_ok;
  __shared__ ItemConst s_ic[HASHED ? kHashItems : 1];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t group = blockIdx.x / per_group, part = blockIdx.x - group * per_group, start = group * size;
  const uint32_t lo = start + min(size, part * share), hi = start + min(size, (part + 1) * share);
  const bool one = share <= kSortTile;  // the share stays in registers between counting and scattering
  uint32_t phase = 0, row0 = 0;

  if (blockIdx.x >= G) {
    fill_zeros(fill, fill_bytes, blockIdx.x - G, gridDim.x - G);
    return;
  }
  if (HASHED) {
    // the group's items, a warp a word: the parameter bank serves one address at a time
    constexpr int kWords = static_cast<int>(sizeof(ItemConst) / 4);
    const int first = static_cast<int>(group) * src.heads * kWords, last = first + src.heads * kWords;
    for (int i = first + warp; i < last; i += kSortWarps) {
      const uint32_t x = reinterpret_cast<const uint32_t*>(src.ic)[i];
      if (lane == 0) reinterpret_cast<uint32_t*>(s_ic)[i] = x;
    }
    __syncthreads();
    row0 = s_ic[group * src.heads].base;  // the group's first row: keys count from it
    __syncthreads();
    if (tid < src.heads) s_ic[group * src.heads + tid].base -= row0;
    __syncthreads();
  }

  uint2 *in_order = b.pair[0], *out_order = b.pair[1];
  for (int p = 0; p < passes; ++p) {
    const int shift = p * BITS;
    Held h;
    uint2 mine = make_uint2(0u, 0u);  // this share's counts of digits 2 tid and 2 tid + 1 (tid < kPairs)
    // ---- ranks and counts. A share of several tiles is read again for the scatter.
    for (uint32_t t0 = lo; t0 < hi; t0 += kSortTile) {
      const int items = tile_items(hi - t0);
      const uint32_t first = t0 + warp * 32 * items, end = min(hi, t0 + kSortTile);
      uint32_t tok0 = 0, head0 = 0;  // hashed lookup: the tile's first token, and where in it
      if (HASHED && p == 0) {
        tok0 = (t0 - start) / src.heads;
        head0 = t0 - start - tok0 * src.heads;
        __syncthreads();
        stage_ids(src, tok0, end - start, reinterpret_cast<uint32_t*>(s_cnt));
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kSortItems; ++j) {
        const uint32_t i = first + j * 32 + lane;
        uint2 v = make_uint2(0u, i);
        if (j < items && i < end) {
          if (p > 0) {
            v = __ldcg(in_order + i);
          } else {
            if constexpr (HASHED) {
              uint64_t hs;
              const uint32_t* ids = reinterpret_cast<const uint32_t*>(s_cnt);
              v.x = src.mode == PG_PAGEGRAM
                        ? hashed_key<true>(src, s_ic, ids, group * src.heads, tok0, i - t0 + head0, &v.y, &hs)
                        : hashed_key<false>(src, s_ic, ids, group * src.heads, tok0, i - t0 + head0, &v.y, &hs);
              store_signs(b.sign, v.y, src.words, hs);
            } else {
              v.x = embed_key(src, i);
            }
            if (!one) in_order[i] = v;
          }
        }
        h.key[j] = v.x;
        h.ref[j] = v.y;
      }
      uint32_t total;
      rank_tile<BITS>(h, first, end, items, shift, s_cnt, s_part, &total);
      if (tid < kPairs) {
        mine.x += total & 0xFFFFu;
        mine.y += total >> 16;
      }
    }

    // ---- where this block's first reference of each digit goes: the digits before it, and the
    // same digit in the blocks before it
    uint2 below = make_uint2(0u, 0u), total_of = mine;
    if (G > 1) {
      if (tid < kPairs) *reinterpret_cast<uint2*>(b.hist + blockIdx.x * kDigits + 2 * tid) = mine;
      if (!grid_barrier(G, &b.ctrl->barrier, &phase, &s_ok, err_word)) return;
      // the group's counts, kSortThreads / kPairs blocks at a time
      constexpr int kAtOnce = kSortThreads / kPairs;
      const uint2* counts = reinterpret_cast<const uint2*>(b.hist + group * per_group * kDigits) + tid % kPairs;
      total_of = make_uint2(0u, 0u);
#pragma unroll 8
      for (uint32_t k = tid / kPairs; k < per_group; k += kAtOnce) {
        const uint2 v = __ldcg(counts + k * kPairs);
        below.x += k < part ? v.x : 0u;
        below.y += k < part ? v.y : 0u;
        total_of.x += v.x;
        total_of.y += v.y;
      }
      // join the kAtOnce partial sums, through the room of the counts that the scatter does not need
#pragma unroll
      for (int step = 0; step < 4; ++step) {
        uint32_t& mine_of = step == 0 ? below.x : step == 1 ? below.y : step == 2 ? total_of.x : total_of.y;
        s_part[tid] = mine_of;
        __syncthreads();
        if (tid < kPairs) {
          uint32_t sum = 0;
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) sum += s_part[k * kPairs + tid];
          mine_of = sum;
        }
        __syncthreads();
      }
      if (tid >= kPairs) below = total_of = make_uint2(0u, 0u);
    }
    uint32_t all;
    const uint32_t ex = block_excl_scan(total_of.x + total_of.y, s_warp, &all);
    if (tid < kPairs) {
      s_base[2 * tid] = start + ex + below.x;
      s_base[2 * tid + 1] = start + ex + total_of.x + below.y;
    }
    __syncthreads();

    // ---- scatter
    for (uint32_t t0 = lo; t0 < hi; t0 += kSortTile) {
      const int items = tile_items(hi - t0);
      const uint32_t first = t0 + warp * 32 * items, end = min(hi, t0 + kSortTile);
      uint32_t total = 0;
      if (!one) {
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
          const uint32_t i = first + j * 32 + lane;
          const uint2 v = j < items && i < end ? __ldcg(in_order + i) : make_uint2(0u, i);
          h.key[j] = v.x;
          h.ref[j] = v.y;
        }
        rank_tile<BITS>(h, first, end, items, shift, s_cnt, s_part, &total);
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kSortItems; ++j) {
        if (j < items && first + j * 32 + lane < end) {
          const uint32_t dig = (h.key[j] >> shift) & (kDigits - 1);
          const uint32_t to = s_base[dig] + s_cnt[warp * kDigits + dig] + h.rank[j];
          out_order[to] = make_uint2(h.key[j], h.ref[j]);
        }
      }
      if (!one) {
        __syncthreads();
        if (tid < kPairs) {
          s_base[2 * tid] += total & 0xFFFFu;
          s_base[2 * tid + 1] += total >> 16;
        }
      }
    }
    uint2* swap = in_order;
    in_order = out_order;
    out_order = swap;
    if ((HASHED || p + 1 < passes) && !grid_barrier(G, &b.ctrl->barrier, &phase, &s_ok, err_word)) return;
  }

  if constexpr (HASHED) {
    // ---- segments of equal rows: their numbers replace the rows (in the free buffer), the rows
    // go to rows_out. A thread takes 8 consecutive references at a time.
    auto flags = [&](uint32_t i, uint2 (&v)[8]) -> uint32_t {  // bit j: a segment starts at i + j
      uint32_t prev = i > start && i < hi ? __ldcg(&in_order[i - 1].x) : 0u, f = 0;
      if (i + 8 <= hi && i % 2 == 0) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint4 x = __ldcg(reinterpret_cast<const uint4*>(in_order + i + j));
          v[j] = make_uint2(x.x, x.y);
          v[j + 1] = make_uint2(x.z, x.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j < hi ? __ldcg(in_order + i + j) : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j < hi && (i + j == start || v[j].x != prev)) f |= 1u << j;
        prev = v[j].x;
      }
      return f;
    };
    uint2 v[8];
    uint32_t f = 0, starts = 0, total;
    for (uint32_t i = lo + 8 * tid; i < hi; i += kSortTile) {
      f = flags(i, v);
      starts += __popc(f);
    }
    uint32_t count, u0 = 0;
    block_excl_scan(starts, s_warp, &total);
    if (G == 1) {
      count = total;
    } else {
      if (tid == 0) b.segs[blockIdx.x] = total;
      if (!grid_barrier(G, &b.ctrl->barrier, &phase, &s_ok, err_word)) return;
      const uint32_t ex = block_excl_scan(tid < G ? __ldcg(b.segs + tid) : 0u, s_warp, &count);
      if (tid == blockIdx.x) s_first = ex;
      __syncthreads();
      u0 = s_first;
    }
    for (uint32_t t0 = lo; t0 < hi; t0 += kSortTile) {
      const uint32_t i = t0 + 8 * tid;
      if (!one) f = flags(i, v);
      uint32_t in_tile;
      uint32_t u = u0 + block_excl_scan(__popc(f), s_warp, &in_tile);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j >= hi) break;
        if ((f >> j) & 1u) rows_out[u++] = row0 + v[j].x;
        v[j].x = u - 1;
        if (i + j >= count) rows_out[i + j] = PG_NO_ROW;
      }
      if (i + 8 <= hi && i % 2 == 0) {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          *reinterpret_cast<uint4*>(out_order + i + j) = make_uint4(v[j].x, v[j].y, v[j + 1].x, v[j + 1].y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < hi) out_order[i + j] = v[j];
      }
      u0 += in_tile;
    }
    if (tid == 0 && blockIdx.x == 0) {
      b.ctrl->count = count;
      *count_out = static_cast<int32_t>(count);
    }
  }
  if (fill_bytes && gridDim.x == G) fill_zeros(fill, fill_bytes, blockIdx.x, G);
  if (tid == 0) {
    if (G == 1)
      b.ctrl->done = 1;  // (nothing zeroed it)
    else
      atomicAdd(&b.ctrl->done, 1u);
  }
}

// ------------------------------------------------------------------------------- the sums

constexpr int kSumThreads = 128;   // small blocks: the last wave of them is short
constexpr int kJoinThreads = 256;

struct SumArgs {
  const void* grad;          // summands, rows of r values; reference i has row i / share
  const uint8_t* sign;       // sign bits of the references, a byte for 8 columns (hashed lookup)
  const uint2* order;        // (output row, reference), rows ascending
  const SortCtrl* ctrl;
  float* parts;
  void* out;
  uint32_t n, share, blocks; // blocks: of the sort (all have to have finished)
  uint32_t sign_bytes;       // of a reference
  uint32_t tiles, none;      // none: the output row of padding, which has none
  int32_t r, accumulate, compact;  // compact: rows from the count on are written as zeros
  float scale;
};

// 8 columns (or 1) of a summand as they lie in memory.
template <int IN, int COLS>
struct Raw {
  uint32_t w[COLS == 1 ? 1 : IN == PG_F32 ? 8 : 4];

  __device__ __forceinline__ void load(const void* __restrict__ base, int64_t at) {
    if constexpr (COLS == 1) {
      w[0] = IN == PG_F32 ? __ldg(static_cast<const uint32_t*>(base) + at)
                          : static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + at));
    } else if constexpr (IN == PG_F32) {
      const uint4 x = ldg_stream(static_cast<const float*>(base) + at), y = ldg_stream(static_cast<const float*>(base) + at + 4);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
      w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    } else {
      const uint4 x = ldg_stream(static_cast<const uint16_t*>(base) + at);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
  }

  // acc += the columns, two at a time; SIGNED: those with a bit in `neg` negated
  template <bool SIGNED>
  __device__ __forceinline__ void add(float (&acc)[COLS], uint32_t neg) const {
    auto value = [&](int j) -> uint32_t {
      uint32_t v;
      if constexpr (IN == PG_F32)
        v = w[j];
      else if constexpr (COLS == 1)
        v = w[0] << 16;
      else
        v = (j & 1) ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16;
      return SIGNED ? v ^ ((neg << (31 - j)) & 0x80000000u) : v;
    };
    if constexpr (COLS == 1) {
      acc[0] += __uint_as_float(value(0));
    } else {
#pragma unroll
      for (int j = 0; j < COLS; j += 2)
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
            "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "+f"(acc[j]), "+f"(acc[j + 1])
            : "r"(value(j)), "r"(value(j + 1)));
    }
  }
};

// Output rows in fp32 leave L2 before what is still to be read (nothing here reads them again): the
// gradient's second readers find more of it there. PageGram 160 -> 155 us, Engram-27B 108 -> 106, flat
// 149 -> 143. (bf16 rows have no such 16-byte store; `.cs` in its place changed nothing.)
template <int OUT, int COLS>
__device__ __forceinline__ void store_out(void* base, int64_t at, const float (&x)[COLS]) {
  if constexpr (OUT == PG_F32 && COLS == 8)
    asm volatile("st.global.L2::evict_first.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                     static_cast<float*>(base) + at),
                 "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  else
    store_cols<OUT, COLS>(base, at, x);
}

template <int OUT, int COLS>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t row, int c, const float (&acc)[COLS]) {
  const int64_t at = static_cast<int64_t>(row) * a.r + c;
  float y[COLS] = {};
  if (a.accumulate) read_cols<OUT, COLS>(a.out, at, y);
#pragma unroll
  for (int j = 0; j < COLS; ++j) y[j] = fmaf(acc[j], a.scale, y[j]);
  store_out<OUT, COLS>(a.out, at, y);
}

// This kernel and the join are scheduled before the kernels ahead of them have ended, so what those
// write (order, sign, parts) is read by coherent loads, which no compiler moves ahead of the wait; the
// join reads what the sort wrote, whose end every block of this kernel has waited for, from L2.
//
// A group of `lanes` consecutive threads per tile of T references and lanes * COLS columns.
// The loads of 8 summands (fp32: 4) are in flight at a time, and behind them those of the next
// references' numbers.
template <int IN, int OUT, int COLS, bool SIGNED>
__global__ void __launch_bounds__(kSumThreads, 5)
    rowgrad_sum_kernel(const __grid_constant__ SumArgs a, int lanes, int T) {
  const int per_block = kSumThreads / lanes;
  const int group = threadIdx.x / lanes;
  const uint32_t tile = blockIdx.x * per_block + group;
  const int c = (blockIdx.y * lanes + threadIdx.x - group * lanes) * COLS;
  grid_dep_wait();
  grid_dep_launch();  // after the wait: the join may read what the sort wrote as soon as it runs
  if (group >= per_block || tile >= a.tiles || c >= a.r || a.ctrl->done != a.blocks) return;
  const uint32_t p0 = tile * T, p1 = min(p0 + T, a.n);
  constexpr int kFly = IN == PG_F32 && COLS == 8 ? 4 : 8;
  uint32_t ref[kFly], seg[kFly];
  auto numbers = [&](uint32_t q0) {
    if (q0 + kFly <= p1) {  // p0 is a multiple of 8
#pragma unroll
      for (int k = 0; k < kFly; k += 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(a.order + q0 + k);
        seg[k] = v.x; ref[k] = v.y; seg[k + 1] = v.z; ref[k + 1] = v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const uint2 v = a.order[min(q0 + k, p1 - 1)];
        ref[k] = v.y;
        seg[k] = v.x;  // (past p1: not used)
      }
    }
  };
  numbers(p0);
  const uint32_t before = p0 > 0 ? a.order[p0 - 1].x : kNoRow, after = p1 < a.n ? a.order[p1].x : kNoRow;
  if (a.compact) {  // rows past the last distinct one are zero: row p for each position p of the tile
    const float zero[COLS] = {};
    for (uint32_t u = max(p0, a.ctrl->count); u < p1; ++u)
      store_out<OUT, COLS>(a.out, static_cast<int64_t>(u) * a.r + c, zero);
  }
  float* part = a.parts + static_cast<int64_t>(tile) * 2 * a.r + c;
  float acc[COLS] = {};
  uint32_t cur = seg[0];
  bool from_before = before == cur;  // the row of `cur` began in an earlier tile
  for (uint32_t q0 = p0; q0 < p1 && cur != a.none; q0 += kFly) {
    Raw<IN, COLS> x[kFly];
    uint32_t neg[kFly];
    uint32_t sg[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      x[k].load(a.grad, static_cast<int64_t>(a.share == 1 ? ref[k] : ref[k] / a.share) * a.r + c);
      neg[k] = SIGNED ? a.sign[static_cast<int64_t>(ref[k]) * a.sign_bytes + (c >> 3)] >> (c & 7) : 0u;
      sg[k] = seg[k];
    }
    if (q0 + kFly < p1) numbers(q0 + kFly);
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      if (q0 + k >= p1) break;
      if (sg[k] != cur) {
        if (from_before)
          store_cols<PG_F32, COLS>(part, 0, acc);
        else
          write_row<OUT, COLS>(a, cur, c, acc);
        from_before = false;
        cur = sg[k];
        if (cur == a.none) break;
#pragma unroll
        for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      }
      x[k].template add<SIGNED>(acc, neg[k]);
    }
  }
  if (cur == a.none) return;
  if (from_before)
    store_cols<PG_F32, COLS>(part, 0, acc);
  else if (after == cur)
    store_cols<PG_F32, COLS>(part, a.r, acc);
  else
    write_row<OUT, COLS>(a, cur, c, acc);
}

// Rows that cross tiles: the tile a row starts in adds its parts. A group of lanes per tile, as
// above; a row over more tiles than a block has groups is added by the whole block, group k
// taking every per_block-th part (at most one such row starts in a block's tiles). Of the kFly parts
// that a round reads about two are in flight: each load has a bound check of its own, and the compiler
// adds behind it (34 registers).
template <int OUT, int COLS>
__global__ void __launch_bounds__(kJoinThreads) rowgrad_join_kernel(const __grid_constant__ SumArgs a, int lanes, int T) {
  __shared__ float s_acc[kJoinThreads][COLS];
  __shared__ uint32_t s_long, s_end;
  if (__ldcg(&a.ctrl->done) != a.blocks) {
    grid_dep_wait();
    return;
  }
  const int per_block = kJoinThreads / lanes, group = threadIdx.x / lanes;
  const uint32_t tile = blockIdx.x * per_block + group;
  const int c = group < per_block ? (blockIdx.y * lanes + threadIdx.x - group * lanes) * COLS : a.r;
  if (threadIdx.x == 0) s_long = kNoRow;
  __syncthreads();
  const uint32_t p0 = tile * T, p1 = p0 + T;
  constexpr int kFly = 8;
  auto add = [&](uint32_t k, uint32_t end, uint32_t step, float (&acc)[COLS]) {  // first parts of tiles k, k + step, ..
    for (; k < end; k += kFly * step) {
      float x[kFly][COLS];
#pragma unroll
      for (int f = 0; f < kFly; ++f) {
#pragma unroll
        for (int j = 0; j < COLS; ++j) x[f][j] = 0.f;
        if (k + f * step < end) load_now<COLS>(a.parts + static_cast<int64_t>(k + f * step) * 2 * a.r + c, x[f]);
      }
#pragma unroll
      for (int f = 0; f < kFly; ++f)
#pragma unroll
        for (int j = 0; j < COLS; ++j) acc[j] += x[f][j];
    }
  };
  uint32_t row = kNoRow, end = 0;  // the row that starts in this tile and goes on; past the last tile with a part
  if (group < per_block && tile < a.tiles && p1 < a.n) {
    const uint32_t u = __ldcg(&a.order[p1].x), prev = __ldcg(&a.order[p1 - 1].x);
    const uint32_t before = p0 > 0 ? __ldcg(&a.order[p0 - 1].x) : kNoRow;
    const uint32_t next = p1 + T < a.n ? __ldcg(&a.order[p1 + T].x) : kNoRow;
    if (u == prev && u != before && u != a.none) {
      row = u;
      end = tile + 2;
      if (next == u) {
        // The row goes on past the next tile: how many tiles start with it. Eight probes at a
        // time, the gap between them growing eightfold while all hold it and shrinking after.
        uint32_t k = tile + 2, gap = 1;  // tile k starts with it
        bool grow = true;
        for (;;) {
          uint32_t held = 0;
#pragma unroll
          for (uint32_t f = 1; f <= 8; ++f) {
            const uint64_t at = (static_cast<uint64_t>(k) + f * static_cast<uint64_t>(gap)) * T;
            held += at < a.n && __ldcg(&a.order[at].x) == u;
          }
          k += held * gap;
          grow = grow && held == 8;
          if (grow)
            gap *= 8;
          else if (gap == 1)
            break;
          else
            gap /= 8;
        }
        end = k + 1;
      }
    }
  }
  grid_dep_wait();  // the sums' parts
  if (row != kNoRow) {
    if (end - tile > static_cast<uint32_t>(per_block)) {
      s_long = tile;
      s_end = end;
    } else if (c < a.r) {
      float acc[COLS];
      load_now<COLS>(a.parts + static_cast<int64_t>(tile) * 2 * a.r + a.r + c, acc);
      add(tile + 1, end, 1, acc);
      write_row<OUT, COLS>(a, row, c, acc);
    }
  }
  __syncthreads();
  if (s_long == kNoRow) return;
  float acc[COLS] = {};
  if (c < a.r) {
    if (group == 0) load_now<COLS>(a.parts + static_cast<int64_t>(s_long) * 2 * a.r + a.r + c, acc);
    add(s_long + 1 + group, s_end, per_block, acc);
  }
#pragma unroll
  for (int j = 0; j < COLS; ++j) s_acc[threadIdx.x][j] = acc[j];
  __syncthreads();
  if (group == 0 && c < a.r) {
    for (int k = 1; k < per_block; ++k)
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] += s_acc[k * lanes + threadIdx.x][j];
    write_row<OUT, COLS>(a, __ldcg(&a.order[(s_long + 1) * T].x), c, acc);
  }
}

using SumFn = void (*)(SumArgs, int, int);

template <int COLS, bool SIGNED>
SumFn sum_fn(int in, int out) {
  if (in == PG_F32)
    return out == PG_F32 ? rowgrad_sum_kernel<PG_F32, PG_F32, COLS, SIGNED> : rowgrad_sum_kernel<PG_F32, PG_BF16, COLS, SIGNED>;
  return out == PG_F32 ? rowgrad_sum_kernel<PG_BF16, PG_F32, COLS, SIGNED> : rowgrad_sum_kernel<PG_BF16, PG_BF16, COLS, SIGNED>;
}

template <int COLS>
SumFn join_fn(int out) {
  return out == PG_F32 ? rowgrad_join_kernel<PG_F32, COLS> : rowgrad_join_kernel<PG_BF16, COLS>;
}

// One block of two arrives at the barrier, gives up and leaves without raising `done`, as a sorting
// block does.
__global__ void __launch_bounds__(64) grad_wait_selftest_kernel(SortCtrl* ctrl, int* gave_up, int* err_word) {
  __shared__ int s_ok;
  uint32_t phase = 0;
  if (!grid_barrier(2, &ctrl->barrier, &phase, &s_ok, err_word)) {
    if (threadIdx.x == 0) *gave_up = 1;
    return;
  }
  if (threadIdx.x == 0) atomicAdd(&ctrl->done, 1u);
}

// Sorts the references and writes the sums. n >= 1, in `groups` groups; `keys` the largest key.
template <bool HASHED>
pg_status row_gradients(const RefSource& src, uint32_t n, uint32_t groups, uint32_t keys, SumArgs a, int in, int out, void* workspace,
                        uint32_t* rows_out, int32_t* count_out, cudaStream_t stream) {
  SortBuffers b;
  carve(static_cast<uint8_t*>(workspace), n, a.r, HASHED, &b);
  int key_bits = 1;
  while (key_bits < 32 && (keys >> key_bits)) ++key_bits;
  const uint32_t sms = static_cast<uint32_t>(min(sm_count(), kMaxSortBlocks)), size = n / groups;
  uint32_t per_group = max(1u, min((size + kRefsPerBlock - 1) / kRefsPerBlock, sms / groups));
  const uint32_t share = (size + per_group - 1) / per_group;
  per_group = (size + share - 1) / share;
  const uint32_t G = groups * per_group;
  const int most = per_group <= kFewBlocks ? kMaxDigitBits : kManyBits;
  const int passes = (key_bits + most - 1) / most;
  const int bits = max((key_bits + passes - 1) / passes, kMinDigitBits);

  const uint64_t fill_bytes = HASHED || a.accumulate ? 0 : static_cast<uint64_t>(src.rows) * a.r * dtype_bytes(out);
  const uint64_t fill_blocks = (fill_bytes + kFillPerBlock - 1) / kFillPerBlock;
  const uint32_t grid_blocks = static_cast<uint32_t>(
      min(G + fill_blocks, static_cast<uint64_t>(max(G, sms))));

  cudaError_t e = cudaSuccess;
  if (G > 1) e = cudaMemsetAsync(b.ctrl, 0, kCtrlBytes, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  auto sort = bits == 6    ? rowgrad_sort_kernel<HASHED, 6>
              : bits == 7  ? rowgrad_sort_kernel<HASHED, 7>
              : bits == 8  ? rowgrad_sort_kernel<HASHED, 8>
              : bits == 9  ? rowgrad_sort_kernel<HASHED, 9>
              : bits == 10 ? rowgrad_sort_kernel<HASHED, 10>
                           : rowgrad_sort_kernel<HASHED, 11>;
  const int smem = max(kSortWarps * (2 << bits), HASHED ? kIdBytes : 0);  // the counts; before them, the canonical IDs
  e = cudaFuncSetAttribute(sort, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the blocks meet at a grid barrier
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = G > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, sort, src, b, n, size, per_group, share, passes, rows_out, count_out, G,
                         static_cast<uint8_t*>(a.out), fill_bytes, device_error_word());
  if (e != cudaSuccess) return cuda_fail(e);
  pg_status st = after_launch(1);
  if (st != PG_OK) return st;

  a.order = b.pair[HASHED ? (passes & 1) ^ 1 : passes & 1];  // hashed lookup: with segment numbers
  a.none = HASHED ? kNoRow : src.rows;
  a.compact = HASHED;
  a.sign = reinterpret_cast<const uint8_t*>(b.sign);
  a.sign_bytes = 8 * static_cast<uint32_t>(src.words);
  a.ctrl = b.ctrl;
  a.parts = b.parts;
  a.n = n;
  a.blocks = G;
  const int T = tile_refs(n, a.r);
  a.tiles = (n + T - 1) / T;
  const bool vec = a.r % 8 == 0 && aligned(a.grad, vec_bytes(in)) && aligned(a.out, vec_bytes(out));
  const int cols = vec ? 8 : 1;
  // each is scheduled while the kernel before it runs out, and waits for its end
  auto launch = [&](SumFn fn, int threads, int most) -> pg_status {
    // threads a row, in equal column blocks of at most `most` (an 80-wide head takes 10, 12 tiles a block)
    const int row_threads = (a.r + cols - 1) / cols, col_blocks = (row_threads + most - 1) / most;
    const int lanes = (row_threads + col_blocks - 1) / col_blocks;
    const uint32_t per_block = threads / lanes;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((a.tiles + per_block - 1) / per_block, col_blocks);
    c.blockDim = dim3(threads);
    c.stream = stream;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = early;
    c.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&c, fn, a, lanes, T);
    return err == cudaSuccess ? after_launch(1) : cuda_fail(err);
  };
  st = launch(vec ? sum_fn<8, HASHED>(in, out) : sum_fn<1, HASHED>(in, out), kSumThreads, 32);
  if (st != PG_OK) return st;
  // A common token's row has parts in hundreds of tiles: narrower blocks add more of them at a time
  // (65,536 x 768: 74 us at 32 lanes, 69 at 16, 71 at 8). Hashed rows are shorter, and every column
  // block looks for the ends of its rows again (flat, 768 columns: 143 at 32, 146 at 16, 149 at 8);
  // and a column a thread, 16 would take more than 65,535 blocks in y for the widest rows.
  return launch(vec ? join_fn<8>(out) : join_fn<1>(out), kJoinThreads, HASHED || !vec ? 32 : 16);
}

}  // namespace
}  // namespace pg

using namespace pg;

extern "C" pg_status pg_embed_grad_workspace_size(int64_t N, int64_t rows, int32_t d, size_t* bytes) {
  if (!bytes) return PG_ERR_NULL;
  if (N < 0 || N >= (1ll << 31) || rows < 1 || rows >= (1ll << 31) || d < 1 || d > kMaxEmbedWidth)
    return PG_ERR_SHAPE;
  SortBuffers b;
  *bytes = N == 0 ? 0 : carve(nullptr, N, d, false, &b);
  return PG_OK;
}

extern "C" pg_status pg_embed_grad(const int32_t* tokens, int64_t N, uint32_t vocab, const uint32_t* canon_map,
                                   const void* grad_out, int32_t grad_dtype, int64_t rows, int32_t d, float scale,
                                   int32_t accumulate, void* grad_table, int32_t table_dtype, void* workspace,
                                   size_t workspace_bytes, int32_t* err_index, pg_stream_t stream) {
  size_t need;
  if (vocab == 0) return PG_ERR_SHAPE;
  pg_status st = pg_embed_grad_workspace_size(N, rows, d, &need);
  if (st != PG_OK) return st;
  if (!real_dtype(grad_dtype) || !real_dtype(table_dtype)) return PG_ERR_DTYPE;
  if (!grad_table || (N > 0 && (!tokens || !grad_out))) return PG_ERR_NULL;
  if (!aligned(tokens, 4) || !aligned(canon_map, 4) || !aligned(err_index, 4) ||
      !aligned(grad_out, dtype_bytes(grad_dtype)) || !aligned(grad_table, dtype_bytes(table_dtype)) ||
      !aligned(workspace, 16))
    return PG_ERR_ALIGN;
  if (workspace_bytes < need || (need && !workspace)) return PG_ERR_WORKSPACE;
  if (device_cc() != 103) return PG_ERR_DEVICE;
  st = prepare_err(err_index, stream);
  if (st != PG_OK) return st;
  if (N == 0) {
    if (accumulate) return PG_OK;
    const cudaError_t e =
        cudaMemsetAsync(grad_table, 0, static_cast<size_t>(rows) * d * dtype_bytes(table_dtype), stream);
    return e == cudaSuccess ? PG_OK : cuda_fail(e);
  }
  RefSource src = {};
  src.tokens = tokens;
  src.canon_map = canon_map;
  src.err = err_index;
  src.vocab = vocab;
  src.rows = static_cast<uint32_t>(rows);
  SumArgs a = {};
  a.grad = grad_out;
  a.out = grad_table;
  a.share = 1;
  a.r = d;
  a.accumulate = accumulate;
  a.scale = scale;
  return row_gradients<false>(src, static_cast<uint32_t>(N), 1, src.rows, a, grad_dtype, table_dtype, workspace, nullptr,
                              nullptr, stream);
}

extern "C" pg_status pg_lookup_grad_workspace_size(const pg_table_desc* desc, int64_t N, size_t* bytes) {
  if (!bytes) return PG_ERR_NULL;
  Geometry g;
  pg_status st = validate_desc(desc, &g);
  if (st != PG_OK) return st;
  if (N < 0 || N * g.O * g.H >= (1ll << 31)) return PG_ERR_SHAPE;
  SortBuffers b;
  *bytes = N == 0 ? 0 : carve(nullptr, N * g.O * g.H, desc->r, true, &b);
  return PG_OK;
}

extern "C" pg_status pg_lookup_grad(const pg_table_desc* desc, const int32_t* tokens, int32_t B, int32_t L,
                                    const uint32_t* canon_map, const void* grad_e, int32_t grad_dtype,
                                    uint32_t* rows_out, void* grads_out, int32_t out_dtype, int32_t* count_out,
                                    void* workspace, size_t workspace_bytes, int32_t* err_index, pg_stream_t stream) {
  Geometry g;
  pg_status st = validate_desc(desc, &g);
  if (st != PG_OK) return st;
  if (desc->hash_kind != PG_HASH_MULXOR) return PG_ERR_UNSUPPORTED;
  if (B < 0 || L < 0) return PG_ERR_SHAPE;
  const int items = g.O * g.H;
  if (items > kHashItems || desc->r > kMaxEmbedWidth) return PG_ERR_UNSUPPORTED;
  const int64_t N = static_cast<int64_t>(B) * L;
  if (N >= (1ll << 31)) return PG_ERR_SHAPE;
  size_t need;
  st = pg_lookup_grad_workspace_size(desc, N, &need);
  if (st != PG_OK) return st;
  if (!real_dtype(grad_dtype) || !real_dtype(out_dtype)) return PG_ERR_DTYPE;
  if (!count_out || (N > 0 && (!tokens || !grad_e || !rows_out || !grads_out))) return PG_ERR_NULL;
  if (!aligned(tokens, 4) || !aligned(canon_map, 4) || !aligned(err_index, 4) || !aligned(rows_out, 4) ||
      !aligned(count_out, 4) || !aligned(grad_e, dtype_bytes(grad_dtype)) ||
      !aligned(grads_out, dtype_bytes(out_dtype)) || !aligned(workspace, 16))
    return PG_ERR_ALIGN;
  if (workspace_bytes < need || (need && !workspace)) return PG_ERR_WORKSPACE;
  if (device_cc() != 103) return PG_ERR_DEVICE;
  st = prepare_err(err_index, stream);
  if (st != PG_OK) return st;
  if (N == 0) {
    cudaError_t e = cudaMemsetAsync(count_out, 0, sizeof(int32_t), stream);
    return e == cudaSuccess ? PG_OK : cuda_fail(e);
  }
  RefSource src = {};
  src.tokens = tokens;
  src.canon_map = canon_map;
  src.err = err_index;
  src.vocab = desc->vocab;
  src.L = static_cast<uint32_t>(L);
  src.fm_L = fastmod_constant(src.L);
  src.items = items;
  // groups (see stage_ids), unless one block sorts all of it
  const uint32_t n = static_cast<uint32_t>(N * items);
  const uint32_t groups = n <= static_cast<uint32_t>(kSortTile) ? 1u : desc->mode == PG_ENGRAM ? items : g.O;
  src.heads = items / static_cast<int>(groups);
  src.per = static_cast<uint32_t>(((1ull << 32) + src.heads - 1) / src.heads);  // (1 head: 0, see hashed_key)
  src.mode = desc->mode;
  src.words = sign_words(desc->r);
  HashParams P;
  fill_hash_params(desc, g, &P);
  for (int i = 0; i < items; ++i) init_item_const(src.ic[i], P, desc->hash_seed, i);
  SumArgs a = {};
  a.grad = grad_e;
  a.out = grads_out;
  a.share = desc->mode == PG_FLAT ? static_cast<uint32_t>(items) : 1u;
  a.r = desc->r;
  a.scale = 1.f;
  uint32_t keys = static_cast<uint32_t>(g.rows - 1);
  if (groups > 1) {
    keys = 0;
    for (uint32_t i = 0; i < groups; ++i) {
      const ItemConst& it = src.ic[i * src.heads];
      const uint64_t rows = static_cast<uint64_t>(it.div_main) * (desc->mode == PG_PAGEGRAM ? it.stride : 1u);
      keys = max(keys, static_cast<uint32_t>(rows - 1));
    }
  }
  return row_gradients<true>(src, n, groups, keys, a, grad_dtype, out_dtype, workspace, rows_out, count_out, stream);
}

// Layout of the scratch: see pg.h. The sums and the join would add the zeros there into `sums` if they did not
// see that the sort did not finish; sizes and numbers are such that this too stays within both.
extern "C" pg_status pg_selftest_training_waits(void* scratch, float* sums, pg_stream_t stream) {
  if (!scratch || !sums) return PG_ERR_NULL;
  if (!aligned(scratch, 128) || !aligned(sums, 32)) return PG_ERR_ALIGN;
  if (device_cc() != 103) return PG_ERR_DEVICE;
  uint8_t* base = static_cast<uint8_t*>(scratch);
  cudaError_t e = cudaMemsetAsync(scratch, 0, PG_SELFTEST_SCRATCH, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  int* gave_up = reinterpret_cast<int*>(base);
  SortCtrl* ctrl = reinterpret_cast<SortCtrl*>(base + 128);  // 256 bytes
  grad_wait_selftest_kernel<<<1, 64, 0, stream>>>(ctrl, gave_up, device_error_word());
  pg_status st = after_launch(1);
  if (st != PG_OK) return st;
  constexpr int kR = 8, kT = 8, kTiles = 2;
  SumArgs a = {};
  a.order = reinterpret_cast<const uint2*>(base + 384);      // 16 x (row 0, reference 0)
  a.grad = base + 512;                                       // a row of 8 zeros
  a.parts = reinterpret_cast<float*>(base + 640);            // [2][2][8]
  a.ctrl = ctrl;
  a.out = sums;
  a.n = kTiles * kT;
  a.share = 1;
  a.blocks = 2;
  a.tiles = kTiles;
  a.none = kNoRow;
  a.r = kR;
  a.scale = 1.f;
  sum_fn<8, false>(PG_F32, PG_F32)<<<1, kSumThreads, 0, stream>>>(a, 1, kT);
  if ((st = after_launch(1)) != PG_OK) return st;
  join_fn<8>(PG_F32)<<<1, kJoinThreads, 0, stream>>>(a, 1, kT);
  if ((st = after_launch(1)) != PG_OK) return st;
  return launch_ortho_wait_selftest(base + 1024, gave_up + 1, stream);
}
