// kq_kv_dev.h — the paged key-value cache as the kernels see it: where an
// element lies in a page, which tokens a batch holds, and how attention's work
// is shared among workgroups.
//
// A page holds 32 positions. Per key-value head it has one region for K and
// one for V, in pieces of 8 elements ordered as matrix instructions take them:
// a wave's loads of an operand are 64 consecutive 16-byte pieces, V comes
// transposed (8 positions of one channel), and the scores' layout is the next
// product's operand layout without any exchange between lanes. With p the
// position in the page, r = 4 (p / 8) + p % 4, t = (p / 4) % 2:
//   16-bit K: (p, d) at element (d / 32 * 2 + t) * 512 + (d % 32 / 8 * 16 + r) * 8 + d % 8
//   16-bit V: (p, d) at element d / 16 * 512 + (p / 8 * 16 + d % 16) * 8 + p % 8
//   Q8_0 K:   (p, d) at byte d / 32 * 1024 + (d % 32 / 8 * 16 + r) * 16 + t * 8 + d % 8
//   Q8_0 V:   (p, d) at byte d / 32 * 1024 + (p / 8 * 16 + d % 16) * 16 + d % 32 / 16 * 8 + p % 8
//   Q8_0: then the fp16 scales of 32 channels, (p, b) at element b * 32 + p.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_dev.h"
#include "kq_internal.h"

namespace kqd {

constexpr int PAGE = 32;

// Bytes of one head's region of a page.
__host__ __device__ constexpr int64_t region_bytes(bool q8, int D) { return q8 ? 34ll * D : 64ll * D; }

// Element (16 bits) or byte (Q8_0) indices in a region, as above.
__device__ __forceinline__ int k_index(bool q8, int p, int d) {
  const int r = 4 * (p >> 3) + (p & 3), t = (p >> 2) & 1, g = (d & 31) >> 3;
  return q8 ? (d >> 5) * 1024 + (g * 16 + r) * 16 + t * 8 + (d & 7)
            : ((d >> 5) * 2 + t) * 512 + (g * 16 + r) * 8 + (d & 7);
}
__device__ __forceinline__ int v_index(bool q8, int p, int d) {
  return q8 ? (d >> 5) * 1024 + ((p >> 3) * 16 + (d & 15)) * 16 + ((d >> 4) & 1) * 8 + (p & 7)
            : (d >> 4) * 512 + ((p >> 3) * 16 + (d & 15)) * 8 + (p & 7);
}

// Device view of kq_kv_batch and kq_kv_cache.
struct Batch {
  const int32_t* table;
  int64_t width;
  const int32_t* q_start;
  const int32_t* lens;
  int n_seqs;
  int n_tokens;
};
struct Cache {
  uint8_t* k;
  uint8_t* v;
  int64_t n_pages;
  int kv_heads;
};

// The new tokens [begin, begin + n) of a sequence and its length; whatever the
// arrays hold, the tokens lie inside the batch.
struct Seq {
  int begin, n, len;
};
__device__ __forceinline__ Seq seq_of(const Batch& b, int s) {
  int begin = b.q_start[s], end = b.q_start[s + 1];
  begin = min(max(begin, 0), b.n_tokens);
  end = min(max(end, begin), b.n_tokens);
  return Seq{begin, end - begin, min(max(b.lens[s], 0), 0x7fffff00)};
}

// Page id of page `page` of sequence s; -1 where the table names none of the
// cache's pages, -2 behind the table.
__device__ __forceinline__ int32_t page_id(const Batch& b, int64_t n_pages, int s, int page) {
  if (page >= b.width) return -2;
  const int32_t id = b.table[(int64_t)s * b.width + page];
  return id >= 0 && id < n_pages ? id : -1;
}

// The ids of a sequence's pages from `first` on, every `step`-th, 64 of them held
// by the lanes of a wave: the walks take one after the other without waiting for
// the table. Called by whole waves.
struct PageIds {
  int32_t held;
  int from;   // the pages' index of lane 0's
  __device__ __forceinline__ void fill(const Batch& b, int64_t n_pages, int s, int first, int step, int index) {
    const int64_t page = first + (int64_t)(index + (int)(threadIdx.x & 63)) * step;
    held = page > b.width ? -2 : page_id(b, n_pages, s, (int)page);
    from = index;
  }
  __device__ __forceinline__ int32_t at(const Batch& b, int64_t n_pages, int s, int first, int step, int index) {
    if (index - from >= 64) fill(b, n_pages, s, first, step, index);
    return __builtin_amdgcn_readlane(held, index - from);
  }
};

// What a wave wrote to LDS is seen by all its lanes from here on.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Inclusive sum over the lanes of a wave: four shifts within rows of 16, then the
// rows' last values carried on.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_shifted(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = add_shifted<0x111, 0xF>(v);   // row_shr:1
  v = add_shifted<0x112, 0xF>(v);
  v = add_shifted<0x114, 0xF>(v);
  v = add_shifted<0x118, 0xF>(v);
  v = add_shifted<0x142, 0xA>(v);   // row_bcast:15 to rows 1 and 3
  v = add_shifted<0x143, 0xC>(v);   // row_bcast:31 to rows 2 and 3
  return v;
}

// ---- Which part of attention a workgroup does. The columns of a sequence and
// key-value head are its n * G queries (token by token, the G heads of a token
// together), taken `tile` at a time; a tile walks the pages that its sequence's
// queries can see, and where there are few tiles these are split into chunks of
// about equal length, joined by a second kernel in chunk order. `per` pages, the
// longest chunk, is at least the mean of all the work over `target` workgroups and
// at least `least`: at most target + (number of tiles) workgroups have a part,
// and at most 2 target of them belong to a split tile (a sequence of np > per
// pages has ceil(np / per) < 2 np / per chunks). The order of the sums depends on the
// batch's lengths alone.
struct Split {
  int G;          // query heads per key-value head
  int kv_heads;
  int tile;       // columns
  int window;     // 0: none
  int target;
  int least;
  int places;     // workgroups the chip holds at once
  int search;     // look for the shortest chunks that fit them (prompts, whose pages take long)
  int slots;      // partial results the workspace holds
};
struct Part {
  int s;          // sequence, or -1: nothing to do
  Seq seq;
  int first, np;  // the sequence's pages [first, first + np)
  int head, tile; // key-value head, column tile
  int chunk, chunks;
  int slot;       // of a split tile's partial result
};
__device__ __forceinline__ void pages_of(const Batch& b, const Seq& q, int window, int& first, int& np) {
  const int lo = window > 0 ? max(q.len - q.n - window + 1, 0) : 0;   // len - n is the first query's position
  first = lo / PAGE;
  np = (q.len + PAGE - 1) / PAGE - first;
  if ((int64_t)q.len > b.width * PAGE) first = (int)b.width, np = 1;   // behind the table: one look at it says so
  np = max(np, 0);
}
__device__ __forceinline__ int tiles_of(const Split& w, int n) {
  return (int)(((int64_t)n * w.G + w.tile - 1) / w.tile);
}
__device__ __forceinline__ int chunks_of(int np, int per) { return max((np + per - 1) / per, 1); }

// What a lane knows of its sequence.
struct Share {
  Seq q;
  int first, np, tiles;   // np, tiles: 0 behind the last sequence
};
__device__ __forceinline__ Share share_of(const Batch& b, const Split& w, int s) {
  Share h{Seq{0, 0, 0}, 0, 0, 0};
  if (s < b.n_seqs) {
    h.q = seq_of(b, s);
    pages_of(b, h.q, w.window, h.first, h.np);
    h.tiles = tiles_of(w, h.q.n);
  }
  return h;
}

// Pages per chunk; mine: the shares of the first 64 sequences. Called by whole waves.
// Where the tiles are few, chunks are long enough for all of them to fit the chip
// at once (a tile has less than one part more than its share of the pages): a few
// workgroups above that cost a second round (three sequences of 16 rows and 6000
// positions, tiles of 32: 528 workgroups for 512 places 35 us, 480 25). Prompts
// look for the shortest such chunks, up to four tries (500 tokens behind 32000:
// 290 us, 324 with the length taken at once); for decode the tries cost more than
// they gain (one token at 1000 11.3 us, 10.8 without).
__device__ __forceinline__ int pages_per_chunk(const Batch& b, const Split& w, const Share& mine) {
  if (w.slots == 0) return 0x3fffffff;   // no walk is longer
  int64_t total = (int64_t)mine.np * mine.tiles * w.kv_heads;
  for (int s0 = 64; s0 < b.n_seqs; s0 += 64) {
    const Share h = share_of(b, w, s0 + (int)(threadIdx.x & 63));
    total += (int64_t)h.np * h.tiles * w.kv_heads;
  }
  // lower and upper bits apart: a lane's total is below 2^55 for what the calls take
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane(wave_scan((int)(total & 0xffffff)), 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane(wave_scan((int)(total >> 24)), 63);
  const int64_t all = (int64_t)lo + ((int64_t)hi << 24);
  const auto share = [&](int parts) {   // pages, at least `least`
    const int64_t each = all >> 31 == 0 ? (int64_t)(((uint32_t)all + parts - 1) / (uint32_t)parts) : (all + parts - 1) / parts;
    return (int)(each < w.least ? w.least : each > 0x3fffffff ? 0x3fffffff : each);
  };
  const int tiles = __builtin_amdgcn_readlane(wave_scan(mine.tiles * w.kv_heads), 63);
  if (b.n_seqs > 64 || 4 * tiles > w.places) return share(w.target);
  const int enough = share(w.places - tiles);
  if (!w.search) return enough;
  int per = share(w.places);   // less may do
  for (int i = 0; i < 4; ++i) {
    const int parts = __builtin_amdgcn_readlane(wave_scan(mine.tiles * w.kv_heads * chunks_of(mine.np, per)), 63);
    if (parts <= w.places || per >= enough) break;
    per = i == 3 ? enough : min(per + (enough - per + 2) / 3, enough);
  }
  return per;
}

// Part `id` of the grid. Sums of parts stay below 2^31: the calls take grids
// below 2^23, and a sum is carried on while it does not pass id.
__device__ __forceinline__ Part part_of(const Batch& b, const Split& w, int id) {
  const int lane = threadIdx.x & 63;
  Share h = share_of(b, w, lane);
  const int per = pages_per_chunk(b, w, h);
  Part p;
  p.s = -1;
  int before = 0, slots = 0;
  for (int s0 = 0; s0 < b.n_seqs; s0 += 64) {
    if (s0 > 0) h = share_of(b, w, s0 + lane);
    const int chunks = chunks_of(h.np, per);
    const int mine = h.tiles * w.kv_heads * chunks, split = chunks > 1 ? mine : 0;
    const int upto = wave_scan(mine) + before, slot = wave_scan(split) + slots;
    const uint64_t hit = __ballot(id < upto);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      p.s = s0 + l;
      p.seq = Seq{of(h.q.begin), of(h.q.n), of(h.q.len)};
      p.first = of(h.first);
      p.np = of(h.np);
      p.chunks = of(chunks);
      const int local = id - of(upto - mine);
      // heads next to each other: with 8 of them every tile and chunk of a head lies on one XCD
      const int rest = local / w.kv_heads;
      p.head = local - rest * w.kv_heads;
      // the last tiles first: they see the most
      const int tile = p.chunks == 1 ? rest : rest / p.chunks;
      p.chunk = rest - tile * p.chunks;
      p.tile = of(h.tiles) - 1 - tile;
      p.slot = of(slot - split) + (p.tile * p.chunks + p.chunk) * w.kv_heads + p.head;
      if (p.chunks > 1 && p.slot >= w.slots) p.s = -1;   // for starts that do not ascend
      return p;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
    slots = __builtin_amdgcn_readlane(slot, 63);
  }
  return p;
}

// The sequence of a token, its new tokens, the first slot of its split tiles and
// its chunks (1: not split); s < 0: none. Called by whole waves.
struct Row {
  int s, begin, n, slot0, chunks, tiles;
};
__device__ __forceinline__ Row row_of(const Batch& b, const Split& w, int token) {
  const int lane = threadIdx.x & 63;
  Share h = share_of(b, w, lane);
  const int per = pages_per_chunk(b, w, h);
  int slots = 0;
  for (int s0 = 0; s0 < b.n_seqs; s0 += 64) {
    if (s0 > 0) h = share_of(b, w, s0 + lane);
    const int chunks = chunks_of(h.np, per);
    const int split = chunks > 1 ? h.tiles * w.kv_heads * chunks : 0;
    const int slot = wave_scan(split) + slots;
    const uint64_t hit = __ballot(token >= h.q.begin && token < h.q.begin + h.q.n);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      return Row{s0 + l, of(h.q.begin), of(h.q.n), of(slot - split), of(chunks), of(h.tiles)};
    }
    slots = __builtin_amdgcn_readlane(slot, 63);
  }
  return Row{-1, 0, 0, 0, 1, 0};
}

// Split tile `id` (of all sequences' split tiles): its sequence's new tokens, the
// slot of its first chunk, its chunks. begin < 0: there are fewer.
struct SplitTile {
  int begin, n, tile, head, slot, chunks;
};
__device__ __forceinline__ SplitTile split_tile(const Batch& b, const Split& w, int id) {
  const int lane = threadIdx.x & 63;
  Share h = share_of(b, w, lane);
  const int per = pages_per_chunk(b, w, h);
  int before = 0, slots = 0;
  for (int s0 = 0; s0 < b.n_seqs; s0 += 64) {
    if (s0 > 0) h = share_of(b, w, s0 + lane);
    const int chunks = chunks_of(h.np, per);
    const int mine = chunks > 1 ? h.tiles * w.kv_heads : 0, split = mine * chunks;
    const int upto = wave_scan(mine) + before, slot = wave_scan(split) + slots;
    const uint64_t hit = __ballot(id < upto);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      const int local = id - of(upto - mine), tile = local / w.kv_heads, head = local - tile * w.kv_heads;
      const int first = of(slot - split) + tile * of(chunks) * w.kv_heads + head;
      const bool fits = first + (of(chunks) - 1) * w.kv_heads < w.slots;   // not for starts that do not ascend
      return SplitTile{fits ? of(h.q.begin) : -1, of(h.q.n), tile, head, first, of(chunks)};
    }
    before = __builtin_amdgcn_readlane(upto, 63);
    slots = __builtin_amdgcn_readlane(slot, 63);
  }
  return SplitTile{-1, 0, 0, 0, 0, 1};
}

}  // namespace kqd
