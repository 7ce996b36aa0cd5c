// A warp's walk over the paged tokens of its plan chunks, in tiles of 32 tokens, ahead of the
// computation: which page and slot each group of 8 tokens lies in (page_size is 8 or a multiple
// of 16 and chunks start at multiples of 32, so a group never crosses a page).
#pragma once

#include "cache_common.cuh"

namespace bskv {
namespace dev {

constexpr int kWalkTile = 32;

// One walk record of the plan (kWalkWords).
struct WalkChunk {
  int unit, begin, end, slot, pbase, item, first_slot, pieces;
};
__device__ __forceinline__ WalkChunk walk_chunk(const int32_t* records, int i) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(records) + 2 * i);
  const int4 b = __ldg(reinterpret_cast<const int4*>(records) + 2 * i + 1);
  return WalkChunk{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

struct PageWalk {
  const int32_t* records;     // of this worker
  const int32_t* kv_indices;
  int left, lane;             // chunks to open yet
  FastDiv heads, page_size;
  int k = -1;                 // chunk being walked
  int tok = 0, end = 0;       // its tokens [tok, end) are still to come
  int kvh = 0, pbase = 0, win = 0;
  // Lane i holds the page and slot of the 8 tokens at win + 8 i, and of those 256 tokens later,
  // read a window ahead so that no copy waits for a page id.
  int page = 0, slot = 0, page2 = 0, slot2 = 0;
  bool fresh = false;

  __device__ __forceinline__ PageWalk(const int32_t* records_, int chunks, const int32_t* indices,
                                      const FastDiv& heads_, const FastDiv& ps, int lane_)
      : records(records_), kv_indices(indices), left(chunks), lane(lane_), heads(heads_), page_size(ps) {
    open();
  }
  __device__ __forceinline__ bool live() const { return left >= 0; }

  __device__ __forceinline__ void lookup(int first, int& pg, int& sl) const {
    const int at = first + 8 * lane;
    if (at < end) {
      pg = __ldg(kv_indices + pbase + page_size.divmod(at, sl));
    }
  }
  __device__ __forceinline__ void open() {
    ++k;
    if (--left < 0) return;
    const WalkChunk c = walk_chunk(records, k);
    heads.divmod(c.unit, kvh);
    tok = win = c.begin;
    end = c.end;
    pbase = c.pbase;
    fresh = true;
    lookup(win, page, slot);
    lookup(win + 256, page2, slot2);
  }
  // Before the tile at `tok` is copied: move on to the next window where it begins one. True when
  // this lane's group is another one than at the last tile.
  __device__ __forceinline__ bool enter() {
    const bool was = fresh;
    fresh = false;
    if (tok - win != 256) return was;
    win = tok;
    page = page2;
    slot = slot2;
    lookup(win + 256, page2, slot2);
    return true;
  }
  // The offset that the lane of row r's group (r in 0..31 of the tile) computed for its group.
  __device__ __forceinline__ int64_t of_group(int64_t offset, int r) const {
    return __shfl_sync(0xffffffffu, static_cast<long long>(offset), ((tok - win) >> 3) + (r >> 3));
  }
  // Whether row r's group of 8 tokens begins before the chunk's end (its last group's rows past
  // `end` lie in the same page).
  __device__ __forceinline__ bool has(int r) const { return tok + (r & ~7) < end; }
  __device__ __forceinline__ void advance() {
    tok += kWalkTile;
    if (tok >= end) open();
  }
};

}  // namespace dev
}  // namespace bskv
