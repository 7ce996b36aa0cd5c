// A warp's walk over the paged tokens of its plan chunks, in tiles of 32 tokens, ahead of the
// computation: which page and slot each group of 8 tokens lies in (page_size is 8 or a multiple
// of 16 and chunks start at multiples of 32, so a group never crosses a page).
#pragma once

#include "common.cuh"
#include "split_merge.cuh"

namespace bskv {
namespace dev {

constexpr int kWalkTile = 32;

struct PageWalk {
  const int4* chunks;         // {unit, first token, end token, slot}; unit = request * heads + head
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  int c0, c1, num_kv_heads, page_size, lane;
  int k = 0;                  // chunk being walked, in chunk_at order
  int tok = 0, end = 0;       // its tokens [tok, end) are still to come
  int kvh = 0, pbase = 0, win = 0;
  // Lane i holds the page and slot of the 8 tokens at win + 8 i, and of those 256 tokens later,
  // read a window ahead so that no copy waits for a page id.
  int page = 0, slot = 0, page2 = 0, slot2 = 0;
  bool fresh = false;

  __device__ __forceinline__ PageWalk(const int32_t* meta, int off_workers, int off_chunks,
                                      int off_aux0, int off_aux1, int worker, int heads, int ps,
                                      int lane_)
      : chunks(reinterpret_cast<const int4*>(meta + off_chunks)), kv_indptr(meta + off_aux0),
        kv_indices(meta + off_aux1), c0(__ldg(meta + off_workers + worker)),
        c1(__ldg(meta + off_workers + worker + 1)), num_kv_heads(heads), page_size(ps), lane(lane_) {
    open();
  }
  __device__ __forceinline__ int count() const { return c1 - c0; }
  __device__ __forceinline__ int4 chunk(int i) const { return __ldg(chunks + chunk_at(c0, c1, i)); }
  __device__ __forceinline__ bool live() const { return k < c1 - c0; }

  __device__ __forceinline__ void lookup(int first, int& pg, int& sl) const {
    const int at = first + 8 * lane;
    if (at < end) {
      const int i = at / page_size;
      pg = __ldg(kv_indices + pbase + i);
      sl = at - i * page_size;
    }
  }
  __device__ __forceinline__ void open() {
    if (!live()) return;
    const int4 ch = chunk(k);
    const int b = ch.x / num_kv_heads;
    kvh = ch.x - b * num_kv_heads;
    tok = win = ch.y;
    end = ch.z;
    pbase = __ldg(kv_indptr + b);
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
    if (tok >= end) {
      ++k;
      open();
    }
  }
};

}  // namespace dev
}  // namespace bskv
