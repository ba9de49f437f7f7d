// The paged 4-bit K/V cache (sm_103a): where a position of a sequence lies.
//
// Pages of P = 2^lg positions, in blocks [pages][H][bytes] of P * 9d/8 bytes per page and K/V head:
// K codes [P][d/2], K statistics [P][d/64] words, V codes, V statistics.  Position p of sequence b
// is position p % P of page table[b][p / P].  A block is one contiguous run, so a page of one head
// moves in one copy, and its K half alone in one too.
#pragma once
#include <stdint.h>

#include "../../include/fg.h"
#include "ragged.cuh"

namespace fg {

struct PagedCache {
  uint8_t* blocks;
  const int32_t* table;
  int64_t table_stride;
  int32_t pages, lg, H, B;

  FG_HD int64_t half_bytes(int d) const { return (int64_t)(9 * d / 16) << lg; }   // K or V
  FG_HD int64_t block_bytes(int d) const { return (int64_t)(9 * d / 8) << lg; }
  FG_HD int64_t cap() const { return table_stride << lg; }      // positions that a table row names
  // The slot (page * P + place in it) of position p < cap() of sequence b, -1 when the table
  // names no page of the cache there.
  FG_HD int64_t slot(int b, int64_t p) const {
    const int32_t page = table[b * table_stride + (p >> lg)];
    if (page < 0 || page >= pages) return -1;
    return ((int64_t)page << lg) | (p & ((1 << lg) - 1));
  }
  // The K half of a slot's block; the V half follows half_bytes(d) behind.
  FG_HD uint8_t* block(int64_t s, int head, int d) const {
    return blocks + ((s >> lg) * H + head) * block_bytes(d);
  }
};

}  // namespace fg
