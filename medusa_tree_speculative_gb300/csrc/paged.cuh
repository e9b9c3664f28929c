// What the paged cache's kernels share: the cache as they see it, the address
// of a token's line, and the rotation angle of a position.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace medusa {

// medusa_pages_t by value, with the page size as a shift (a power of two).
struct PagesDev {
  int32_t* refs;
  uint32_t* free_bits;
  int32_t* length;
  int32_t* held;
  int32_t* table;
  int num_pages, page_size, shift, rows, max_pages;
};

inline PagesDev pages_dev(const medusa_pages_t* p) {
  PagesDev d;
  d.refs = p->refs; d.free_bits = p->free_bits; d.length = p->length; d.held = p->held; d.table = p->table;
  d.num_pages = p->num_pages; d.page_size = p->page_size; d.rows = p->rows; d.max_pages = p->max_pages;
  d.shift = 0;
  while ((1 << d.shift) < p->page_size) ++d.shift;
  return d;
}

// Row r is usable iff its length fits the pages it holds and those its table.
MDEV bool row_state_ok(const PagesDev& p, int len, int held) {
  return held >= 0 && held <= p.max_pages && len >= 0 && (int64_t)len <= (int64_t)held * p.page_size;
}
MDEV bool page_ok(const PagesDev& p, int page) { return (unsigned)page < (unsigned)p.num_pages; }

// Lines (of Dh elements) before line `line` of head h of a page: pools are
// [num_pages][Hkv][page_size][Dh].
MDEV int64_t page_line(const PagesDev& p, int page, int Hkv, int h, int line) {
  return (((int64_t)page * Hkv + h) << p.shift) + line;
}

// cos and sin of pos * theta^(-2j/Dh).  `turns` is theta^(-2j/Dh) / (2 pi) as a
// 64-bit binary fraction of a turn, so that pos * turns mod 2^64 is the angle's
// fraction of a turn, wrapped exactly, where a float32 product
// pos * theta^(-2j/Dh) is off by up to pos * 2^-25 radians.  `turns` comes from a
// power and a quotient of doubles (for theta >= 1 below 0.16 and off by less than
// 2^-53), and the wrapped fraction is rounded to float32 (at most half a turn
// either way in 24 bits: 2^-26): 2^-26 + pos * 2^-53 turns in all.
MDEV void rope_cos_sin(int pos, uint64_t turns, float& c, float& s) {
  const uint64_t f = (uint64_t)(uint32_t)pos * turns;
  const float half_turns = (float)(int32_t)(f >> 32) * 4.656612873077393e-10f;  // 2^-31: [-1, 1) half turns
  sincospif(half_turns, &s, &c);
}

}  // namespace medusa
