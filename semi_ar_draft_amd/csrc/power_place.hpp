// Where the powers of an MXFP4 cache's token begin: bytes [n_pages][heads][page]
// [blocks of a head].  64 bits: pages times heads alone may pass 32.
#pragma once

#include <cstdint>

namespace dspark {

constexpr int64_t power_place(int page, int heads, int head, int page_shift, int place, int blocks) {
  return ((((int64_t)page * heads + head) << page_shift) + place) * blocks;
}

}  // namespace dspark
