// The small block of device words that a context keeps beside its workspace:
// the error flag and the counters of launches whose workgroups wait for or
// count each other.  All are zero between calls.  One 128-byte line a word
// that is polled; no word belongs to two users.
#pragma once
#include <cstddef>
#include <cstdint>

namespace dspark {

// Chained draft: word 0 is the ticket counter, words 32 .. 127 count finished
// items of (position, group), of which at most 32 positions of two groups are
// in use.  The draft's merge clears all of these words.
constexpr int kChainFirst = 32, kChainCounters = 96;

struct DeviceWords {
  int32_t err;                                         // device error flag (dspark_check)
  int32_t pad0[31];
  unsigned int bar;                                    // grid barrier of the whole-draft kernel
  unsigned int pad1[31];
  unsigned int pages_done;                             // finished workgroups of a page call
  unsigned int pad2[63];
  unsigned int chain[kChainFirst + kChainCounters];    // chained draft
};

static_assert(offsetof(DeviceWords, bar) == 128 && offsetof(DeviceWords, pages_done) == 256 &&
                  offsetof(DeviceWords, chain) == 512 && sizeof(DeviceWords) == 1024,
              "words that different workgroups poll stand on lines of their own");

}  // namespace dspark
