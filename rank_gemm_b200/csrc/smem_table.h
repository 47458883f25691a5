// smem_table.h -- which kernels have had their dynamic shared-memory limit
// raised, and how far: (kernel, device) -> bytes.
//
// Open addressing, nothing is ever taken out.  The library has fewer than 250
// kernels that can enter, so 8 devices fill half of it; past three quarters
// new pairs are not kept (their limit is then set on every call: right, only
// slower), so a search always meets an empty place.  The caller locks.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace svdq {

class SmemTable {
 public:
  static constexpr int SIZE = 4096;   // a power of two

  // The limit that was noted last, 0 when none was.
  size_t raised(const void* fn, int dev) const { return table_[find(fn, dev)].bytes; }
  void note(const void* fn, int dev, size_t bytes) {
    Entry& e = table_[find(fn, dev)];
    if (!e.fn) {
      if (used_ >= SIZE / 4 * 3) return;
      ++used_;
      e.fn = fn;
      e.dev = dev;
    }
    e.bytes = bytes;
  }

 private:
  struct Entry {
    const void* fn;
    int dev;
    size_t bytes;
  };
  // Where the pair is, or the empty place that ends the search for it.
  int find(const void* fn, int dev) const {
    const uint64_t key = (uint64_t)reinterpret_cast<uintptr_t>(fn) + (uint64_t)dev * 0x9E3779B97F4A7C15ull;
    int i = (int)((key * 0xD1342543DE82EF95ull) >> 52) & (SIZE - 1);
    while (table_[i].fn && !(table_[i].fn == fn && table_[i].dev == dev)) i = (i + 1) & (SIZE - 1);
    return i;
  }
  Entry table_[SIZE] = {};
  int used_ = 0;
};

}  // namespace svdq
