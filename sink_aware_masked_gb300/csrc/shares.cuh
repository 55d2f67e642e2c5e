// A decode call's work shared out between its workers.
#pragma once

#include "common.cuh"

namespace sa {

// The line of all blocks cut into equal shares: worker c takes [start(c), start(c + 1)).
struct Shares {
  long long work, each;
  int workers, more;  // the first `more` workers take one block more than `each`
  float per_block;
  SA_DEV Shares(long long w, int n) : work(w), workers(n) {
    if (w < (1LL << 32)) {  // the cheaper division
      each = static_cast<uint32_t>(w) / static_cast<uint32_t>(n);
    } else {
      each = w / n;
    }
    more = static_cast<int>(w - each * n);
    per_block = __fdividef(static_cast<float>(n), static_cast<float>(w));
  }
  SA_DEV long long start(int c) const { return c * each + min(c, more); }
  SA_DEV int owner(long long x) const {  // the share that holds block x: an estimate, off by one at most, put right
    int c = min(max(static_cast<int>(static_cast<float>(x) * per_block), 0), workers - 1);
    while (start(c) > x) --c;
    while (start(c + 1) <= x) ++c;
    return c;
  }
};

}  // namespace sa
