// When a bounded wait gives up, in plain C++ so that a host build can check it.
#pragma once

#ifdef __CUDACC__
#define WAIT_HD __host__ __device__
#else
#define WAIT_HD
#endif

namespace jepa {

// A wait may last as long as the work that it waits for, so its limit counts from the last time that
// work was seen to move: after `limit` the count of it is noted, and the wait is over where one more
// limit finds the same count. The wait ends, since the work does: at most two limits after it stood.
struct WaitClock {
  unsigned long long since;
  unsigned seen;

  WAIT_HD explicit WaitClock(unsigned long long now) : since(now), seen(0xffffffffu) {}

  WAIT_HD bool due(unsigned long long now, unsigned long long limit) const { return now - since > limit; }

  // Whether nothing moved since the last time that the wait was due.
  WAIT_HD bool stuck(unsigned long long now, unsigned progress) {
    const bool same = progress == seen;
    seen = progress;
    since = now;
    return same;
  }
};

}  // namespace jepa
