// How long a bounded wait of the tensor-core kernels may last.
#pragma once

#ifdef __CUDACC__
#define ZFS_HOST_DEVICE __host__ __device__
#else
#define ZFS_HOST_DEVICE
#endif

namespace zfs {

// Products and copies take microseconds: after kWaitNs of polling they never
// will come.
constexpr unsigned long long kWaitNs = 1000000000ull;
// Two polls further apart than this have the time in between taken off: the
// kernel was not running (another process's time slice, a debugger), nor were
// the products it waits for.  At most kMaxGaps times, so that every wait ends.
constexpr unsigned long long kGapNs = 10000000ull;
constexpr int kMaxGaps = 1000;

struct Patience {
  unsigned long long start, last;
  int gaps;
  ZFS_HOST_DEVICE explicit Patience(unsigned long long now) : start(now), last(now), gaps(0) {}
  // Whether the wait, polled in vain at `now` (ns), has lasted long enough.
  ZFS_HOST_DEVICE bool spent(unsigned long long now) {
    if (now - last > kGapNs && gaps < kMaxGaps) {
      start += now - last;
      ++gaps;
    }
    last = now;
    return now - start > kWaitNs;
  }
};

}  // namespace zfs
