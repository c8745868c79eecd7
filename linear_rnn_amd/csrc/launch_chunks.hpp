// Launches of more workgroups than one grid may have.
#pragma once

#include <stdint.h>

namespace rwkv7 {

// A grid's threads are counted in 32 bits, so how many workgroups fit depends on their size: 2^30 threads a launch.
constexpr uint64_t kLaunchThreads = uint64_t(1) << 30;

// launch(first, n), 0 where it went well, for workgroups first .. first + n - 1 of `blocks` in launches of at most
// kLaunchThreads threads; ends at the first that did not.
template <class Launch>
int in_chunks(uint64_t blocks, int threads, Launch launch) {
  const uint64_t most = kLaunchThreads / threads;
  for (uint64_t first = 0; first < blocks; first += most) {
    const int e = launch((uint32_t)first, (uint32_t)(blocks - first < most ? blocks - first : most));
    if (e != 0) return e;
  }
  return 0;
}

}  // namespace rwkv7
