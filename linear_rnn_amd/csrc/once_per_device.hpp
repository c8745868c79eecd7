// What has to be asked of the runtime once on every device before a kernel's first launch there.
#pragma once

#include <stdint.h>

#include <atomic>

namespace rwkv7 {

// ask() (0: granted) unless it was granted on this device before; a refusal is asked again by the next call. `granted`: a bit
// for each device (devices past 63 ask every time).
template <class Ask>
int once_per_device(std::atomic<uint64_t>& granted, int device, Ask ask) {
  const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
  if (granted.load(std::memory_order_acquire) & bit) return 0;
  const int status = ask();
  if (status == 0) granted.fetch_or(bit, std::memory_order_release);
  return status;
}

}  // namespace rwkv7
