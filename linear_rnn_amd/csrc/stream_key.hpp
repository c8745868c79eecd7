// Which stream a handle names, for what the library keeps for each stream (workspaces, rocBLAS handles).
#pragma once

#include <stdint.h>

#include <atomic>
#include <tuple>

namespace rwkv7 {

// A number of the calling thread that no other thread of the process ever has.
inline uint64_t thread_number() {
  static std::atomic<uint64_t> next{1};
  thread_local const uint64_t mine = next.fetch_add(1);
  return mine;
}

// Device, handle, and the thread where the handle is `per_thread` (hipStreamPerThread): that one constant names another
// stream in every thread, and those run side by side.
using StreamKey = std::tuple<int, uintptr_t, uint64_t>;
inline StreamKey stream_key(int device, const void* stream, const void* per_thread) {
  return StreamKey{device, reinterpret_cast<uintptr_t>(stream), stream == per_thread ? thread_number() : 0};
}

}  // namespace rwkv7
