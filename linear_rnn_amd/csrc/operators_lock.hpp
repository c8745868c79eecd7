// Calls that use the operators' workspace hold this while they launch, so that the kernels of two threads' calls on one stream
// do not fall between each other: the workspace belongs to one call from its first kernel to its last.
#pragma once

#include <mutex>

namespace rwkv7 {

inline std::mutex& operators_mutex() {
  static std::mutex m;
  return m;
}

}  // namespace rwkv7
