// Host threads that share a workspace.
//
// The kernels of a call hand each other data through the workspace (split
// partials and their sum, parts of rows and their join), and the stream keeps
// them in the order they were launched in.  Two host threads that launch on
// one stream would mix the kernels of their calls, and the second kernel of
// one would read what the first of the other has left.  So a call holds the
// lock of its workspace from its first launch to its last.  A few locks are
// shared by all workspaces, by address: the library allocates nothing.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>

namespace awq {

class WorkspaceLock {
 public:
  // NULL: no workspace, nothing to hold.
  explicit WorkspaceLock(const void* workspace) {
    if (workspace) hold_ = std::unique_lock<std::mutex>(lock_of(workspace));
  }

 private:
  static std::mutex& lock_of(const void* workspace) {
    static std::mutex locks[kLocks];
    // Allocations begin at multiples of 512 bytes or more.
    const uint64_t x = static_cast<uint64_t>(reinterpret_cast<uintptr_t>(workspace)) >> 9;
    return locks[x * 0x9E3779B97F4A7C15ull >> 58];
  }
  static constexpr size_t kLocks = 64;   // 2^(64 - 58)
  std::unique_lock<std::mutex> hold_;
};

}  // namespace awq
