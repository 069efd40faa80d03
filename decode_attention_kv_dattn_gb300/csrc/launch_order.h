// What the last launch on each stream leaves for the next one to wait for. A kernel
// launched with programmatic stream serialization may run while the launch before it on
// the stream finishes; that launch is the only one that can still be writing.
// Plain C++, so that the host test suite builds it too.
#pragma once

#include <stdint.h>

#include <mutex>
#include <unordered_map>

namespace dattn {

// What names a stream: its handle, but for the default streams, whose handles (0, 1 and 2)
// are the same on every device, and of the last of which each thread has its own.
inline const void* stream_key(const void* stream, int device) {
  static char legacy[64];
  thread_local char own[64];
  const uintptr_t s = reinterpret_cast<uintptr_t>(stream);
  return s > 2 ? stream : (s == 2 ? own : legacy) + (device & 63);
}

class LaunchOrder {
 public:
  // A launch that writes into the cache with K array `cache_k` (null: into no cache).
  void record(const void* stream, const void* cache_k) { put(stream, Last{cache_k, false}); }
  // A launch whose results the next call may take as its inputs. Kernels fetch their
  // inputs before they wait for the launch ahead of them, and only that wait (or a launch
  // in the stream's full order) makes what the launch wrote visible: that its CTAs have
  // all ended, which is when a kernel that gives no signal lets the next one start, is not
  // enough.
  void record_results(const void* stream) { put(stream, Last{nullptr, true}); }

  // Whether the last launch writes into that cache.
  bool writes(const void* stream, const void* cache_k) const {
    const Last l = get(stream);
    return l.written != nullptr && l.written == cache_k;
  }
  // Whether the next launch has to wait for the whole of the last one before it starts
  // (or, in the kernel, before it reads anything).
  bool in_order(const void* stream) const { return get(stream).results; }
  // A launch that waits so has been made: those behind it need not.
  void started(const void* stream) {
    std::lock_guard<std::mutex> lock(mutex_);
    const auto it = last_.find(stream);
    if (it != last_.end()) it->second.results = false;
  }

 private:
  struct Last {
    const void* written;
    bool results;
  };
  void put(const void* stream, Last l) {
    std::lock_guard<std::mutex> lock(mutex_);
    last_[stream] = l;
  }
  Last get(const void* stream) const {
    std::lock_guard<std::mutex> lock(mutex_);
    const auto it = last_.find(stream);
    return it == last_.end() ? Last{nullptr, false} : it->second;
  }
  mutable std::mutex mutex_;
  std::unordered_map<const void*, Last> last_;
};

}  // namespace dattn
