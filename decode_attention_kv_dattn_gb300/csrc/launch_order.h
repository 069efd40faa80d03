// What the last launch on each stream leaves for the next one to wait for. A kernel
// launched with programmatic stream serialization may run while the launch before it on
// the stream finishes; that launch is the only one that can still be writing.
// Plain C++, so that the host test suite builds it too.
#pragma once

#include <mutex>
#include <unordered_map>

namespace dattn {

class LaunchOrder {
 public:
  // A launch that writes into the cache with K array `cache_k` (null: into no cache).
  void record(void* stream, const void* cache_k) { put(stream, Last{cache_k, false}); }
  // A launch whose results the next call may take as its inputs. Kernels fetch their
  // inputs before they wait for the launch ahead of them, and only that wait (or a launch
  // in the stream's full order) makes what the launch wrote visible: that its CTAs have
  // all ended, which is when a kernel that gives no signal lets the next one start, is not
  // enough.
  void record_results(void* stream) { put(stream, Last{nullptr, true}); }

  // Whether the last launch writes into that cache.
  bool writes(void* stream, const void* cache_k) const {
    const Last l = get(stream);
    return l.written != nullptr && l.written == cache_k;
  }
  // Whether the next launch has to wait for the whole of the last one before it starts.
  bool in_order(void* stream) const { return get(stream).results; }
  // A launch that waits so has been made: those behind it need not.
  void started(void* stream) {
    std::lock_guard<std::mutex> lock(mutex_);
    const auto it = last_.find(stream);
    if (it != last_.end()) it->second.results = false;
  }

 private:
  struct Last {
    const void* written;
    bool results;
  };
  void put(void* stream, Last l) {
    std::lock_guard<std::mutex> lock(mutex_);
    last_[stream] = l;
  }
  Last get(void* stream) const {
    std::lock_guard<std::mutex> lock(mutex_);
    const auto it = last_.find(stream);
    return it == last_.end() ? Last{nullptr, false} : it->second;
  }
  mutable std::mutex mutex_;
  std::unordered_map<void*, Last> last_;
};

}  // namespace dattn
