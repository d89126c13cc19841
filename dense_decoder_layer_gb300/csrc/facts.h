// What a component call looks up once per device: its status word and its SMs.
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>

namespace pds {

class DeviceFacts {
 public:
  // False, with nothing kept, where the lookup fails: a later call looks again.
  // lookup(uint32_t** status, int* sms) says whether it found both.
  template <typename Lookup>
  bool get(Lookup&& lookup, uint32_t** status, int* sms) {
    if (!ready_.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> hold(lock_);
      if (!ready_.load(std::memory_order_relaxed)) {
        uint32_t* s = nullptr;
        int n = 0;
        if (!lookup(&s, &n)) return false;
        status_ = s;
        sms_ = n;
        ready_.store(true, std::memory_order_release);
      }
    }
    *status = status_;
    *sms = sms_;
    return true;
  }

 private:
  std::atomic<bool> ready_{false};
  std::mutex lock_;
  uint32_t* status_ = nullptr;
  int sms_ = 0;
};

}  // namespace pds
