// device_once.h -- set-up and checks that a kernel needs once per device: a
// call that succeeded is not made again, one that failed is (a failure may be
// another call's pending error, or another device's).
#pragma once

#include <mutex>

namespace pa {

template <int DEVICES, int SLOTS>
class DeviceOnce {
public:
    // fn() -> 0 on success, else an error, which is returned and not kept.
    // Devices and slots outside the table are asked every time.
    template <typename Fn>
    auto run(int device, int slot, Fn fn) -> decltype(fn()) {
        if (device < 0 || device >= DEVICES || slot < 0 || slot >= SLOTS) return fn();
        std::lock_guard<std::mutex> lock(mu_);
        if (done_[device][slot]) return decltype(fn())(0);
        const auto e = fn();
        done_[device][slot] = e == decltype(fn())(0);
        return e;
    }

private:
    std::mutex mu_;
    bool done_[DEVICES][SLOTS] = {};
};

}  // namespace pa
