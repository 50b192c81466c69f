// smem_limit.cuh -- how much dynamic shared memory each kernel may use on each device.
// The runtime keeps one limit for a kernel and device and a launch above it fails, so it
// is raised and never lowered, whichever host threads launch the kernel with whichever
// sizes.  (Host code without CUDA's headers: a test compiles it by itself.)
#pragma once

#include <map>
#include <mutex>
#include <utility>

namespace exl3 {

class SmemLimits {
    std::mutex lock_;
    std::map<std::pair<const void *, int>, int> set_;

public:
    // Raises the limit of `kernel` on device `dev` to `bytes` where it is lower; set()
    // does so and returns 0, or an error, which is handed on.
    template <typename Set> int raise(const void *kernel, int dev, int bytes, Set set) {
        const std::lock_guard<std::mutex> held(lock_);
        int &now = set_[{kernel, dev}];
        if (now >= bytes)
            return 0;
        const int e = set();
        if (e == 0)
            now = bytes;
        return e;
    }
};

}  // namespace exl3
