// limits.cuh -- what has been raised already, per device and kernel (host code).
#pragma once
#include <stddef.h>

#include <mutex>
#include <vector>

namespace moe {

// A kernel's dynamic shared-memory limit is kept by the runtime per device, so
// raising it on one GPU says nothing about another.
class RaisedLimits {
public:
    // True if the kernel's limit on `device` is at least `bytes`, by an earlier
    // call or by raise(), which returns whether it succeeded.
    template <typename F>
    bool ensure(int device, const void *kernel, size_t bytes, F raise) {
        std::lock_guard<std::mutex> lk(mu_);
        Entry *have = nullptr;
        for (Entry &e : done_)
            if (e.kernel == kernel && e.device == device) have = &e;
        if (have && have->bytes >= bytes) return true;
        if (!raise()) return false;
        if (have) have->bytes = bytes;
        else done_.push_back({device, kernel, bytes});
        return true;
    }

private:
    struct Entry {
        int device;
        const void *kernel;
        size_t bytes;
    };
    std::mutex mu_;
    std::vector<Entry> done_;
};

}  // namespace moe
