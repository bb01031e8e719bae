// How many clusters of a kernel a device holds at once: the driver is asked once for each kernel, device, cluster size and
// orientation, on the way to its first launch, however many kernels there are. (An array of 64 answers could fill up, and from
// then on every launch of the kernels that were not in it asked again.)
#pragma once

#include <map>
#include <mutex>
#include <tuple>

namespace lowbit {

class CapacityCache {
public:
    template <class Ask>
    int get(const void* kernel, int device, int cluster, bool along_x, Ask ask) {
        const Key key(kernel, device, cluster, along_x);
        {
            std::lock_guard<std::mutex> lock(mu_);
            const auto at = answers_.find(key);
            if (at != answers_.end()) return at->second;
        }
        const int n = ask();   // (outside the lock: two threads may both ask, and get the same answer)
        std::lock_guard<std::mutex> lock(mu_);
        try {
            answers_.emplace(key, n);
        } catch (...) {   // (no memory: asked again next time; nothing is thrown through a C entry point)
        }
        return n;
    }

private:
    using Key = std::tuple<const void*, int, int, bool>;
    std::mutex mu_;
    std::map<Key, int> answers_;
};

}  // namespace lowbit
