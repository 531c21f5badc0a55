// largest_set.h -- a setting that has to reach at least some size and is only ever raised
// (host side): the dynamic shared memory limit of a kernel, per kernel and context.
//
// A call that finds its size covered skips the setter.  Finding, setting and remembering
// are one step under a lock: a thread that sets a smaller size beside one that sets a
// larger would otherwise leave the smaller set and the larger remembered, and every
// later launch of the larger size would fail.
#pragma once
#include <algorithm>
#include <map>
#include <mutex>
#include <new>

namespace moe {

template <class Key>
class LargestSet {
   public:
    // Whether the setting of `key` is at least `size`, after set(size or the largest so far)
    // where needed.  forget: earlier calls do not count (the setting may be gone).
    template <class Set>
    bool ensure(const Key &key, int size, bool forget, Set &&set) {
        std::lock_guard<std::mutex> lock(mu_);
        int *largest;
        try {
            largest = &done_[key];
        } catch (const std::bad_alloc &) {
            return false;
        }
        if (!forget && *largest >= size) return true;
        const int to = std::max(*largest, size);
        if (!set(to)) return false;
        *largest = to;
        return true;
    }

   private:
    std::mutex mu_;
    std::map<Key, int> done_;
};

}  // namespace moe
