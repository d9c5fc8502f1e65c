// The dynamic shared-memory limit of kernels, per CUDA context.
//
// A launch above 48 KB needs the kernel's limit raised in the current context
// first.  The attribute belongs to (kernel, context), threads set it under one
// lock but launch outside of it, so it must never go down: a thread that has
// raised it for a long sequence launches after another one's short call.
#pragma once
#include <stddef.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

namespace rf2 {

class SmemLimits {
public:
    // Sees that `func` may take `bytes` in context `ctx` (have_ctx false: unknown,
    // set on every call); set(func, n) applies a limit and returns whether it
    // could.  Applied limits are the largest any context has asked for.
    template <typename Set>
    bool ensure(const void* func, bool have_ctx, unsigned long long ctx, size_t bytes, Set set)
    {
        std::lock_guard<std::mutex> lock(mu_);
        try {
            if (have_ctx) {
                const auto it = applied_.find({func, ctx});
                if (it != applied_.end() && it->second >= bytes) return true;
            }
            size_t& largest = largest_[func];
            const size_t n = std::max(largest, bytes);
            if (have_ctx) applied_[{func, ctx}];           // (allocates, if it has to, before the limit is set)
            if (!set(func, n)) return false;
            largest = n;
            if (have_ctx) applied_[{func, ctx}] = n;
            return true;
        } catch (...) {                                    // no memory for the tables
            return false;
        }
    }

private:
    std::mutex mu_;
    std::map<std::pair<const void*, unsigned long long>, size_t> applied_;
    std::map<const void*, size_t> largest_;
};

}  // namespace rf2
