// Bookkeeping of the buffers that sherry_reserve sets aside per device (host),
// over the caller's functions: bool alloc(void**, size_t), void release(void*),
// bool zero(void*, size_t), bool sync(), true on success.
#pragma once

#include <cstddef>
#include <vector>

namespace sherry {

struct Workspace {
    void* ptr = nullptr;
    size_t bytes = 0;
    // smaller buffers of before that captured graphs may still use
    struct Kept {
        void* ptr;
        size_t bytes;
    };
    std::vector<Kept> kept;
};

// Grows a buffer to at least `bytes` (host-synchronous), zero-filled.  keep_old:
// the older buffer stays allocated, since captured graphs may hold its address
// (the split-K workspace: it grows at most four times, with the token tile, and
// all its sizes together are 33 MB); else it is freed once the device is idle.
template <class Alloc, class Release, class Zero, class Sync>
bool grow_reserved(Workspace& w, size_t bytes, bool keep_old, Alloc alloc, Release release, Zero zero, Sync sync)
{
    if (w.bytes >= bytes) return true;
    if (w.ptr && !keep_old) {
        if (!sync()) return false;
        release(w.ptr);
        w.ptr = nullptr;
        w.bytes = 0;
    }
    if (w.ptr) w.kept.reserve(w.kept.size() + 1);
    void* ptr = nullptr;
    if (!alloc(&ptr, bytes)) return false;
    if (!zero(ptr, bytes) || !sync()) {
        release(ptr);
        return false;
    }
    if (w.ptr) w.kept.push_back({w.ptr, w.bytes});
    w.ptr = ptr;
    w.bytes = bytes;
    return true;
}

// Zero-fills the buffer and those kept (host-synchronous).
template <class Zero, class Sync>
bool clear_reserved(const Workspace& w, Zero zero, Sync sync)
{
    if (!w.ptr) return true;
    bool ok = zero(w.ptr, w.bytes);
    for (const Workspace::Kept& k : w.kept) ok = ok && zero(k.ptr, k.bytes);
    return ok && sync();
}

}  // namespace sherry
