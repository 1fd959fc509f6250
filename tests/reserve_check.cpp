// Host-side check of the reserved buffers (reserve.h) over a fake allocator:
// growing keeps or frees the older buffer, a reset clears every buffer that a
// captured graph may still use, failures leave the buffer as it was.
// Prints "ok" and exits 0, or prints the failed line and exits 1.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>

#include "reserve.h"

static std::set<void*> live;
static int syncs = 0;
static bool fail_alloc = false, fail_zero = false;

static bool alloc(void** p, size_t n)
{
    if (fail_alloc) return false;
    *p = std::malloc(n);
    std::memset(*p, 0x5a, n);
    live.insert(*p);
    return true;
}
static void release(void* p)
{
    live.erase(p);
    std::free(p);
}
static bool zero(void* p, size_t n)
{
    if (fail_zero || !live.count(p)) return false;
    std::memset(p, 0, n);
    return true;
}
static bool wait_idle() { return ++syncs, true; }

static bool grow(sherry::Workspace& w, size_t bytes, bool keep_old)
{
    return sherry::grow_reserved(w, bytes, keep_old, alloc, release, zero, wait_idle);
}
static bool clear(sherry::Workspace& w) { return sherry::clear_reserved(w, zero, wait_idle); }

static bool all_zero(const void* p, size_t n)
{
    for (size_t i = 0; i < n; ++i)
        if (static_cast<const unsigned char*>(p)[i]) return false;
    return true;
}

#define CHECK(c)                                              \
    do {                                                      \
        if (!(c)) return std::printf("%d: " #c "\n", __LINE__), 1; \
    } while (0)

int main()
{
    using namespace sherry;
    Workspace w;
    CHECK(clear(w));
    CHECK(grow(w, 64, true) && all_zero(w.ptr, 64));
    void* first = w.ptr;
    CHECK(grow(w, 32, true) && w.ptr == first && w.bytes == 64);
    CHECK(grow(w, 128, true) && w.ptr != first && live.count(first));
    void* second = w.ptr;
    CHECK(grow(w, 256, true) && live.size() == 3);
    // a launch that gave up left words behind in each
    std::memset(first, 1, 64);
    std::memset(second, 1, 128);
    std::memset(w.ptr, 1, 256);
    const int before = syncs;
    CHECK(clear(w) && syncs > before);
    CHECK(all_zero(first, 64) && all_zero(second, 128) && all_zero(w.ptr, 256));

    void* third = w.ptr;
    fail_alloc = true;
    CHECK(!grow(w, 512, true) && w.ptr == third && w.bytes == 256);
    fail_alloc = false;
    fail_zero = true;
    CHECK(!grow(w, 512, true) && w.ptr == third && live.size() == 3);
    CHECK(!clear(w));
    fail_zero = false;

    Workspace a;
    CHECK(grow(a, 64, false));
    CHECK(grow(a, 128, false) && a.kept.empty() && live.size() == 4);
    fail_alloc = true;
    CHECK(!grow(a, 256, false) && !a.ptr && a.bytes == 0);
    std::printf("ok\n");
    return 0;
}
