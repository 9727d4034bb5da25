// gn_args.hpp -- what the API files of gn_ops.h and gn_join.h check arguments with: types, alignment,
// devices, sizes of rows and overlaps. Every function lives in an unnamed namespace.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gn_ops.h"

namespace {

bool dtype_ok(int d) { return d == GN_F32 || d == GN_BF16 || d == GN_F16; }
int64_t size_of(int d) { return d == GN_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(a - 1)) == 0; }
int launch_status(hipError_t e) { return e == hipSuccess ? GN_OK : GN_ERR_LAUNCH; }

// The device that owns p, or -1 if p is not device memory.
int device_of(const void* p)
{
    hipPointerAttribute_t attr;
    if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
        (void)hipGetLastError();
        return -1;
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return -1;
    return attr.device;
}

// Makes the device that owns p current for the duration of a call; a stream or another
// pointer argument of another device is refused.
class OnDeviceOf {
  public:
    // known: the device that the caller has seen every pointer and the stream to belong to, or
    // -1 (they are looked at here).
    explicit OnDeviceOf(int known = -1) : known_(known) {}
    int enter(const void* p, void* stream)
    {
        const int dev = known_ >= 0 ? known_ : device_of(p);
        int cur = -1;
        if (dev < 0 || hipGetDevice(&cur) != hipSuccess) return GN_ERR_DEVICE;
        if (stream && known_ < 0) {
            hipDevice_t sdev = -1;
            if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev) != hipSuccess) {
                (void)hipGetLastError();
                return GN_ERR_DEVICE;
            }
            if (sdev != dev) return GN_ERR_DEVICE;
        }
        if (cur != dev) {
            if (hipSetDevice(dev) != hipSuccess) return GN_ERR_DEVICE;
            prev_ = cur;
        }
        dev_ = dev;
        return GN_OK;
    }
    int holds(std::initializer_list<const void*> ptrs) const
    {
        if (known_ >= 0) return GN_OK;
        for (const void* p : ptrs)
            if (p && device_of(p) != dev_) return GN_ERR_DEVICE;
        return GN_OK;
    }
    ~OnDeviceOf()
    {
        if (prev_ >= 0) (void)hipSetDevice(prev_);
    }

  private:
    int known_, prev_ = -1, dev_ = -1;
};

// The bytes that an argument covers.
struct Span {
    uintptr_t b = 0, e = 0;
    Span() = default;
    Span(const void* p, int64_t bytes)
        : b(reinterpret_cast<uintptr_t>(p)), e(p ? reinterpret_cast<uintptr_t>(p) + uintptr_t(bytes) : 0)
    {
    }
    bool meets(const Span& o) const { return b < o.e && o.b < e; }
    bool is(const Span& o) const { return b == o.b && e == o.e; }
};

[[maybe_unused]] bool meets_any(const Span& s, std::initializer_list<Span> all)
{
    for (const Span& o : all)
        if (s.meets(o)) return true;
    return false;
}

// Rows of the largest launch, in workgroups (the threads of a launch stay below 2^32).
constexpr int64_t kMaxGroups = int64_t(1) << 21;

int rows_check(int64_t T, int64_t H, int64_t stride)
{
    if (T < 0 || H < 1 || H > GN_RMS_MAX_COLUMNS || stride < H) return GN_ERR_ROWS;
    // Offsets stay within 62 bits of bytes.
    if (T > 0 && (T > (int64_t(1) << 44) || stride > (int64_t(1) << 58) / T)) return GN_ERR_ROWS;
    return GN_OK;
}

// The bytes of T rows of H elements, `stride` apart.
int64_t rows_bytes(int64_t T, int64_t H, int64_t stride, int dt)
{
    return T > 0 ? ((T - 1) * stride + H) * size_of(dt) : 0;
}

const void* at(const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + bytes : nullptr; }
void* at(void* p, int64_t bytes) { return p ? static_cast<char*>(p) + bytes : nullptr; }

}  // namespace
