// The device check shared by the C-ABI translation units of libqmv.so.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "../../include/qmv.h"

namespace qmv {

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// QMV_OK if the current device is gfx950.  Cached per device: 1 = gfx950,
// 2 = something else.
inline int check_device() {
    static std::atomic<int> dev_ok[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return QMV_EUNSUPPORTED_DEVICE;
    if (dev < 64) {
        const int v = dev_ok[dev].load(std::memory_order_relaxed);
        if (v) return v == 1 ? QMV_OK : QMV_EUNSUPPORTED_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return QMV_EUNSUPPORTED_DEVICE;
    const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) dev_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? QMV_OK : QMV_EUNSUPPORTED_DEVICE;
}

inline int launched(int hip_rc) { return hip_rc == 0 ? QMV_OK : QMV_ELAUNCH; }

}  // namespace qmv
