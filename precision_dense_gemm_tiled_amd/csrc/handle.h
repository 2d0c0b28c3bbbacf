// The handle behind mpgemm_handle_t and the device guard of its calls.
#pragma once

#include <hip/hip_runtime.h>

#include "mpgemm_internal.h"

struct mpgemm_ctx {
    int device;
    int cu_count;
    int forced_tile_cfg;   // -1: heuristic; else a TileCfg index (MPGEMM_TILE_CFG)
    int forced_w4a16_cfg;  // -1: heuristic; else a W4A16Cfg index (MPGEMM_W4A16_CFG)
    int streamk_mode;      // mpg::StreamKMode (MPGEMM_STREAMK=0/1 forces it off/on)
    // One device buffer of partial sums, used by the weight-only path's K
    // split and by stream-K tile GEMMs (calls sharing a handle are serialized
    // by the caller), and the stream-K arrival counters (zero between calls).
    mpg::W4A16Workspace ws;
    mpg::TileWorkspace tile_ws;
};

namespace mpg {

// Makes the handle's device current for the duration of a call and restores
// the caller's current device afterwards.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int device) {
        if (hipGetDevice(&prev) != hipSuccess) {
            prev = -1;
            return;
        }
        ok = prev == device || hipSetDevice(device) == hipSuccess;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev)
            (void)hipSetDevice(prev);
    }
};

}  // namespace mpg
