// host_common.h -- host-side pieces shared by the files that define entry points
// of include/apex_attn.h: RoPE frequencies, tensor maps and the per-device state.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/apex_attn.h"
#include "kernel_params.h"

namespace apex {

constexpr int kMaxSeq = 1 << 24;

// RoPE frequency parameters: base and the YaRN scaling (s <= 1: none).
struct RopeFreq {
    float base, yarn_s, beta_fast, beta_slow;
    bool operator==(const RopeFreq &o) const
    {
        return base == o.base && yarn_s == o.yarn_s && beta_fast == o.beta_fast && beta_slow == o.beta_slow;
    }
};

// theta_i of a d_h-dimensional RoPE vector (Part 1, §4.3, §5.3-§5.4)
double rope_frequency(int i, int d_h, const RopeFreq &f);

// Options -> frequency parameters, with the documented defaults; false when invalid.
bool freq_of(const apex_attn_options &o, RopeFreq *f);

// 3-D bf16 map over a dense [outer][rows][d_h] tensor, 128-byte swizzle, box
// {64 dims, box_rows, box_outer}; out-of-range elements read as zero.
bool make_map(CUtensorMap *m, const void *base, int d_h, int rows, int outer, int box_rows, int box_outer);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool supported_group(int G) { return G == 1 || G == 2 || G == 4 || G == 8 || G == 16; }

// The current device, initialised, with its lock held (calls on one device
// serialise while they enqueue); status is APEX_OK or the error to return.
struct DeviceScope {
    apex_status status;
    int sm_count = 0;
    WaitCtl wait{nullptr, 0};
    std::unique_lock<std::mutex> lock;
    DeviceScope();
};

}  // namespace apex
