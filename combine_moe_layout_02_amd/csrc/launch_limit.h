// What one launch can number.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int64_t kMaxLaunchThreads = UINT32_MAX;  // threads of one launch along x

}  // namespace moe
