// launches.h -- launch accounting shared by the entry points.
#pragma once

#include <stdint.h>

namespace gsa {

// Records the launches of this thread's last successful call (gsa_last_launch_count).
void set_last_launches(int32_t n);

}  // namespace gsa
