// The operational wait limit set by sparse_attn_set_wait_limit, in ns (0: the
// kernels' default).
#pragma once

#include <cstdint>

namespace sa_host {
uint64_t wait_limit();
}
