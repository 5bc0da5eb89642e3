// status.cuh -- the bits of the device status word (cbs_read_device_status).
#pragma once

namespace cbs {

// A bounded wait ran out; a device array of a token operator's call (page
// table, lengths, starts) held a value out of range.
constexpr unsigned int kStatusTimeout = 1u, kStatusBadIndex = 2u;

}  // namespace cbs
