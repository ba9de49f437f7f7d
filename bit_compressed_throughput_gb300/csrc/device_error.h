// What the device error words of the kernel families say, as a status and a message (host code
// without CUDA, so that its tests run anywhere).
#pragma once
#include <string>

#include "../../include/fg.h"
#include "ragged.cuh"

namespace fg {

struct DeviceErrorWord {
  const char* family;
  unsigned int bits;
};

// FG_OK when every word is 0; FG_ERR_TIMEOUT when a wait ran out, with every family that it
// happened to in the message and an extent that did not fit too, since reading the words clears
// them; FG_ERR_CAPACITY for an extent alone.
inline int device_error_status(const DeviceErrorWord* words, int n, std::string* message) {
  std::string waits, extents;
  for (int i = 0; i < n; ++i) {
    const unsigned int wait = words[i].bits & ~kErrExtent;
    if (wait)
      waits += std::string(waits.empty() ? "" : ", ") + words[i].family + " flag " +
               std::to_string(wait);
    if (words[i].bits & kErrExtent)
      extents += std::string(extents.empty() ? "" : ", ") + words[i].family;
  }
  if (waits.empty() && extents.empty()) return FG_OK;
  message->clear();
  if (!waits.empty()) *message = "bounded device wait timed out (" + waits + ")";
  if (!extents.empty())
    *message += std::string(waits.empty() ? "" : "; ") +
                "a length, position or row offset in a device array does not fit its buffers (" +
                extents + ")";
  return waits.empty() ? FG_ERR_CAPACITY : FG_ERR_TIMEOUT;
}

}  // namespace fg
