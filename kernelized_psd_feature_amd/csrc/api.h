// Host helpers shared by the files that define the C ABI's entry points (kata_api.cpp,
// layer_api.cpp).  Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "device.h"
#include "kata.h"

namespace kata {

// Records `why` as this host thread's last error and returns s.
kata_status set_error(kata_status s, const std::string& why);
void clear_error(void);

// KATA_OK if the current device is a gfx950 (the code objects are built for nothing else).
kata_status check_device(void);

// A launch's hipError_t as a status, with `what` in the message.
kata_status launch_status(hipError_t e, const char* what);

// One timing record per scope when timing is on: the span from the start of the scope's first
// kernel to the end of its last (no record if it launched nothing).
struct Timed {
  int kind;
  LaunchTiming lt;
  LaunchTiming* prev = nullptr;
  bool open = false;
  Timed(int kind_, hipStream_t);
  ~Timed();
  Timed(const Timed&) = delete;
  Timed& operator=(const Timed&) = delete;
};

}  // namespace kata
