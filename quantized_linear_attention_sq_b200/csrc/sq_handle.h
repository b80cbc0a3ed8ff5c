// sq_handle.h -- the handle behind include/sq.h, shared by the host sources
// that launch work on a state pool.
#pragma once
#include <cuda_runtime.h>

#include <vector>

#include "sq.h"
#include "sq_kernels.cuh"

namespace sqi {
// Default limit of the kernels' bounded waits (a stage's data, the partials buffer).
constexpr uint64_t kWaitNs = 2000000000ull;
}  // namespace sqi

struct sq_handle {
  sq_state_desc desc{};
  int d = 0;
  int device = 0;
  int num_sms = 0;
  // host copies of the layout
  std::vector<uint32_t> rec_off, rec_bytes;
  std::vector<uint16_t> row_off;
  std::vector<uint8_t> row_code;
  uint64_t slot_bytes = 0, pool_bytes = 0, max_rec = 0;
  // device tables (one allocation)
  void* dev_block = nullptr;
  sqk::Tables tables{};
  // launch configuration of the step kernel
  int step_grid = 0;
  int nstage = 0;
  uint32_t rec_cap = 0, stage_bytes = 0;
  uint64_t stage_rec = 0;  // largest record that goes through a stage
  size_t step_smem = 0;
  uint64_t launches = 0;
  uint64_t wait_ns = sqi::kWaitNs;  // limit of the kernels' bounded waits
  uint32_t test_extra_tx = 0;     // testing only (sq_test_stall_stage)
  // sq_decode_step_host: two device staging sets used in turn, the internal
  // stream their host-to-device copies run on, and the events that order
  // the copies after the step that last read a set.
  struct HostStage {
    void* block = nullptr;
    int32_t cap_B = 0;
    cudaEvent_t copied = nullptr;  // the set's inputs are on the device
    cudaEvent_t read = nullptr;    // the step that used the set has run
  };
  HostStage host_stage[2];
  cudaStream_t copy_stream = nullptr;
  uint64_t host_calls = 0;
  // sq_window_step: launch plan of the last window length used
  int win_W = 0, win_grid = 0;
  uint32_t win_smem = 0;
};
