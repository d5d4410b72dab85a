// null_launcher.cpp -- Launcher and OptimDevice that enqueue nothing. Linked only into the
// host-only test library so the plan and the readiness state machine can be
// exercised on a machine without a GPU. It moves no data: gradients are left
// untouched, so it is never a substitute for the HIP launcher.
#include <atomic>

#include "core.hpp"
#include "optim.hpp"

namespace {
// Joins requested by every null launcher of the process (read by the host
// tests through ddpb_hostonly_join_count).
std::atomic<long long> g_joins{0};
// Whether the null streams pretend to be captured (ddpb_hostonly_set_capture).
std::atomic<int> g_capture{0};
}  // namespace

namespace ddpb {
namespace {

class NullLauncher final : public Launcher {
 public:
  int bind(const Plan&, const BindArgs&, std::string*) override { return kOk; }
  int launch(int32_t, int32_t, int64_t, std::string*) override { return kOk; }
  int join(std::string*) override {
    ++g_joins;
    return kOk;
  }
  bool in_capture() override { return g_capture != 0; }
  int accumulate(void* const*, int32_t, bool, std::string*) override { return kOk; }
  int read_stamps(const std::vector<LaunchRecord>& log, std::vector<int64_t>* t0, std::vector<int64_t>* t1,
                  std::string*) override {
    t0->assign(log.size(), 0);
    t1->assign(log.size(), 0);
    return kOk;
  }
  int read_times(int64_t, const std::vector<LaunchRecord>&, std::vector<float>*, std::vector<float>*,
                 std::string* err) override {
    *err = "no device in the host-only test build";
    return kErrState;
  }
  void set_max_blocks(int32_t) override {}
  int set_workgroups_per_cu(int32_t, std::string*) override { return kOk; }
  int set_used(const uint8_t*, const uint8_t*, std::string*) override { return kOk; }
  int set_sync_step(void* const*, int32_t, bool, std::string*) override { return kOk; }
  int clock_hz(int64_t* hz, std::string*) override {
    *hz = 0;
    return kOk;
  }
};

class NullOptimDevice final : public OptimDevice {
 public:
  int current(int* device, std::string*) override {
    *device = 0;
    return kOk;
  }
  int upload(int, void*, void*, const void*, size_t, std::string*) override { return kOk; }
  int download(int, void*, void*, const void*, size_t, std::string* err) override {
    *err = "no device in the host-only test build";
    return kErrState;
  }
  int norm(const NormLaunch&, std::string*) override { return kOk; }
  int adamw(const AdamwLaunch&, std::string*) override { return kOk; }
};

}  // namespace

OptimDevice* optim_device() {
  static NullOptimDevice d;
  return &d;
}

std::unique_ptr<Launcher> make_launcher() { return std::make_unique<NullLauncher>(); }

}  // namespace ddpb

// Host-only test build: how many times the state machine asked a launcher to
// make the compute stream wait for the side streams.
extern "C" long long ddpb_hostonly_join_count(void) { return g_joins.load(); }

// Host-only test build: from here on the null launcher reports its stream as
// being captured (or not).
extern "C" void ddpb_hostonly_set_capture(int yes) { g_capture = yes; }
