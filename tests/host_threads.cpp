// Host threads that share a stream, without a GPU: this program defines the HIP calls that libskgemm.so makes (its own
// definitions come before the runtime's), lets two threads call the library on one stream, and checks that one call's
// launches follow each other: nothing another call launches or frees comes between a call's first launch and its
// last, since they hand data on in the stream's scratch.  Argument: the calls to make.  Exit status 0 where that holds.

#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>

#include <atomic>
#include <chrono>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "../include/sk_gemm.h"

namespace {

struct Event {
  int call;
  char what;   // 'L' a launch, 'F' a buffer given back
};
std::mutex mu;
std::vector<Event> events;
std::atomic<int> calls{0};
thread_local int this_call = -1;

void note(char what) {
  {
    std::lock_guard<std::mutex> lk(mu);
    events.push_back({this_call, what});
  }
  std::this_thread::sleep_for(std::chrono::microseconds(300));   // time for the other thread
}

}  // namespace

extern "C" {

hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {   // (a macro for the runtime's name of it)
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  p->multiProcessorCount = 256;
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t n) {   // addresses only: nothing reads them
  static std::atomic<uintptr_t> next{(uintptr_t)1 << 40};
  *p = (void*)next.fetch_add((n + 4095) & ~(size_t)4095);
  return hipSuccess;
}
hipError_t hipFree(void*) { return note('F'), hipSuccess; }
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipMemsetAsync(void*, int, size_t, hipStream_t) { return hipSuccess; }
hipError_t hipMemcpy(void* d, const void*, size_t n, hipMemcpyKind) { return std::memset(d, 0, n), hipSuccess; }
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) { return *s = hipStreamCaptureStatusNone, hipSuccess; }
hipError_t hipExtStreamGetCUMask(hipStream_t, uint32_t words, uint32_t* mask) {   // every stream but NULL: one unit
  std::memset(mask, 0, 4 * words);
  return mask[0] = 1, hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
// (the two halves of a <<<...>>> launch: the second is the first's own thread's)
thread_local struct {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
} config;
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  return config = {grid, block, lds, stream}, hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  return *grid = config.grid, *block = config.block, *lds = config.lds, *stream = config.stream, hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { return note('L'), hipSuccess; }

}  // extern "C"

namespace {

uint8_t* at(int i) { return (uint8_t*)(((uintptr_t)1 << 44) + ((uintptr_t)i << 36)); }   // operands, far apart

sk_status block_backward(int size, int cap) {
  return sk_gemm_fp8_block_backward(at(0), at(1), (float*)at(2), at(3), (float*)at(4), at(5), at(6), at(7), 128 + 256 * size,
                                    384, 512, cap, nullptr);
}
sk_status bf16_backward(int size) {
  return sk_gemm_bf16_backward(at(0), at(1), at(2), at(3), at(4), at(5), 128 + 256 * size, 384, 512, 0, nullptr);
}
sk_status norm_backward(int size, int64_t D = 1024, void* stream = nullptr) {
  sk_norm_grad_args a;
  std::memset(&a, 0, sizeof(a));
  a.dout = at(0);
  a.h = at(1);
  a.weight = at(2);
  a.rstd = (float*)at(3);
  a.dx = at(4);
  a.dresidual = at(5);
  a.dweight = at(6);
  a.T = 16 + 32 * size;
  a.D = D;
  a.stream = stream;
  return sk_norm_backward(&a);
}
sk_status relaid_scales(int size) {
  sk_gemm_args g;
  std::memset(&g, 0, sizeof(g));
  g.dtype = SK_MXFP4;
  g.policy = SK_POLICY_HYBRID;
  g.A = at(0);
  g.B = at(1);
  g.A_scale = at(2);
  g.B_scale = at(3);
  g.C = at(4);
  g.M = 256 + 256 * size;
  g.N = 512;
  g.K = 1024;
  g.debug_flags = SK_DEBUG_RELAYOUT;
  g.drop_signal_wg = -1;
  return sk_gemm_ex(&g);
}
sk_status release() {
  sk_release_workspace();
  std::this_thread::sleep_for(std::chrono::milliseconds(1));
  return SK_OK;
}

}  // namespace

int main(int argc, char** argv) {
  typedef std::function<sk_status(int)> Call;   // (of a size)
  const std::map<std::string, std::vector<Call>> scenes = {
      {"block_backward", {[](int s) { return block_backward(s, 0); }, [](int s) { return block_backward(s + 1, 0); }}},
      {"block_backward_capped", {[](int s) { return block_backward(s, 7); }, [](int s) { return block_backward(s + 1, 7); }}},
      {"norm_backward", {[](int s) { return norm_backward(s); }, [](int s) { return norm_backward(s + 1); }}},
      {"bf16_backward", {bf16_backward, [](int s) { return bf16_backward(s + 1); }}},
      {"block_and_bf16", {[](int s) { return block_backward(s, 0); }, bf16_backward}},
      {"block_and_norm", {[](int s) { return block_backward(s, 0); }, [](int s) { return norm_backward(s); }}},
      {"relaid_scales", {relaid_scales, [](int s) { return relaid_scales(s + 1); }}},
      // rows of 64 to 1024 threads on a stream held to one compute unit
      {"one_unit", {[](int s) { return norm_backward(s, 300 << s, at(9)); }, [](int s) { return norm_backward(s, 9000, at(9)); }}},
      {"release", {[](int s) { return block_backward(s, 0); }, [](int) { return release(); }}},
  };
  const auto scene = argc == 2 ? scenes.find(argv[1]) : scenes.end();
  if (scene == scenes.end()) return std::fprintf(stderr, "unknown calls\n"), 2;
  std::atomic<int> ready{0}, bad{0};
  std::vector<std::thread> threads;
  for (const Call& call : scene->second)
    threads.emplace_back([&, call] {
      ++ready;
      while (ready < (int)scene->second.size()) std::this_thread::yield();
      for (int i = 0; i < 40; ++i) {
        this_call = calls++;
        const sk_status st = call(i % 4 * 2);
        if (st != SK_OK) bad = (int)st;
      }
    });
  for (std::thread& t : threads) t.join();
  if (bad) return std::fprintf(stderr, "a call returned %d\n", (int)bad), 2;

  std::map<int, std::pair<size_t, size_t>> span;   // of a call's launches
  for (size_t i = 0; i < events.size(); ++i)
    if (events[i].what == 'L') span.emplace(events[i].call, std::make_pair(i, i)).first->second.second = i;
  int between = 0, several = 0;
  for (const auto& s : span) {
    several += s.second.first != s.second.second;
    for (size_t i = s.second.first; i <= s.second.second; ++i) between += events[i].call != s.first;
  }
  std::printf("%zu calls launched, %d of them several times, %d events of other calls in between\n", span.size(), several, between);
  if (!several) return std::fprintf(stderr, "no call launched more than once: nothing was tested\n"), 2;
  return between != 0;
}
