// libkvq's host side over a stand-in for the CUDA runtime: no device, every launch recorded instead of run.
//
// The functions below take the place of the runtime's own (the program's symbols come first).  A kernel's dynamic shared
// memory is limited as on a device: 48 KB until cudaFuncSetAttribute says otherwise, and a launch above the limit fails.
//   fake_runtime limits   the limits that calls of different batches set must not depend on the batch
//   fake_runtime threads  two threads' first calls, the larger batch's setting overtaken by the smaller's; then all calls again
//   fake_runtime grid SMS the append's grid at batches 1 and 1024 of a device with SMS SMs: "batch blocks smem" lines
#include <cuda_runtime.h>

#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <mutex>
#include <set>
#include <string>
#include <thread>
#include <vector>

#include "../../include/kvq.h"

namespace {
std::mutex mu;
std::condition_variable cv;
std::map<const void*, size_t> limit;
std::map<const void*, std::set<size_t>> settings;
int sms = 152;
size_t park_above = 0;  // a setting above this waits, once done, until another one is done as well (or 2 s)
int sets = 0;
struct Launch {
  dim3 grid, block;
  size_t smem;
};
std::vector<Launch> launches;
thread_local Launch pending;

cudaError_t launch(const void* func, dim3 grid, dim3 block, size_t smem) {
  std::lock_guard<std::mutex> g(mu);
  const auto it = limit.find(func);
  if (smem > (it == limit.end() ? 49152 : it->second)) return cudaErrorInvalidValue;
  launches.push_back({grid, block, smem});
  return cudaSuccess;
}
thread_local cudaError_t last = cudaSuccess;
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? sms
       : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 227 * 1024
       : a == cudaDevAttrMaxSharedMemoryPerMultiprocessor ? 228 * 1024
       : a == cudaDevAttrReservedSharedMemoryPerBlock ? 1024
                                                      : 0;
  return *v ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int value) {
  if (a != cudaFuncAttributeMaxDynamicSharedMemorySize || value > 227 * 1024) return cudaErrorInvalidValue;
  std::unique_lock<std::mutex> g(mu);
  limit[f] = value;
  settings[f].insert(value);
  const int mine = ++sets;
  cv.notify_all();
  if (park_above && static_cast<size_t>(value) > park_above) cv.wait_for(g, std::chrono::seconds(2), [&] { return sets > mine; });
  return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, struct CUstream_st*) {
  pending = {grid, block, smem};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
  *grid = pending.grid;
  *block = pending.block;
  *smem = pending.smem;
  *static_cast<void**>(stream) = nullptr;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3 block, void**, size_t smem, cudaStream_t) {
  return last = launch(reinterpret_cast<const void*>(k), grid, block, smem);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  return last = launch(f, c->gridDim, c->blockDim, c->dynamicSmemBytes);
}
}

namespace {
void* const kFake = reinterpret_cast<void*>(4096);  // never dereferenced
kvq_cache cache(int fmt) {
  kvq_cache c;
  std::memset(&c, 0, sizeof c);
  c.k_fmt = c.v_fmt = fmt;
  c.num_kv_heads = 2;
  c.num_pages = 1 << 20;
  c.k_data = c.v_data = kFake;
  c.k_scale = c.v_scale = c.witness = static_cast<uint16_t*>(kFake);
  if (fmt == KVQ_FMT_BF16 || fmt == KVQ_FMT_E4M3) c.k_scale = c.v_scale = nullptr;
  return c;
}
const int32_t* const ints = static_cast<const int32_t*>(kFake);

kvq_status append(int fmt, int dtype, int batch) {
  const kvq_cache c = cache(fmt);
  return kvq_append_runs(&c, kFake, 256, kFake, 256, dtype, ints, batch, 64 * batch, ints, 64, ints, nullptr, nullptr);
}
kvq_status attn(int fmt, int dtype, int max_run, int batch) {
  const kvq_cache c = cache(fmt);
  return kvq_attn_runs(&c, kFake, 512, dtype, 4, ints, batch, max_run * batch, max_run, ints, 64, ints, 1.f, kFake, nullptr, kFake,
                       static_cast<size_t>(1) << 50, nullptr, nullptr);
}
kvq_status decode(int fmt, int dtype, int batch) {
  const kvq_cache c = cache(fmt);
  return kvq_decode_attn(&c, nullptr, 0, kFake, dtype, batch, 4, ints, 64, ints, 1.f, nullptr, static_cast<float*>(kFake), nullptr,
                         kFake, static_cast<size_t>(1) << 50, nullptr, nullptr);
}

struct Call {
  std::string name;
  std::function<kvq_status(int)> run;  // of a batch
};
std::vector<Call> calls() {
  std::vector<Call> v;
  for (int dt : {KVQ_DTYPE_F32, KVQ_DTYPE_BF16}) {
    const std::string t = dt == KVQ_DTYPE_F32 ? " f32" : " bf16";
    for (int f : {KVQ_FMT_E4M3_PAGE, KVQ_FMT_INT8_PAGE}) {
      const std::string n = (f == KVQ_FMT_E4M3_PAGE ? "e4m3p" : "int8p") + t;
      v.push_back({"append " + n, [=](int b) { return append(f, dt, b); }});
      for (int run : {1, 6, 40})
        v.push_back({"attn " + n + " " + std::to_string(run), [=](int b) { return attn(f, dt, run, b); }});
    }
    for (int f : {KVQ_FMT_BF16, KVQ_FMT_E4M3, KVQ_FMT_E4M3_SCALED, KVQ_FMT_INT8_DITHER, KVQ_FMT_INT8_DITHER_G32})
      v.push_back({"decode " + std::to_string(f) + t, [=](int b) { return decode(f, dt, b); }});
  }
  return v;
}
void reset() {
  std::lock_guard<std::mutex> g(mu);
  settings.clear();
}
constexpr int kSmall = 1, kLarge = 1024;
}  // namespace

int main(int argc, char** argv) {
  const std::string mode = argc > 1 ? argv[1] : "";
  int bad = 0;
  auto expect = [&](const Call& c, int batch, kvq_status s) {
    if (s != KVQ_OK) std::printf("%s, batch %d: %s\n", c.name.c_str(), batch, kvq_status_string(s)), ++bad;
  };
  if (mode == "limits") {
    for (const Call& c : calls()) {
      reset();
      for (int b : {kSmall, 300, kLarge}) expect(c, b, c.run(b));
      for (const auto& s : settings)
        if (s.second.size() > 1) std::printf("%s: %zu different limits for one kernel\n", c.name.c_str(), s.second.size()), ++bad;
    }
  } else if (mode == "threads") {
    for (const Call& c : calls()) {
      // what this kernel is set to for the small batch is not known before, so every setting parks until a second one is done
      park_above = 1;
      kvq_status s1 = KVQ_OK, s2 = KVQ_OK;
      std::thread large([&] { s1 = c.run(kLarge); });
      {  // the larger one's setting is done, its thread not yet past it
        std::unique_lock<std::mutex> g(mu);
        const int before = sets;
        cv.wait_for(g, std::chrono::milliseconds(200), [&] { return sets > before; });
        park_above = 0;
      }
      std::thread small([&] { s2 = c.run(kSmall); });
      small.join();
      large.join();
      expect(c, kSmall, s2);
      expect(c, kLarge, s1);
      expect(c, kLarge, c.run(kLarge));  // and ever after
    }
  } else if (mode == "grid") {
    sms = std::atoi(argv[2]);
    for (int dt : {KVQ_DTYPE_F32, KVQ_DTYPE_BF16})
      for (int b : {kSmall, kLarge}) {
        launches.clear();
        const kvq_cache c = cache(KVQ_FMT_INT8_PAGE);
        if (kvq_append_runs(&c, kFake, 256, kFake, 256, dt, ints, b, 1 << 20, ints, 1 << 16, ints, nullptr, nullptr) != KVQ_OK) ++bad;
        else std::printf("%d %d %u %zu\n", dt, b, launches.at(0).grid.x, launches.at(0).smem);
      }
  } else {
    return 2;
  }
  return bad ? 1 : 0;
}
