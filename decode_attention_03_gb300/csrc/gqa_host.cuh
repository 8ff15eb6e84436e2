// Host helpers shared by the translation units of the C ABI.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

namespace gqa {

constexpr size_t kHeaderBytes = 256;        // status word (+ reserved) at the start of every workspace
constexpr uint64_t kDefaultTimeoutNs = 1000000000ull;
constexpr uint64_t kMinTimeoutNs = 5000000ull;

// The limit of a kernel's waits.  A CTA that gives one up waits as long for its own copies before it leaves its shared memory:
// a limit near the memory's latency would let it leave while they are on their way.
inline uint64_t wait_limit_ns(uint32_t timeout_us) {
  const uint64_t ns = (uint64_t)timeout_us * 1000ull;
  return timeout_us == 0 ? kDefaultTimeoutNs : (ns < kMinTimeoutNs ? kMinTimeoutNs : ns);
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The launches of one call hand partials on through its workspace, so that no other call's launches on it may come between
// them: host threads that share a stream and its workspace take turns.
inline std::mutex& turn_of(const void* ws) {
  constexpr int kTurns = 64;
  static std::mutex turns[kTurns];
  return turns[(reinterpret_cast<uintptr_t>(ws) >> 8) % kTurns];
}

// Launch with programmatic stream serialisation: the kernel may begin launching while the
// previous kernel in the stream finishes (it waits in griddepcontrol.wait before reading).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_smem(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t st,
                            int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), unsigned grid, unsigned block, cudaStream_t st, Args... args) {
  return launch_pdl_smem(kernel, dim3(grid, 1, 1), block, 0, st, 1, args...);
}

}  // namespace gqa
