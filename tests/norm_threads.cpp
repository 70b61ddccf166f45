// Host threads that call the gated sum with norm, or its gradient, at the same time; the test
// hands over the library's entry points and the arrays.
#include <atomic>
#include <thread>
#include <vector>

#include "nabla.h"

extern "C" {

struct NormCall {
  const void *in[4];  // forward: x, u; backward: s, u, dsum, dy
  void *out[2];       // s, y; or dx, du
  const void *weight, *post_weight;  // or null
  void *dweight, *dpost_weight, *workspace;
  size_t ws_bytes;
  nabla_stream_t stream;
  int S, C, dt, grad;
};

using Forward = decltype(&nabla_block_norm);
using Backward = decltype(&nabla_block_norm_bwd);

// Every call from a thread of its own, `times` times.  Returns the last error, or 0.
int norm_threads(Forward fwd, Backward bwd, const NormCall *calls, int n, int times) {
  std::atomic<int> waiting{n}, error{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < n; ++t)
    threads.emplace_back([&, t] {
      const NormCall &c = calls[t];
      const auto dt = static_cast<nabla_dtype>(c.dt);
      waiting.fetch_sub(1);
      while (waiting.load() > 0) std::this_thread::yield();
      for (int i = 0; i < times; ++i) {
        const nabla_status e =
            c.grad ? bwd(c.in[0], nullptr, c.in[1], nullptr, c.in[2], nullptr, c.in[3], nullptr, dt,
                         1, c.S, c.C, NABLA_NORM_LAYER, NABLA_NORM_RMS, c.weight, c.post_weight,
                         NABLA_F32, nullptr, 0, nullptr, 0, NABLA_F32, 1, 1.f, 1e-6f, c.out[0],
                         nullptr, c.out[1], nullptr, nullptr, nullptr, nullptr, c.dweight,
                         c.dpost_weight, c.workspace, c.ws_bytes, c.stream)
                   : fwd(c.in[0], nullptr, c.in[1], nullptr, dt, 1, c.S, c.C, NABLA_NORM_LAYER,
                         NABLA_NORM_RMS, c.weight, c.post_weight, NABLA_F32, nullptr, 0, nullptr, 0,
                         nullptr, 0, NABLA_F32, 1, 1.f, 1e-6f, c.out[0], nullptr, c.out[1], nullptr,
                         c.stream);
        if (e != NABLA_OK) error.store(e);
      }
    });
  for (std::thread &t : threads) t.join();
  return error.load();
}

}  // extern "C"
