// c_call_threads.cpp -- calls of a C entry point (handle, arguments) from several host threads at once, without an
// interpreter's lock between them.
#include <atomic>
#include <thread>
#include <vector>

// Thread i calls fns[i](handles[i], args[i]) `times` times; returns the first code that is not 0, or 0.
extern "C" int call_at_once(int threads, int times, int (**fns)(void*, void*), void** handles, void** args) {
  std::atomic<int> ready{0}, code{0};
  std::vector<std::thread> all;
  for (int i = 0; i < threads; ++i)
    all.emplace_back([&, i] {
      ready.fetch_add(1);
      while (ready.load() < threads) std::this_thread::yield();
      for (int k = 0; k < times && code.load(std::memory_order_relaxed) == 0; ++k) {
        const int rc = fns[i](handles[i], args[i]);
        if (rc) code.store(rc);
      }
    });
  for (auto& t : all) t.join();
  return code.load();
}
