// Calls of the C entry points from host threads of their own, for tests (no interpreter between them).
#include <atomic>
#include <chrono>
#include <cstdint>
#include <thread>

#include "pagedattn.h"

namespace {

template <typename T>
T arg(int64_t v) {
  if constexpr (std::is_pointer_v<T>) return reinterpret_cast<T>(v);
  else return static_cast<T>(v);
}

template <typename... A, size_t... I>
pa_status spread(pa_status (*f)(A...), const int64_t* v, std::index_sequence<I...>) {
  return f(arg<A>(v[I])...);
}

template <typename... A>
pa_status invoke(pa_status (*)(A...), void* f, const int64_t* v) {
  return spread(reinterpret_cast<pa_status (*)(A...)>(f), v, std::index_sequence_for<A...>());
}

pa_status call(int which, void* f, const int64_t* v) {
  if (which == 0) return invoke(&pa_build_block_tables, f, v);
  if (which == 1) return invoke(&pa_select_pages, f, v);
  return invoke(&pa_sparse_paged_attention, f, v);
}

std::atomic<int> released{0}, entered{0};

}  // namespace

extern "C" {

// n calls with the arguments a (whole numbers and addresses, in order) and n with b, at once; the calls refused
int two_threads(int which, void* f, const int64_t* a, const int64_t* b, int n) {
  std::atomic<int> refused{0}, ready{0};
  auto loop = [&](const int64_t* v) {
    ++ready;
    while (ready < 2) {
    }
    for (int i = 0; i < n; ++i) refused += call(which, f, v) != PA_OK;
  };
  std::thread other(loop, a);
  loop(b);
  other.join();
  return refused;
}

// stands in for an entry point that takes long: waits until release() is called, two seconds at most
int slow_entry_point() {
  entered = 1;
  const auto end = std::chrono::steady_clock::now() + std::chrono::seconds(2);
  while (!released && std::chrono::steady_clock::now() < end) std::this_thread::yield();
  return released ? PA_OK : PA_ERR_CUDA;
}
int has_entered() { return entered; }
void release() { released = 1; }
void reset() { entered = released = 0; }
}
