// Questions to the runtime that the FP8 launches ask once.  Host code only, no
// CUDA headers, so that it can be tested by itself.
#pragma once
#include <atomic>

namespace cql {

// The answer of `ask(int& n) -> int` (0: success) once it has succeeded; a failure
// is returned and forgotten, so that the next call asks again.
class KeptAnswer {
 public:
  template <class Ask>
  int get(int& n, Ask ask) {
    n = kept_.load(std::memory_order_relaxed) - 1;
    if (n >= 0) return 0;
    const int e = ask(n);
    if (e == 0) kept_.store(n + 1, std::memory_order_relaxed);
    return e;
  }

 private:
  std::atomic<int> kept_{0};                      // one more than the answer, 0 until there is one
};

// setmaxnreg draws on the registers that a block was launched with: whether `regs`
// a thread of `threads` hold the roles' shares, `sum` together, and are no fewer than
// `dec`, the largest share that a role shrinks to.  Otherwise an increase would wait
// for good.
constexpr bool register_split_fits(int regs, int threads, int sum, int dec) {
  return regs * threads >= sum && regs >= dec;
}

}  // namespace cql
