// A number that is asked for until there is an answer, and kept from then on.
#pragma once

#include <atomic>

namespace h32 {

// `*out` = what `ask(int *)`, 0 where it succeeds, once said (never 0); its error otherwise, and the
// next call asks again.
template <typename Ask>
auto ask_once(std::atomic<int> &known, Ask ask, int *out) -> decltype(ask(out)) {
    *out = known.load(std::memory_order_relaxed);
    if (*out != 0) return {};
    const auto e = ask(out);
    if (e == decltype(ask(out)){}) known.store(*out, std::memory_order_relaxed);
    return e;
}

}  // namespace h32
