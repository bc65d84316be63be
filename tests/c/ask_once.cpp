// A query that fails twice, then answers: the failures are reported and not kept, the answer is.
#include <stdio.h>

#include "h32_once.h"

enum Error { kOk = 0, kBusy = 7 };

int main() {
    std::atomic<int> known{0};
    int asked = 0, out = 0;
    const auto ask = [&](int *v) {
        *v = ++asked < 3 ? -1 : 168;
        return asked < 3 ? kBusy : kOk;
    };
    for (int call = 0; call < 5; ++call) {
        const Error e = h32::ask_once(known, ask, &out);
        if (e != (call < 2 ? kBusy : kOk) || (e == kOk && out != 168)) return 1;
    }
    return asked == 3 ? 0 : 2;
}
