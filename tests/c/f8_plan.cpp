// Prints how an 8-bit floating-point product of each "M N K E experts sms" of the input is run:
// "columns cluster bn ctas runs tiles".
#include <stdio.h>

#include "h32_f8_plan.h"

int main() {
    long long M, N, K, E;
    int experts, sms;
    while (scanf("%lld %lld %lld %lld %d %d", &M, &N, &K, &E, &experts, &sms) == 6) {
        const h32::F8Plan p = h32::plan_f8(M, N, K, E, experts != 0, sms);
        printf("%d %d %d %d %d %lld\n", p.columns, p.cluster, p.bn, p.ctas, p.runs, static_cast<long long>(p.tiles));
    }
    return 0;
}
