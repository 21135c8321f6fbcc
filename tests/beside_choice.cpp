/* Prints how the log probabilities and the adapters split a call's work, by the
 * library's own rules.  Reads lines "logprobs M V" or "lora M N K r"; prints
 * "threads segments group_segments groups parts part_segments" for the first and
 * "few fused shrink_slots expand_slots product_rows" for the second. */
#include <stdio.h>
#include <string.h>

#include "beside_choice.hpp"

int main()
{
    char op[16];
    long m, n, k, r;
    while (scanf("%15s", op) == 1) {
        if (!strcmp(op, "logprobs") && scanf("%ld %ld", &m, &n) == 2) {
            const moe::LogprobPlan p = moe::logprob_plan(m, (int)n);
            printf("%d %d %d %d %d %d\n", p.threads, p.segments, p.group_segments, p.groups, p.parts, p.part_segments);
        } else if (!strcmp(op, "lora") && scanf("%ld %ld %ld %ld", &m, &n, &k, &r) == 4) {
            const moe::LoraPlan p = moe::lora_plan(m, n, k, (int)r);
            printf("%d %d %d %d %ld\n", p.few, p.fused, p.shrink_slots, p.expand_slots, (long)moe::lora_product_rows(n));
        } else {
            return 1;
        }
    }
    return 0;
}
