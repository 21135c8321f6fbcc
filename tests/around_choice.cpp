/* Prints which kernel variant a call's sizes choose, by the library's own rules.
 * Reads lines "norm M H", "quant rows cols" or "int8 M N K"; prints a line
 * "variant" for each, for the tiles of the int8 product "variant steps ring
 * direct": the whole steps of K, those its ring holds, and whether rows are a
 * multiple of 16 codes and go straight to LDS.  "count" prints the number of
 * variants of the three. */
#include <stdio.h>
#include <string.h>

#include "around_choice.hpp"

int main()
{
    char op[16];
    long a, b, k;
    while (scanf("%15s", op) == 1) {
        if (!strcmp(op, "count")) {
            printf("%d %d %d\n", (int)moe::kNormVariants, (int)moe::kQuantVariants, (int)moe::kInt8Variants);
        } else if (!strcmp(op, "norm") && scanf("%ld %ld", &a, &b) == 2) {
            printf("%d\n", (int)moe::norm_variant(a, (int)b));
        } else if (!strcmp(op, "quant") && scanf("%ld %ld", &a, &b) == 2) {
            printf("%d\n", (int)moe::quant_variant(a, b));
        } else if (!strcmp(op, "int8") && scanf("%ld %ld %ld", &a, &b, &k) == 3) {
            const int v = (int)moe::int8_variant(a, b, k);
            if (v < moe::kTiles) {
                const moe::TileShape& t = moe::kTileShapes[v];
                printf("%d %ld %d %d\n", v, k / t.bk, t.ring, k % 16 == 0 ? 1 : 0);
            } else {
                printf("%d\n", v);
            }
        } else {
            return 1;
        }
    }
    return 0;
}
