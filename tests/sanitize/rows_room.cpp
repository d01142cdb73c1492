// The rows of v that the adapters' first product writes, over all parts of K, against
// the room of the workspace.  Prints "N sizes fit" and exits 0, or the first size that
// does not.
#include <stdio.h>

#include <initializer_list>

#include "../../packed_int4_convrot_amd/csrc/rows_launch.h"

int main()
{
    long sizes = 0;
    for (int64_t K = 64; K <= 32768; K += K < 2560 ? 64 : 1920)
        for (int64_t R = 8; R <= 256; R += 8)
            for (int64_t L : {1, 2, 3, 7, 15, 16, 17, 63, 64, 1000})
                for (int64_t M = 1; M < 20000; M += M < 1100 ? 1 : 57) {
                    ++sizes;
                    if (ck::lora_splits(M, K, R, L) * M > ck::lora_room_rows(M, K)) {
                        printf("M=%ld K=%ld R=%ld L=%ld: too little room\n", (long)M, (long)K, (long)R, (long)L);
                        return 1;
                    }
                }
    printf("%ld sizes fit\n", sizes);
    return 0;
}
