// Prints what the sizes on its standard input choose (csrc/plan.hpp), a line each:
//   experts ROWS EXPERTS N K             the kernel, and the gradient's rows a piece
//   lora M N K ADAPTERS RANK             the kernel, the gradient's rows a tile, and for the product and the
//                                        gradient: parts of the long axis of h (and u), of the output, of the rows
#include <cstdio>
#include <cstring>

#include "plan.hpp"

int main()
{
    static const char *const experts[] = {"stream1", "stream2", "skinny", "tile64", "tile128", "tile256"};
    static const char *const lora[] = {"skinny", "tile64", "tile128", "tile256"};
    char word[16];
    while (std::scanf("%15s", word) == 1) {
        long long a[5] = {};
        const int n = std::strcmp(word, "experts") == 0 ? 4 : 5;
        for (int i = 0; i < n; ++i)
            if (std::scanf("%lld", &a[i]) != 1)
                return 1;
        if (n == 4) {
            std::printf("%s %d\n", experts[(int)q4::experts_kernel(a[0], a[1], a[2], a[3])],
                        q4::experts_dx_rows(a[0], a[3]));
            continue;
        }
        const q4::LoraLayout f = q4::lora_layout(a[0], a[1], a[2], (int)a[3], (int)a[4], 0);
        const q4::LoraLayout b = q4::lora_layout(a[0], a[1], a[2], (int)a[3], (int)a[4], 1);
        std::printf("%s %d %d %d %d %d %d\n", lora[(int)q4::lora_kernel(a[0], a[1])], q4::lora_dx_rows(a[0], a[2]),
                    f.plan.parts, f.out_parts, b.plan.parts, b.out_parts, b.splits);
    }
    return 0;
}
