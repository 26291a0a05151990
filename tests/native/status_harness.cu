// Prints, for each state of the status word given as an argument, what queries return until the word is empty.
#include <cstdio>
#include <cstdlib>

#include "moe/status.cuh"

int main(int argc, char **argv) {
    for (int i = 1; i < argc; ++i) {
        uint32_t word = static_cast<uint32_t>(std::strtoul(argv[i], nullptr, 0));
        for (;;) {
            const uint32_t r = gemm_status::next_report(word);
            std::printf("%d ", static_cast<int>(gemm_status::status_of(r)));
            if (!r) break;
            word &= ~r;
        }
        std::printf("\n");
    }
    return 0;
}
