// The shared memory of the norm and rotation kernels: their tables are read 16
// bytes at a time, and what the append of the largest batch takes is within what
// a kernel has without asking for more.
#include <cstddef>
#include <cstdio>

#include "rotate.cu"

using namespace moira;

int main()
{
    if (alignof(RotateSmem) % 16 || offsetof(RotateSmem, cos) % 16 || offsetof(RotateSmem, sin) % 16 || sizeof(RotateSmem::cos[0]) % 16)
        return std::printf("tables of alignment %zu at %zu and %zu\n", alignof(RotateSmem), offsetof(RotateSmem, cos), offsetof(RotateSmem, sin)), 1;
    const size_t all = sizeof(RotateSmem) + append_smem(kMaxUnits);
    if (all > 48 * 1024) return std::printf("%zu bytes\n", all), 1;
    std::printf("ok\n");
    return 0;
}
