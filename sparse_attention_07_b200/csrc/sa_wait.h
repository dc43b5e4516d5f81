// sa_wait.h — time limits of waits that read only the low 32 bits of the
// nanosecond timer (plain C++: the arithmetic is checked on the CPU).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SA_HOST_DEVICE __host__ __device__
#else
#define SA_HOST_DEVICE
#endif

namespace sa {

// The low word comes round every 4.295 s, and an elapsed time of 32 bits is never
// above 2^32 - 1.  A limit of at most 2^31 ns leaves another 2.1 s in which a wait
// that looks at the clock sees that it has run out.
constexpr uint32_t kMaxWait32Ns = 1u << 31;

SA_HOST_DEVICE constexpr uint32_t wait32_limit(uint32_t limit_ns) {
    return limit_ns < kMaxWait32Ns ? limit_ns : kMaxWait32Ns;
}

SA_HOST_DEVICE constexpr bool wait32_over(uint32_t t0, uint32_t now, uint32_t limit_ns) { return now - t0 > limit_ns; }

}  // namespace sa
