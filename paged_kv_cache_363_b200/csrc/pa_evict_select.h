// The arithmetic of pa_evict's selection: keys, and the ranges that its passes count them in.  Plain C++, so that a
// host program can run the same passes.
#pragma once

#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define PA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PA_HOST_DEVICE inline
#endif

namespace pa {

constexpr int kEvictBins = 2048;

// Recent tokens come above every score.
constexpr uint32_t kRecentKey = 0xffffffffu;

// Scores in an unsigned order: larger is better, -0 and +0 alike, NaN above +inf.
PA_HOST_DEVICE uint32_t score_key(float score)
{
    if (score != score) return kRecentKey - 1u;
    const float x = score + 0.f;
#ifdef __CUDA_ARCH__
    const uint32_t b = __float_as_uint(x);
#else
    uint32_t b;
    std::memcpy(&b, &x, sizeof(b));
#endif
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The keys lo .. hi, both among them, that a pass counts in bins of 2^shift() from lo on.  A pass goes on in one bin:
// 32 bits become 21 at most, 21 become 10, and 10 fit the bins one by one, so the third pass is the last.
constexpr int kEvictPasses = 3;

struct KeyRange {
    uint32_t lo, hi;

    PA_HOST_DEVICE int shift() const
    {
        const uint32_t span = hi - lo;
#ifdef __CUDA_ARCH__
        const int bits = 32 - __clz((int)span);
#else
        const int bits = span ? 32 - __builtin_clz(span) : 0;
#endif
        return bits > 11 ? bits - 11 : 0;  // 2^11 bins
    }
    PA_HOST_DEVICE bool has(uint32_t key) const { return key >= lo && key <= hi; }
    PA_HOST_DEVICE uint32_t bin(uint32_t key, int shift) const { return (key - lo) >> shift; }
    PA_HOST_DEVICE uint32_t first(uint32_t bin, int shift) const { return lo + (bin << shift); }
    // The bin that begins at `first`.  The top one ends at hi: its full width may reach past 2^32.
    PA_HOST_DEVICE KeyRange narrow(uint32_t first, int shift) const
    {
        const uint32_t width = (1u << shift) - 1u;
        return KeyRange{first, hi - first > width ? first + width : hi};
    }
};

}  // namespace pa
