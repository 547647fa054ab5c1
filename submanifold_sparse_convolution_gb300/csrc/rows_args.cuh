// Argument checks shared by the C entries of the row-wise operators.
#pragma once
#include "rows.cuh"

namespace spconv {

constexpr int32_t kMaxChannels = 65536;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A row matrix as the caller gave it: n rows of c elements, ld elements apart.
struct Rows {
    const void* p;
    int64_t n, c, ld;
    size_t es;
    bool ok() const { return p && aligned(p, es) && ld >= c && ld < (int64_t(1) << 38); }
    size_t bytes() const { return n == 0 ? 0 : (static_cast<size_t>(n - 1) * ld + c) * es; }
    bool overlaps(const Rows& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        if (!p || !o.p || a >= b + o.bytes() || b >= a + bytes()) return false;
        // column ranges of one wider matrix: the rows interleave without touching
        const uintptr_t pitch = static_cast<uintptr_t>(ld) * es;
        if (n > 1 && o.n > 1 && pitch == static_cast<uintptr_t>(o.ld) * o.es) {
            const uintptr_t d = b >= a ? (b - a) % pitch : (pitch - (a - b) % pitch) % pitch;   // o's row after this one's
            return d < static_cast<uintptr_t>(c) * es || d + static_cast<uintptr_t>(o.c) * o.es > pitch;
        }
        return true;
    }
    // the same rows at the same places: an in-place update
    bool same(const Rows& o) const { return p == o.p && (ld == o.ld || n <= 1); }
};

// fp32 values in a row (absent: null, which overlaps nothing)
inline Rows vec(const float* p, int64_t c) { return {p, 1, c, c, 4}; }

inline size_t size_of(int32_t dtype) { return dtype == SPCONV_FP32 ? 4 : dtype == SPCONV_E4M3 ? 1 : 2; }

inline bool bad_sizes(int64_t n, int32_t c_in, int32_t c_out) {
    return n < 0 || n >= (int64_t(1) << 30) || c_in < 1 || c_out < 1 || c_in > kMaxChannels || c_out > kMaxChannels;
}
inline bool bad_act(int32_t a) { return a < SPCONV_ACT_NONE || a > SPCONV_ACT_GELU_TANH; }
inline bool bad_vec(const float* v) { return !aligned(v, 4); }

inline int zero(void* p, size_t bytes, cudaStream_t s) { return p ? cuda_status(cudaMemsetAsync(p, 0, bytes, s)) : SPCONV_OK; }

}  // namespace spconv
