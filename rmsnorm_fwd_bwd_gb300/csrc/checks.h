// checks.h -- argument checks and small integer helpers shared by the entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/rmsnorm.h"

namespace rmsnorm {

inline int elem_bytes(int dt) { return dt == RMSNORM_F32 ? 4 : 2; }
inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline rmsnorm_status check_common(int64_t M, int64_t N, rmsnorm_dtype dt, int offset) {
    if (dt != RMSNORM_F32 && dt != RMSNORM_F16 && dt != RMSNORM_BF16) return RMSNORM_ERR_DTYPE;
    if (offset != 0 && offset != 1) return RMSNORM_ERR_ARG;
    if (M < 0 || M > RMSNORM_MAX_M || N < 1 || N > RMSNORM_MAX_N) return RMSNORM_ERR_SHAPE;
    return RMSNORM_OK;
}

inline bool pitch_ok(int64_t ld, int64_t N, int64_t M, size_t s) {
    // ld >= N, and the whole span (M - 1) * ld + N elements addressable
    return ld >= N && ld <= (int64_t(1) << 40) / static_cast<int64_t>(s) &&
           (M <= 1 || (M - 1) <= (int64_t(1) << 46) / ld);
}

}  // namespace rmsnorm
