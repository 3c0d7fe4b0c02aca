// strides.h -- whether a result's rows lie apart.  Host code without CUDA: the C entry
// points and the binding in C++ ask alike.
#pragma once

#include <algorithm>
#include <cstdint>

namespace w4 {

// Whether two of the T * H rows of D values at t * tok + h * head share one.  Tokens and
// heads may lie in either order or interleaved, so rows that do not nest (the longer
// stride past all of the shorter one's) are compared: of token differences only the two
// next to a head difference can bring rows together.
inline bool rows_overlap(int64_t T, int64_t H, int64_t D, int64_t tok, int64_t head)
{
    if (T < 1 || H < 1)
        return false;
    tok = tok < 0 ? -tok : tok;                // only differences count, of either sign
    head = head < 0 ? -head : head;
    if ((T > 1 && tok < D) || (H > 1 && head < D))
        return true;
    if (T == 1 || H == 1)
        return false;
    if (head >= tok ? (head - D) / tok >= T - 1 : (tok - D) / head >= H - 1)
        return false;
    for (int64_t dh = 1; dh < H; dh++) {
        const int64_t at = dh * head, below = std::min(at / tok, T - 1);
        if (at - below * tok < D || (below + 1 < T && (below + 1) * tok - at < D))
            return true;
        if (at / tok >= T)                     // past the last token by a stride, D at least
            break;
    }
    return false;
}

}  // namespace w4
