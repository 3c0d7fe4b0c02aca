// packed.cu -- the entry points with the longest argument lists once more, their
// arguments in one buffer: name_packed(p) calls name with what lies at p, each argument
// at the next multiple of its size, as in a C struct.  For the Python binding, whose
// foreign calls convert argument by argument (5.5 us for the longest list, 0.8 us
// packed: as much as a small call takes on the GPU).
#include <cstring>
#include <tuple>
#include <type_traits>

#include "../../include/w4moe.h"

namespace {

template <class T> struct Type {
    using type = T;
};

template <class... A> int call_packed(int (*fn)(A...), const void *buffer)
{
    const char *p = static_cast<const char *>(buffer);
    size_t at = 0;
    auto next = [&](auto tag) {
        typename decltype(tag)::type v;
        at = (at + sizeof(v) - 1) / sizeof(v) * sizeof(v);
        std::memcpy(&v, p + at, sizeof(v));
        at += sizeof(v);
        return v;
    };
    // in the order written
    std::tuple<A...> args{next(Type<A>{})...};
    return std::apply(fn, args);
}

}  // namespace

#define W4_PACKED(name) \
    extern "C" int name##_packed(const void *buffer) { return call_packed(name, buffer); }

W4_PACKED(w4_w4a16_linear_few)
W4_PACKED(w4_qk_norm_rope)
W4_PACKED(w4_kv_append_rope)
W4_PACKED(w4_kv_keep)
W4_PACKED(w4_attn_shared_prefix)
W4_PACKED(w4_attn_tree)
