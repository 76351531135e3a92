// kernels_attn.hip -- linear attention, bf16: the walk's instances for rows of whole
// aligned 16-byte pieces, and the choice between them and those of kernels_attn_any.hip.
#include "attn_walk.hpp"

namespace ssd {

// whole 16-byte pieces at whole 16-byte places, a tile's rows within 24 bits of each other
static bool whole_pieces(const void* p, int64_t bs, uint32_t rs, int d) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bs % 8 == 0 && rs % 8 == 0 && d % 8 == 0 && rs < (1u << 22);
}

hipError_t launch_attn_any(const AttnArgs& A, bool full, hipStream_t st);

hipError_t launch_attn_bf16(const AttnArgs& A, bool full, hipStream_t st) {
    bool whole = true;
    for (unsigned i = 0; i < A.walks; ++i) {
        const AttnPass& p = A.p[i];
        whole = whole && whole_pieces(p.c, p.cb, p.cr, p.cd) && whole_pieces(p.x, p.xb, p.xr, p.xd);
        if (full) whole = whole && whole_pieces(p.a, p.ab, p.ar, p.cd) && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
    }
    return whole ? launch<true>(A, full, st) : launch_attn_any(A, full, st);
}

}  // namespace ssd
