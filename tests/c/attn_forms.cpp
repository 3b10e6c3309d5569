// Reads problems, one a line:
//   elem_bytes B Tq Tk H Hkv D reach left right pad
// (left, right negative: no limit; pad: elements between a frame's heads and the
// next frame of q, k and v) and prints the instances that the attention's
// launch plan takes for each, by the kernels' template arguments.
#include <cstdio>

#include "attn_plan.h"

using namespace dw;

static void print(const char* kernel, int elem, const AttnForm& f, bool with_packed) {
    printf("%s<%s, %d, %d, %s", kernel, elem == 2 ? "unsigned short" : "float", f.dp, f.own, f.direct ? "true" : "false");
    if (with_packed) printf(", %s", f.packed ? "true" : "false");
    printf(">;");
}

int main() {
    long long elem, B, Tq, Tk, H, Hkv, D, reach, left, right, pad;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &elem, &B, &Tq, &Tk, &H, &Hkv, &D, &reach, &left,
                 &right, &pad) == 11) {
        AttnShape s = {};
        s.B = B, s.Tq = Tq, s.Tk = Tk, s.H = H, s.Hkv = Hkv, s.D = D, s.reach = reach, s.scale = 1.0f;
        s.left = left < 0 ? kNoLimit : left, s.right = right < 0 ? kNoLimit : right;
        auto stride = [&](int64_t T, int64_t heads, int64_t more) {
            return AttnStride{T * (heads * D + more), heads * D + more, D};
        };
        const int e = (int)elem;
        const bool keys = direct_fits(nullptr, stride(Tk, Hkv, pad), D, e);
        const bool queries = direct_fits(nullptr, stride(Tq, H, pad), D, e) && direct_fits(nullptr, stride(Tq, H, 0), D, e);
        print("attn_fwd_kernel", e, fwd_form(fwd_plan(s), D, e, keys), true);
        print("attn_dq_kernel", e, bwd_form(owned(s, e, true), D, e, keys), false);
        print("attn_dkv_kernel", e, bwd_form(owned(s, e, false), D, e, queries), false);
        printf("\n");
    }
    return 0;
}
