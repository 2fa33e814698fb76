// Host build of the acceptance kernel's residual arithmetic: the integer of one residual, and the
// sum of eight as the kernel's passes take them.
#include "../../mla_speculative_verify_attention_gb300/csrc/residual.cuh"

using namespace mla;

static long long of_one(int form, float p, float q, Coef c) {
    if (form == FROM_P) return residual<FROM_P>(p, q, c);
    if (form == MINUS_Q) return residual<MINUS_Q>(p, q, c);
    return residual<MINUS_AQ>(p, q, c);
}

extern "C" void residual_units(int form, double A, const float* p, const float* q, long long n, long long* out) {
    Coef c;
    c.ah = (float)A;
    c.al = (float)(A - (double)c.ah);
    for (long long i = 0; i < n; ++i) out[i] = of_one(form, p[i], q[i], c);
}

extern "C" long long residual_sum8(double A, const float* p, const float* q) {
    Coef c;
    c.ah = (float)A;
    c.al = (float)(A - (double)c.ah);
    Few few = {0, 0};
    for (int i = 0; i < 8; i += 2) add_residuals<MINUS_AQ>(p[i], p[i + 1], q[i], q[i + 1], c, few);
    return few.sum(8);
}

extern "C" double residual_unit() { return UNIT; }
