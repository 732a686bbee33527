// The plans of linear attention's sweeps for shapes "batch seqlen nheads q_heads k_heads v_heads dk dv dtype", one a
// line: for each sweep (fwd, bwd, dv) segments, their rows, parts of a segment and their rows.
#include "ssm_host.h"

#include <cstdio>
#include <initializer_list>

int main() {
    ssm_linattn_shape s{};
    long long x[9];
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", x, x + 1, x + 2, x + 3, x + 4, x + 5, x + 6, x + 7, x + 8) == 9) {
        s.batch = x[0]; s.seqlen = x[1]; s.nheads = x[2];
        s.q_heads = x[3]; s.k_heads = x[4]; s.v_heads = x[5];
        s.dk = x[6]; s.dv = x[7];
        s.dtype = static_cast<int32_t>(x[8]);
        ssm::LinAttnPlan p;
        if (ssm::plan_linattn(&s, true, &p) != SSM_OK) return 1;
        for (const ssm::LinAttnPlan::Sweep *w : {&p.fwd, &p.bwd, &p.dv})
            std::printf("%lld %lld %lld %lld ", (long long)w->nseg, (long long)w->seg_len, (long long)w->nsub, (long long)w->sub_len);
        std::printf("\n");
    }
    return 0;
}
