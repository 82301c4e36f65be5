// Host-only probe of dispatch_expert_plan.hpp (built and run by
// tests/test_expert_plan.py on the CPU): for each line "rows experts N K
// workspace" of the input, the tokens of a tile, the workgroups that share one,
// the workspace's bytes and whether a SwiGLU product widens its operands.
#include <cstdio>

#include "dispatch_expert_plan.hpp"

int main() {
    long long rows, experts, n, k;
    int workspace;
    while (std::scanf("%lld %lld %lld %lld %d", &rows, &experts, &n, &k, &workspace) == 5) {
        const moe_dispatch::ProductSizes s{rows, (int32_t)experts, (int32_t)n, (int32_t)((k + 127) / 128), workspace != 0};
        const int tokens = moe_dispatch::tile_tokens(s);
        const moe_dispatch::ProductPlan plan = moe_dispatch::plan_product(tokens, s);
        std::printf("%d %d %zu %d\n", tokens, plan.parts, plan.bytes, (int)(tokens == 16 && moe_dispatch::wide_operands(s)));
    }
    return 0;
}
