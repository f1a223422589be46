// Test shim: the planner's row plans (windowed or 4-bit attention) as flat arrays.
#include <algorithm>
#include <cstring>

#include "../shared_prefix_fan_gb300/csrc/plan.h"

using namespace fanout;

// Plans for suffix_lens, after patching a plan made for prev_lens when prev_lens
// is not null. Writes up to cap units; returns the unit count, or -1 - status.
extern "C" int row_plan(const int32_t* prev_lens, const int32_t* suffix_lens,
                        const int32_t* q_rows, int32_t B, int32_t P, int32_t H_q, int32_t H_kv,
                        int32_t page, int32_t causal, int32_t window, int32_t sinks, int32_t sms,
                        int32_t splits, int32_t row_bytes, int32_t* units, int32_t cap,
                        int32_t* tok_pos, int32_t* info, int32_t* merge_cnt) {
    PlanInput in{suffix_lens, q_rows, B, P, H_q, H_kv, page, causal, sms, splits};
    in.rows = 1;
    in.window = window;
    in.sinks = sinks;
    in.row_bytes = row_bytes;
    Plan plan;
    bool kept = false;
    if (prev_lens) {
        PlanInput prev = in;
        prev.suffix_lens = prev_lens;
        if (const int st = build_plan(prev, plan)) return -1 - st;
        kept = patch_plan(in, plan);
    }
    if (!kept)
        if (const int st = build_plan(in, plan)) return -1 - st;
    const int n = static_cast<int>(plan.units.size());
    for (int i = 0; i < std::min(n, cap); ++i) std::memcpy(units + 8 * i, &plan.units[i], 32);
    std::copy(plan.tok_pos.begin(), plan.tok_pos.end(), tok_pos);
    std::copy(plan.merge_cnt.begin(), plan.merge_cnt.end(), merge_cnt);
    info[0] = plan.split_at;
    info[1] = plan.nq;
    info[2] = plan.tpt;
    info[3] = plan.n_parts;
    info[4] = kept;
    info[5] = plan.n_cta();
    return n;
}
