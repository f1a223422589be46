// Test shim: what the planner's candidates cost by their own account, and by the
// units they are made of.
#include "../shared_prefix_fan_gb300/csrc/plan.cpp"

using namespace fanout;

namespace {

int64_t unit_tiles(const Unit& u, int32_t page, int32_t split_at) {
    const int64_t begin = u.key_begin / page * page;
    const int64_t first = u.key_begin >= split_at ? split_at : 0;
    return (u.key_end - begin + kBN - 1) / kBN +
           (u.pos_base > 0 ? (u.pos_base - first + kBN - 1) / kBN : 0);
}

double busiest(const std::vector<Unit>& units, const std::vector<int32_t>& cta_of, int32_t n_cta,
               int32_t page, int32_t split_at, double ovh) {
    std::vector<double> load(n_cta, 0.0);
    for (size_t i = 0; i < units.size(); ++i)
        load[cta_of[i]] += unit_tiles(units[i], page, split_at) + ovh;
    return *std::max_element(load.begin(), load.end());
}

}  // namespace

// cost[3]: by account, equal chunks (of `chunk` tiles), exact balance, tail cuts;
// load[3]: their busiest CTA, from the units; merge[3]: the account's merge term.
// chosen: the busiest CTA of the plan that is built.
extern "C" int row_plan_cost(const int32_t* suffix_lens, const int32_t* q_rows, int32_t B, int32_t P,
                             int32_t H_q, int32_t H_kv, int32_t page, int32_t causal, int32_t window,
                             int32_t sinks, int32_t sms, int32_t row_bytes, int32_t chunk,
                             double* cost, double* load, double* merge, double* chosen) {
    PlanInput in{suffix_lens, q_rows, B, P, H_q, H_kv, page, causal, sms, 0};
    in.rows = 1;
    in.window = window;
    in.sinks = sinks;
    in.row_bytes = row_bytes;
    std::vector<Range> ranges;
    std::vector<int32_t> tok_pos;
    int32_t R = 0, nq = 0, tpt = 0, split_at = 0;
    make_row_ranges(in, true, ranges, R, nq, tpt, tok_pos, split_at);
    const double ovh = nq == 1 ? kUnitOverhead1 : kUnitOverheadRows2;
    Cand c[3];
    make_candidate(ranges, chunk, 0, sms, ovh, c[0]);
    make_streamk(ranges, sms, ovh, c[1]);
    make_lpt_cut(ranges, sms, ovh, c[2]);
    for (int i = 0; i < 3; ++i) {
        int64_t parts = 0;
        for (const Unit& u : c[i].units) parts += u.part >= 0;
        cost[i] = c[i].cost;
        merge[i] = parts > 0 ? kMergeLaunch + kMergePerPart * parts / c[i].n_cta : 0.0;
        load[i] = busiest(c[i].units, c[i].cta_of, c[i].n_cta, page, split_at, ovh);
    }
    Plan plan;
    if (const int st = build_plan(in, plan)) return -1 - st;
    std::vector<int32_t> cta_of(plan.units.size());
    for (int32_t k = 0; k < plan.n_cta(); ++k)
        for (int32_t i = plan.cta_first[k]; i < plan.cta_first[k + 1]; ++i) cta_of[i] = k;
    *chosen = busiest(plan.units, cta_of, plan.n_cta(), page, plan.split_at,
                      plan.nq == 1 ? kUnitOverhead1 : kUnitOverheadRows2);
    return 0;
}
