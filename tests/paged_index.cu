// Rows, sequences and pages of a paged call on the host, by the kernels' own
// functions: reads n_seqs n_rows max_pages page_size n_pages uniform, then
// row_start (unless uniform), kv_len and the table, and prints for every row its
// sequence, position, page and slot; last, divisions n q for given n d.
#include <cstdio>
#include <vector>

#include "../block_speculative_drafting_gb300/csrc/paged.cuh"

using namespace dflash;

int main() {
    long long ns, nr, mp, ps, np, uniform;
    while (scanf("%lld %lld %lld %lld %lld %lld", &ns, &nr, &mp, &ps, &np, &uniform) == 6 && ns >= 0) {
        std::vector<int32_t> start(ns + 1), len(ns), table(ns * mp);
        if (!uniform)
            for (auto& x : start) scanf("%d", &x);
        for (auto& x : len) scanf("%d", &x);
        for (auto& x : table) scanf("%d", &x);
        PagedRows R{};
        R.n_seqs = (int)ns, R.max_pages = (int)mp, R.n_rows = (int)nr, R.cap = (int)(mp * ps);
        R.per = uniform && ns ? (int)(nr / ns) : 0;
        R.row_start = uniform ? nullptr : start.data();
        R.kv_len = len.data(), R.table = table.data(), R.table_stride = mp;
        R.page = fast_div((int)ps);
        for (int r = 0; r < nr; ++r) {
            const int s = seq_of(R, r);
            if (s < 0) {
                printf("-1 0 -1 0\n");
                continue;
            }
            int a, b, slot = 0;
            rows_of(R, s, a, b);
            const int64_t pos = (int64_t)len[s] - (b - a) + (r - a);
            const int64_t page = page_of(R, np, s, pos < -1 ? -1 : (int)pos, slot);
            printf("%d %lld %lld %d\n", s, (long long)pos, (long long)page, page < 0 ? 0 : slot);
        }
        printf("end\n");
    }
    long long n, d;
    while (scanf("%lld %lld", &n, &d) == 2) printf("%d\n", div_by(fast_div((int)d), (int)n));
    return 0;
}
