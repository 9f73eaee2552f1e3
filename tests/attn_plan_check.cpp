// Checks of attention's launch plan on the host: over random batches, that the
// grids, the shares and the workspace hold whatever lengths the device finds.
// Prints "ok <batches>", or what is wrong.
#include <cstdlib>
#include <random>
#include <vector>

#include "attn_plan.hpp"

using namespace mmq;

static std::mt19937_64 rng(7);
static int64_t upto(int64_t n) { return int64_t(rng() % uint64_t(n + 1)); }
static int64_t log_upto(int64_t n) { return std::min(n, upto((int64_t(2) << upto(40)) - 1) % (n + 1)); }

#define CHECK(x)                                                                                                       \
    do {                                                                                                               \
        if (!(x)) {                                                                                                    \
            std::printf("%s: T=%lld B=%lld max_q=%lld Hq=%d Hkv=%d D=%d pages=%lld of %d CUs=%d\n", #x, (long long)T,   \
                        (long long)B, (long long)max_q, Hq, Hkv, D, (long long)max_pages, page, cus);                   \
            std::exit(1);                                                                                              \
        }                                                                                                              \
    } while (0)

int main() {
    int planned = 0, refused = 0;
    for (int round = 0; round < 20000; round++) {
        const int Ds[] = {64, 128, 256}, pages[] = {16, 32, 64, 128, 256}, cu[] = {1, 8, 64, 256, 304};
        const int D = Ds[upto(2)], page = pages[upto(4)], cus = cu[upto(4)];
        const int Hkv = int(1 + log_upto(63)), G = int(1 + log_upto(1024 / Hkv - 1)), Hq = Hkv * G;
        const int64_t B = 1 + log_upto(2000), max_pages = log_upto((int64_t(1) << 24) / page);
        // lengths as a device may find them: new tokens of each sequence, within T and max_q
        std::vector<int64_t> n(B), keys(B);
        int64_t T = 0, longest = 1;
        for (int64_t b = 0; b < B; b++) {
            n[b] = upto(3) ? log_upto(3) : log_upto(3000);
            T += n[b];
            longest = std::max(longest, n[b]);
            keys[b] = log_upto(max_pages * page);
        }
        T += upto(2) ? 0 : log_upto(5000);                     // rows behind the last sequence
        const int64_t max_q = upto(1) ? longest : std::max<int64_t>(T, 1);
        AttnPlan p;
        char why[256];
        if (T == 0 || check_attention(T, B, Hq, Hkv, D, max_pages, page, max_q)) continue;
        if (!make_plan_attention(T, B, Hq, Hkv, D, max_pages, page, max_q, cus, &p, why, sizeof(why))) {
            CHECK(B * Hkv >= (1 << 22) || (T * G / 128 + B) * Hkv >= (1 << 22));
            refused++;
            continue;
        }
        planned++;
        CHECK(p.few_tiles || p.tile_rows);
        CHECK(p.few_bytes >= 0 && p.few_bytes % 256 == 0 && p.tile_bytes >= 0 && p.tile_bytes % 256 == 0);
        const int64_t few = p.few_tiles ? kAttnFewRows : 0;
        // a few-row sequence of many keys has the kernel that splits them, unless T says that there is none
        if (G <= kAttnFewRows && T < B * std::min(max_q, T) && max_pages * page >= 8192) CHECK(p.few_tiles);
        if (!p.tile_rows) CHECK(longest * G <= 16 * p.few_tiles);        // all rows have a place in the rows kernel
        if (p.few_tiles) {
            CHECK(p.few_grid == B * Hkv * p.few_split && p.few_grid * 256 < (int64_t(1) << 32));
            CHECK(p.few_split >= 1 && (p.few_tiles == 2 || std::min(max_q, T) * G <= 16));
            const int64_t slots = p.few_grid * 16 * p.few_tiles;
            if (p.few_split > 1) CHECK(p.few_bytes >= slots * (D + 2) * 4 + B * Hkv * 4);
            // the device's share: few_chunk of the rows kernel
            int64_t most = 0;
            float total = 0.0f;
            for (int64_t b0 = 0; b0 < B; b0 += 64) {
                int64_t blocks = 0;
                for (int64_t b = b0; b < std::min(B, b0 + 64); b++)
                    if (n[b] > 0 && n[b] * G <= few) most = std::max(most, keys[b]), blocks += keys[b] >> 7;
                total += float(blocks) + 1.0f;
            }
            const int64_t by_device = int64_t(std::fmin(total * float(Hkv) / float(p.few_target), 1e6f)) + 1;
            const int64_t by_slots = ((most + p.few_split - 1) / p.few_split + 127) >> 7;
            const int64_t chunk = std::max<int64_t>(std::max(by_device, by_slots), 1) << 7;
            if (p.few_split > 1) CHECK((most + chunk - 1) / chunk <= p.few_split);
        }
        if (p.tile_rows) {
            CHECK(p.tile_rows == (D == 128 ? 256 : 128) && p.tile_split >= 1);
            CHECK(p.tile_grid == p.tiles * Hkv * p.tile_split && p.tile_grid * 2 * p.tile_rows < (int64_t(1) << 32));
            int64_t tiles = 0;
            for (int64_t b = 0; b < B; b++)
                if (n[b] * G > few) tiles += (n[b] * G + p.tile_rows - 1) / p.tile_rows;
            CHECK(tiles <= p.tiles);
            if (p.tile_split > 1) {
                CHECK(p.tile_bytes >= p.tile_grid * p.tile_rows * (D + 2) * 4);
                CHECK(p.tiles * Hkv * (int64_t(p.tile_rows) * D / 1024) * 256 < (int64_t(1) << 32));      // the join
            }
        }
    }
    // the refusals' borders: a grid that is refused is one of 2^23 workgroups of the rows kernel or 2^22 of the tile kernel
    {
        const int Hq = 64, Hkv = 64, D = 64, page = 16, cus = 256;
        const int64_t max_pages = 4;
        AttnPlan p;
        char why[256] = "";
        int64_t T = 1 << 17, B = (1 << 17) - 1, max_q = 1;
        CHECK(make_plan_attention(T, B, Hq, Hkv, D, max_pages, page, max_q, cus, &p, why, sizeof(why)));
        B++;
        CHECK(!make_plan_attention(T, B, Hq, Hkv, D, max_pages, page, max_q, cus, &p, why, sizeof(why)) && why[0]);
        B = 1, T = max_q = (int64_t(1) << 16) * 128 - 129;               // 2^16 - 2 tiles and one more, of 64 heads
        CHECK(make_plan_attention(T, B, Hq, Hkv, D, max_pages, page, max_q, cus, &p, why, sizeof(why)));
        T = max_q = (int64_t(1) << 16) * 128 - 128;
        CHECK(!make_plan_attention(T, B, Hq, Hkv, D, max_pages, page, max_q, cus, &p, why, sizeof(why)));
    }
    if (planned < 5000) {
        std::printf("only %d batches were planned (%d refused)\n", planned, refused);
        return 1;
    }
    std::printf("ok %d\n", planned);
}
