// Host-side check of the costs that attention's shares go by (no GPU needed): what all blocks before one
// cost together is the sum of what each of them does, for prompts (fewer, as many and more keys than rows),
// chains of drafted tokens and trees, also where the page table cuts their tokens off.
// Compiled and run by tests/test_flash_shares.py; exits non-zero on a failure.
#include "flash.cuh"

#include <cstdio>
#include <random>

using namespace edge0::flash;

struct Drafts {                      // blocks and steps as attention of drafted tokens has them
    static constexpr int kBlock = kRowsQ, kTile = 64, kOwn = 4;
};

static int fails = 0, checked = 0;

template <class Sh>
static void check(const Seq& s, int G, const char* what) {
    const Costs<Sh> c(s, G);
    long long sum = 0;
    for (int t = 0; t < c.blocks; ++t) {
        ++checked;
        if (c.before(t) != sum && ++fails < 20)
            printf("FAIL %s n_q %d n_k %d off %d G %d block %d of %d: %lld before it, not %lld\n", what, s.n_q, s.n_k, s.off, G, t,
                   c.blocks, c.before(t), sum);
        sum += c.own + c.tokens(t);
        if (c.tokens(t) < 0 || c.tokens(t) > c.all) ++fails;
    }
    if (c.total() != sum && ++fails < 20) printf("FAIL %s total %lld, not %lld\n", what, c.total(), sum);
}

template <class Sh>
static void check_all(std::mt19937& rng) {
    auto draw = [&](int most) { return (int)(rng() % (unsigned)(most + 1)) >> rng() % 8; };
    for (int i = 0; i < 4000; ++i) {
        const int G = 1 + draw(63), n_q = draw(5000), ctx = draw(20000), cap = 16 * (1 + draw(1500));
        Seq s{0, n_q, 0, draw(20000), 0, 0};
        s.off = s.n_k - s.n_q;
        check<Sh>(s, G, "prompt");
        s.ctx = ctx < cap ? ctx : cap;
        s.n_k = s.ctx + n_q < cap ? s.ctx + n_q : cap;
        s.off = s.ctx;
        check<Sh>(s, G, "chain");
        s.off = s.n_k;
        check<Sh>(s, G, "tree");
    }
}

int main() {
    std::mt19937 rng(1);
    check_all<Shape<64>>(rng);
    check_all<Shape<256>>(rng);
    check_all<Drafts>(rng);
    printf("%d blocks\n", checked);
    if (fails || checked < 10000) return 1;
    printf("ALL OK\n");
    return 0;
}
