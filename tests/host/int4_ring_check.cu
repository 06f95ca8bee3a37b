// Host-side check of the waits that end a warp of the int4 products when a
// copy did not come in time (csrc/int4_mv.cuh stage_parity, drain), on a model
// of its ring: a barrier completes one phase per load of its slot, and a wait
// for a parity passes once the current phase has the other one.  For every
// number of stages and every stage whose wait gave up, with that stage and the
// ones behind it still on their way: the waits of the loop before it passed,
// its own did not, and the drain waits for each load in flight and for no
// phase that nothing will complete.  Prints "OK <cases>" or the first violation.
#include <cstdio>

#include "int4_mv.cuh"

using namespace l4moe::mv;

template <int STAGES>
static bool walk(int stages, int at) {
    int issued = 0, done[STAGES] = {}, loads[STAGES] = {};
    auto bad = [&](const char* what, int slot) {
        printf("%s: ring of %d, stage %d of %d, slot %d\n", what, STAGES, at, stages, slot);
        return false;
    };
    auto passes = [&](int slot, uint32_t parity) { return ((uint32_t)done[slot] & 1u) != parity; };
    for (; issued < STAGES && issued < stages; ++issued) ++loads[issued % STAGES];
    for (int i = 0; i < at; ++i) {  // stages that came: each is used, then its slot loaded again
        ++done[i % STAGES];
        if (!passes(i % STAGES, stage_parity<STAGES>(i))) return bad("a stage that came is not seen", i % STAGES);
        if (issued < stages) ++loads[issued++ % STAGES];
    }
    if (passes(at % STAGES, stage_parity<STAGES>(at))) return bad("a stage on its way is taken", at % STAGES);
    bool fine = true;
    drain<STAGES>(at, stages, [&](int slot, uint32_t parity) {
        if (passes(slot, parity)) return;
        if (done[slot] == loads[slot]) fine = bad("a wait for a load that was not issued", slot);
        ++done[slot];  // it comes while it is waited for
    });
    for (int s = 0; s < STAGES; ++s)
        if (fine && done[s] != loads[s]) fine = bad("a copy in flight is not waited for", s);
    return fine;
}

int main() {
    long long cases = 0;
    for (int stages = 1; stages <= 40; ++stages)
        for (int at = 0; at < stages; ++at, ++cases)
            if (!walk<Cfg<1, float>::STAGES>(stages, at) || !walk<3>(stages, at) || !walk<4>(stages, at)) return 1;
    printf("OK %lld\n", cases);
    return 0;
}
