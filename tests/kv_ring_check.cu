// Host replay of a worker's ring of copies (no GPU, no library): barriers that
// count as the hardware's do, copies that land after random times or never.
// No barrier is armed while its phase still awaits bytes, every slot that is
// read holds the copy it should, and after a wait that gave up nothing is sent
// and exactly the copies in flight are waited for again.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gdn_kv.cuh"

struct Barrier {
    int completed = 0;  // phases
    bool awaits = false;
    long lands = 0;     // time
    int holds = -1;     // the copy in the slot
    int coming = -1;
};

template <int kUnits>
static int replay(unsigned seed, int copies, long slow, long limit, long drain) {
    srand(seed);
    Barrier bar[kUnits];
    long now = 0;
    auto settle = [&](Barrier& b) {
        if (b.awaits && b.lands <= now) {
            b.awaits = false;
            ++b.completed;
            b.holds = b.coming;
        }
    };
    auto wait = [&](Barrier& b, unsigned parity, long most) {  // a wait of parity p returns once the phase of parity p is over
        const long until = now + most;
        while (true) {
            settle(b);
            if ((unsigned)(b.completed & 1) != parity) return true;
            if (now >= until) return false;
            ++now;
        }
    };
    gdn::CopyRing<kUnits> ring;
    int issued = 0, faults = 0, waited_again = 0, in_flight_at_end = 0;
    bool all_landed = true;
    auto issue = [&]() {
        if (issued >= copies || ring.gave_up) return;
        Barrier& b = bar[ring.send];
        settle(b);
        if (b.awaits) ++faults;
        b.awaits = true;
        b.coming = issued;
        b.lands = now + (rand() % 100 == 0 ? slow : rand() % 5);
        ring.sent();
        ++issued;
    };
    for (int i = 0; i < kUnits; ++i) issue();
    for (int i = 0; i < copies; ++i) {
        if (!ring.gave_up) {
            if (!wait(bar[ring.slot], ring.parity, limit)) {
                ring.gave_up = true;
                gdn::CopyRing<kUnits> left = ring;
                for (int k = ring.pending(); k > 0; --k, left.read()) {
                    ++waited_again;
                    all_landed &= wait(bar[left.slot], left.parity, drain);
                }
                if (waited_again != issued - i) return printf("seed %u: %d copies waited for again, %d in flight\n", seed, waited_again, issued - i), 1;
                for (auto& b : bar) in_flight_at_end += b.awaits;
                if (all_landed && in_flight_at_end) return printf("seed %u: %d copies left in flight\n", seed, in_flight_at_end), 1;
            } else if (bar[ring.slot].holds != i) {
                return printf("seed %u: read %d, holds %d\n", seed, i, bar[ring.slot].holds), 1;
            }
        }
        now += rand() % 4;
        ring.read();
        issue();
    }
    if (faults) return printf("seed %u: %d barriers armed while they awaited bytes\n", seed, faults), 1;
    return 0;
}

int main() {
    int runs = 0;
    for (unsigned seed = 0; seed < 4000; ++seed)
        for (long slow : {3L, 60L, 100000000L})  // within the limit; past it, within the drain's; never
            for (long limit : {0L, 20L}) {
                const int copies = 1 + seed % 97;
                if (replay<3>(seed, copies, slow, limit, 200) || replay<4>(seed, copies, slow, limit, 200)) return 1;
                runs += 2;
            }
    printf("%d replays OK\n", runs);
    return 0;
}
