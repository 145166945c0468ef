// A model, on the host, of how the tcgen05 tree decode's producers and
// consumers share a ring: every role as a little state machine, every barrier
// as its count of completed phases, and schedules that hold roles back as long
// as they like. A role that waits for phase k of a barrier sees a parity only:
// the wait is sound while k or k + 1 phases are complete, and wrong at any
// other count (it would stop the role for good, or let it through too early).
//
//   ring_model          the kernel's rule, for the rings that its forms have
//   ring_model planted  a rule that is wrong: load i by producer i % producers,
//                       each of which waits for the places of all loads
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "pd_tree_tc.cuh"

namespace {

// Consumers wait for every load in order and give its place back, up to one load late (V of a block goes back after
// the wait for the next block's K).
template <int kPlaces, int kProducers, bool kPlanted>
bool sound(int consumers, int walks, unsigned seed) {
    const int loads = 12 * kPlaces;
    std::mt19937 rng(seed);
    for (int w = 0; w < walks; ++w) {
        std::vector<int> at(kProducers, 0), seen(consumers, 0), back(consumers, 0);
        std::vector<int> full(kPlaces, 0), empty(kPlaces, 0), gone(kPlaces, 0);  // phases; consumers done in this phase
        // priorities: the runnable role of the highest one moves; a few times a walk they are drawn again
        std::vector<unsigned> rank(kProducers + consumers);
        auto draw = [&] {
            for (auto& r : rank) r = rng();
        };
        draw();
        bool fine = true;
        auto wait = [&](int count, int k) {  // passes?
            fine &= count == k || count == k + 1;
            return (count & 1) != (k & 1);
        };
        auto step = [&](int role) {  // moves? (a wait is polled each time that the role runs)
            if (role < kProducers) {
                const int i = at[role], place = i % kPlaces;
                if (i == loads) return false;
                const bool mine = kPlanted ? i % kProducers == role : pd::TreeProducers<kPlaces, kProducers>::mine(place, role);
                if ((kPlanted || mine) && i >= kPlaces && !wait(empty[place], i / kPlaces - 1)) return false;
                if (mine) ++full[place];
                ++at[role];
                return true;
            }
            const int c = role - kProducers;
            auto give = [&] {
                const int place = back[c]++ % kPlaces;
                if (++gone[place] == consumers) {
                    gone[place] = 0;
                    ++empty[place];
                }
                return true;
            };
            const int i = seen[c];
            if (back[c] < i && (i == loads || back[c] < i - 1 || rng() % 2 == 0)) return give();
            if (i < loads && wait(full[i % kPlaces], i / kPlaces)) return ++seen[c], true;
            return back[c] < i && give();
        };
        for (int left = kProducers + consumers; left > 0;) {
            if (rng() % 16 == 0) draw();
            // roles in the order of their ranks until one moves
            std::vector<int> order;
            for (int r = 0; r < kProducers + consumers; ++r) order.push_back(r);
            for (size_t x = 1; x < order.size(); ++x)
                for (size_t y = x; y > 0 && rank[order[y]] > rank[order[y - 1]]; --y) std::swap(order[y], order[y - 1]);
            bool moved = false;
            for (int r : order)
                if ((moved = step(r))) break;
            if (!fine) return false;
            left = 0;
            for (int p : at) left += p < loads;
            for (int c : back) left += c < loads;
            if (!moved && left > 0) return false;  // nobody can go on
        }
    }
    return true;
}

template <int D, bool kWide, bool kFp8, bool kPlanted>
bool form(const char* name) {
    using C = pd::CfgTree<D, kWide, kFp8>;
    constexpr int places = kFp8 ? C::kStages : C::kSlots;
    const bool ok = sound<places, C::kProducers, kPlanted>(kFp8 ? C::kInspectors : C::kPipes + C::kInspectors, 2000, 7);
    std::printf("%s: %d places, %d producers: %s\n", name, places, C::kProducers, ok ? "sound" : "not sound");
    return ok;
}

template <bool kPlanted>
int count() {
    return form<64, false, false, kPlanted>("16-bit, head_dim 64, narrow") + form<64, true, false, kPlanted>("16-bit, 64, wide") +
           form<128, false, false, kPlanted>("16-bit, 128, narrow") + form<128, true, false, kPlanted>("16-bit, 128, wide") +
           form<256, false, false, kPlanted>("16-bit, 256") + form<64, false, true, kPlanted>("E4M3, 64, narrow") +
           form<64, true, true, kPlanted>("E4M3, 64, wide") + form<128, false, true, kPlanted>("E4M3, 128, narrow") +
           form<128, true, true, kPlanted>("E4M3, 128, wide") + form<256, false, true, kPlanted>("E4M3, 256");
}

}  // namespace

int main(int argc, char** argv) {
    const int ok = argc > 1 && std::strcmp(argv[1], "planted") == 0 ? count<true>() : count<false>();
    std::printf("%d of 10 sound\n", ok);
    return 0;
}
