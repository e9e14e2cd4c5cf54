// The protocol of csrc/scan_chain.h on the host, one lane to a wave: tiles and
// carriers of one column in orders and at times that a device may give them.
// Every tile has to get the state of the plain recurrence, bit for bit, and every
// wait has to end.  Prints a line for each order; the exit code counts failures.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __all(x) (x)
#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_load(p, order, scope) __atomic_load_n(p, order)
#define __hip_atomic_store(p, w, order, scope) __atomic_store_n(p, w, order)
#define __builtin_amdgcn_s_sleep(n) std::this_thread::yield()

using std::max;
using std::min;

static uint32_t __float_as_uint(float f) {
    uint32_t u;
    std::memcpy(&u, &f, 4);
    return u;
}
static float __uint_as_float(uint32_t u) {
    float f;
    std::memcpy(&f, &u, 4);
    return f;
}

#include "scan_chain.h"

namespace {

constexpr int kRuns = 2;  // waves of a tile

struct Column {
    int tiles;
    float start;
    std::vector<float> A, H;             // [tile][run]
    std::vector<float> want;             // the state before each tile, and behind the last
    std::vector<pdn::u64> agg, inc;
    pdn::Chain chain;
    std::vector<float> before, behind;

    Column(int n, unsigned seed, bool carrier) : tiles(n), chain{} {
        std::mt19937 gen(seed);
        std::uniform_real_distribution<float> uni(0.0f, 1.0f);
        start = 4.0f * uni(gen) - 2.0f;
        for (int i = 0; i < n * kRuns; ++i) {
            A.push_back(uni(gen) < 0.03f ? 0.0f : 0.5f + 0.5f * uni(gen));
            H.push_back(uni(gen) < 0.02f ? INFINITY : 2.0f * uni(gen) - 1.0f);
        }
        float h = start;
        for (int i = 0; i < n; ++i) {
            want.push_back(h);
            float tA = A[i * kRuns], tH = H[i * kRuns];
            for (int w = 1; w < kRuns; ++w) {
                const float a = A[i * kRuns + w], b = H[i * kRuns + w];
                tH = a == 0.0f ? b : std::fma(a, tH, b);
                tA = a == 0.0f ? 0.0f : tA * a;
            }
            h = tA == 0.0f ? tH : std::fma(tA, h, tH);
        }
        want.push_back(h);
        agg.assign(static_cast<size_t>(n) * pdn::kCols, pdn::kEmpty);
        inc = agg;
        before.assign(n, NAN);
        behind.assign(n, NAN);
        chain.agg = agg.data();
        chain.inc = inc.data();
        chain.tiles = n;
        chain.carrier = carrier;
    }

    void carry() { pdn::carry(chain, 0, 0); }

    void tile(int at) {
        float totA[kRuns][pdn::kCols] = {}, totH[kRuns][pdn::kCols] = {};
        for (int w = 0; w < kRuns; ++w) {
            totA[w][0] = A[at * kRuns + w];
            totH[w][0] = H[at * kRuns + w];
        }
        before[at] = pdn::meet<kRuns>(chain, totA, totH, 0, at, 0, at == 0 ? start : 0.0f, behind[at]);
    }

    bool right() const {
        for (int i = 0; i < tiles; ++i)
            if (__float_as_uint(before[i]) != __float_as_uint(want[i]) ||
                __float_as_uint(behind[i]) != __float_as_uint(want[i + 1]))
                return false;
        return true;
    }
};

int report(const char* order, int tiles, bool ok) {
    std::printf("%s, %d tiles: %s\n", order, tiles, ok ? "right" : "WRONG");
    std::fflush(stdout);
    return !ok;
}

}  // namespace

int main() {
    int bad = 0;
    for (int n : {2, 3, 33, 34, 150}) {
        {
            Column c(n, 1 + n, false);
            for (int i = 0; i < n; ++i) c.tile(i);
            bad += report("no carrier, one tile after another", n, c.right());
        }
        {
            // other work holds the device from the carrier's start until it gives up
            Column c(n, 2 + n, true);
            c.carry();
            for (int i = 0; i < n; ++i) c.tile(i);
            bad += report("the carrier gone before the first tile", n, c.right());
        }
        {
            // the same after some of the tiles
            Column c(n, 3 + n, true);
            const int some = n / 2;
            for (int i = 0; i < some; ++i) c.tile(i);
            c.carry();
            for (int i = some; i < n; ++i) c.tile(i);
            bad += report("the carrier gone between the tiles", n, c.right());
        }
        {
            Column c(n, 4 + n, true);
            for (int i = 0; i < n; ++i) c.tile(i);
            c.carry();
            bad += report("the carrier behind all tiles", n, c.right());
        }
        for (int carrier = 0; carrier < 2; ++carrier)
            for (unsigned seed = 0; seed < 20; ++seed) {
                Column c(n, 100 * n + seed, carrier);
                std::atomic<int> next{0};
                std::vector<std::thread> threads;
                if (carrier) threads.emplace_back([&] { c.carry(); });
                for (int t = 0; t < 8; ++t)
                    threads.emplace_back([&] {
                        for (int i = next++; i < n; i = next++) c.tile(i);
                    });
                for (auto& t : threads) t.join();
                if (!c.right() || seed == 19) bad += report(carrier ? "all at once, carried" : "all at once", n, c.right());
            }
    }
    return bad;
}
