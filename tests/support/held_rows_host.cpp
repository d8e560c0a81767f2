// Rows held by a workgroup (HeldRow of token_loss_device.h), run on the CPU one
// thread after another: every element of a row is summed once and written once,
// what a thread parks stays in its LDS slots, nothing else is touched.  LOGPROB_HELD
// and DISTILL_HELD are the chunks a thread holds in either kernel.  Vocabularies go
// up to each workgroup's capacity, dense where a thread's last chunks begin.
#include <algorithm>
#include <cstdio>
#include <set>
#include <vector>

#include "token_loss_device.h"

extern "C" __bf16 __truncsfbf2(float x)   // exact here: the values have eight bits at most
{
    return __builtin_bit_cast(__bf16, (uint16_t)(__builtin_bit_cast(uint32_t, x) >> 16));
}

namespace zero {
int device_cu_count() { return 256; }
}

using namespace zero;
using namespace zero::dev;

namespace {

template <typename T>
T of_value(int v)
{
    if constexpr (sizeof(T) == 2)
        return (T)(__builtin_bit_cast(uint32_t, (float)v) >> 16);
    else
        return (T)v;
}

template <typename T, int NT, int H, bool SAME>
int check(int vocab, int phase, int out_phase)
{
    typedef HeldRow<T, NT, H, SAME> Held;
    constexpr int P = parked(NT), kGuard = 2 * NT;
    const u32x4 mark = {0xa5a5a5a5u, 1, 2, 3};
    alignas(kLine) static T in[(H + 2) * 1024 * 8 + 256], out[(H + 2) * 1024 * 8 + 256];
    // the index by its low eight bits, then by what is left of it
    for (int digit = 0; digit < 2; ++digit) {
        auto value = [&](int i) { return digit ? i >> 8 & 255 : i & 255; };
        const T outside = of_value<T>(-3);
        for (int i = 0; i < vocab + 2 * 128; ++i)
            in[i] = out[i] = outside;
        for (int i = 0; i < vocab; ++i)
            in[phase + i] = of_value<T>(value(i));
        const Row<T> row(in + phase, vocab);
        std::vector<u32x4> park(NT * P + kGuard, mark);
        std::vector<int> seen(256, 0), want(256, 0);
        for (int i = 0; i < vocab; ++i)
            ++want[value(i)];
        int wrong = 0;
        for (int t = 0; t < NT; ++t) {
            threadIdx.x = t;
            Held held;
            held.park = park.data();
            held.read(row);
            held.take(row);
            auto see = [&](float x) {
                if (x == -kInf)
                    return;
                if (x >= 0.0f && x < 256.0f && x == (float)(int)x)
                    ++seen[(int)x];
                else
                    ++wrong;
            };
            held.each_group([&](int, const float (&x)[Held::G * Held::W]) {
                for (float v : x)
                    see(v);
            });
            if (held.e >= 0)
                see(held.edge);
            held.map(out + out_phase, true, Row<T>(), [](float x) { return x; });
        }
        for (int i = NT * P; i < NT * P + kGuard; ++i)
            wrong += std::memcmp(&park[i], &mark, sizeof(mark)) != 0;
        const bool summed = seen == want;
        bool written = true;
        for (int i = 0; i < vocab + 2 * 128; ++i) {
            const int e = i - out_phase;
            written = written && out[i] == (e >= 0 && e < vocab ? of_value<T>(value(e)) : outside);
        }
        if (wrong || !summed || !written) {
            std::printf("%zu-byte elements, %d threads of %d chunks, vocab %d at place %d, gradient at %d: %s%s%s\n",
                        sizeof(T), NT, H, vocab, phase, out_phase, summed ? "" : "not summed once; ",
                        written ? "" : "not written once; ", wrong ? "other values or slots touched" : "");
            return 1;
        }
    }
    return 0;
}

template <typename T, int NT, int H>
int sizes()
{
    constexpr int W = Row<T>::W, kPlaces = kLine / (int)sizeof(T);
    // the largest vocabulary that this workgroup is chosen for
    const int most = (NT * H) * W - (kPlaces - 1);
    std::set<int> vocab = {1, W, 3 * W + 1, NT * W, NT * W + 1, most};
    for (int c = H - 3; c < H; ++c)   // into a thread's last chunks, and through them
        for (int d : {-kPlaces, -1, 0, 1, W, kPlaces, NT * W / 2 + 3})
            vocab.insert(NT * W * c + d);
    int bad = 0, n = 0;
    for (int v : vocab) {
        if (v < 1 || v > most || (chunks_per<T>(v, 1) > NT * H))
            continue;
        for (int phase : {0, 1, W, kPlaces - 1}) {
            bad += check<T, NT, H, true>(v, phase, phase);
            bad += check<T, NT, H, false>(v, phase, (phase + 3) % kPlaces);
            n += 2;
        }
    }
    std::printf("%zu-byte elements, %d threads of %d chunks: %d cases, %d wrong\n", sizeof(T), NT, H, n, bad);
    return bad;
}

}  // namespace

int main()
{
    constexpr int L = LOGPROB_HELD, D = DISTILL_HELD;
    int bad = sizes<uint16_t, 64, L>() + sizes<uint16_t, 256, L>() + sizes<uint16_t, 512, L>() +
              sizes<uint16_t, 1024, L>() + sizes<float, 64, L>() + sizes<float, 256, L>() +
              sizes<float, 512, L>() + sizes<float, 1024, L>();
    bad += sizes<uint16_t, 64, D>() + sizes<uint16_t, 192, D>() + sizes<uint16_t, 448, D>() +
           sizes<uint16_t, 960, D>() + sizes<float, 64, D>() + sizes<float, 192, D>() +
           sizes<float, 448, D>() + sizes<float, 960, D>();
    return bad ? 1 : 0;
}
