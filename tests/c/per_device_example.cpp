// What the host keeps per CUDA device, with a fake of the calls that make it: prints "ok" lines.
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

static int failures = 0;
static void check(bool good, const char* what) {
    std::printf("%s %s\n", good ? "ok" : "FAIL", what);
    failures += !good;
}

int main() {
    {
        pkv::PerDevice p;
        std::vector<int> made(4, 0);
        auto make = [&](int dev) {
            return [&made, dev](int* v) {
                ++made[dev];
                *v = 100 + dev;
                return 0;
            };
        };
        bool right = true;
        for (int round = 0; round < 3; ++round)
            for (int dev = 0; dev < 4; ++dev) {
                int v = 0;
                right &= p.get(dev, &v, make(dev)) == 0 && v == 100 + dev;
            }
        check(right, "every device has its own value");
        check(made == std::vector<int>(4, 1), "made once for each device, a second one's too");
    }
    {
        pkv::PerDevice p;
        int calls = 0, v = 0;
        auto fails_once = [&](int* x) {
            *x = 7;
            return ++calls == 1 ? 13 : 0;
        };
        check(p.get(1, &v, fails_once) == 13, "an error is returned");
        check(p.get(1, &v, fails_once) == 0 && v == 7 && calls == 2, "and not remembered");
        check(p.get(1, &v, fails_once) == 0 && v == 7 && calls == 2, "what worked is");
    }
    {
        pkv::PerDevice p;
        int calls = 0, v = 0;
        for (int dev : {-1, 64, 1000000})
            for (int i = 0; i < 2; ++i) p.get(dev, &v, [&](int* x) { ++calls; *x = 5; return 0; });
        check(calls == 6 && v == 5, "devices past the table are asked every time");
    }
    {
        pkv::PerDevice p;
        std::atomic<int> wrong{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 8; ++t)
            threads.emplace_back([&] {
                for (int i = 0; i < 10000; ++i) {
                    int v = 0;
                    const int dev = i % 8;
                    if (p.get(dev, &v, [&](int* x) { *x = 1 + dev; return 0; }) != 0 || v != 1 + dev) ++wrong;
                }
            });
        for (auto& t : threads) t.join();
        check(wrong == 0, "threads together");
    }
    return failures != 0;
}
