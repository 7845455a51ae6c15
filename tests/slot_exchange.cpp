// Runs slot_reduce() and slot_meet() of csrc/slot_exchange.cuh on the CPU, a
// thread to a warp of one slot, and checks that all of them leave at the same
// row when one gives up.  Every pair of a slow warp (held after each barrier
// until every other one is at its next barrier or has left) and of a warp and
// row that give up is run.  A barrier that cannot fill any more, because a
// warp has left, is noticed and counts as a failure; nothing waits on time.
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline
struct float2 {
    float x, y;
};
struct alignas(16) float4 {
    float x, y, z, w;
};

struct Slot {
    std::mutex m;
    std::condition_variable c;
    int W = 0, slow = 0;
    int waiting = 0, turn = 0;
    std::vector<int> arrived;  // barriers a warp has come to
    std::vector<bool> gone;
    bool stuck = false;
};
static Slot *slot;
static thread_local int self;

static void named_barrier(int, int) {
    Slot &s = *slot;
    std::unique_lock<std::mutex> l(s.m);
    const int mine = ++s.arrived[self], turn = s.turn;
    ++s.waiting;
    s.c.notify_all();
    if (s.waiting == s.W) {
        s.waiting = 0;
        ++s.turn;
        s.c.notify_all();
    } else {
        s.c.wait(l, [&] {
            for (int w = 0; w < s.W; ++w)
                if (s.gone[w] && s.arrived[w] < mine) return true;
            return s.turn != turn || s.stuck;
        });
        if (s.turn == turn) {
            s.stuck = true;  // a warp has left, this barrier never fills
            s.c.notify_all();
            return;
        }
    }
    if (self == s.slow)
        s.c.wait(l, [&] {
            if (s.stuck) return true;
            for (int w = 0; w < s.W; ++w)
                if (w != self && !s.gone[w] && s.arrived[w] <= mine) return false;
            return true;
        });
}
static unsigned __any_sync(unsigned, bool p) { return p; }
static float warp_sum(float v) { return v; }
static void warp_sum2(float &, float &) {}

#include "slot_exchange.cuh"

// the row at which each warp left (rows: none gave up), or -1 where a barrier never filled
static std::vector<int> run(bool reduce, int W, int rows, int slow, int who, int when) {
    Slot s;
    s.W = W, s.slow = slow;
    s.arrived.assign(W, 0);
    s.gone.assign(W, false);
    slot = &s;
    alignas(16) static float buf[2][gbn::kRedStride];
    for (auto &b : buf)
        for (float &f : b) f = 0.f;
    int flag = 0;
    std::vector<int> at(W, rows);
    std::vector<std::thread> t;
    for (int w = 0; w < W; ++w)
        t.emplace_back([&, w] {
            self = w;
            for (int k = 0; k < rows; ++k) {
                const bool give_up = w == who && k == when;
                float v[1] = {static_cast<float>(w + 1)};
                bool stop;
                if (reduce) {
                    stop = gbn::slot_reduce<1>(v, buf[k & 1], &flag, k + 1, give_up, W, w, 0, 1, 32 * W);
                } else {
                    gbn::slot_meet(&flag, k + 1, give_up, 1, 32 * W);
                    stop = gbn::slot_stops(&flag, k + 1);
                }
                if (stop || (reduce && v[0] != W * (W + 1) / 2)) {
                    at[w] = k;
                    break;
                }
            }
            std::lock_guard<std::mutex> l(s.m);
            s.gone[w] = true;
            s.c.notify_all();
        });
    for (auto &x : t) x.join();
    if (s.stuck) at.assign(W, -1);
    return at;
}

int main() {
    int runs = 0, bad = 0;
    for (bool reduce : {false, true})
        for (int W : {2, 4})
            for (int rows : {1, 2, 5})
                for (int slow = 0; slow < W; ++slow)
                    for (int who = 0; who < W; ++who)
                        for (int when = 0; when <= rows; ++when) {
                            const std::vector<int> at = run(reduce, W, rows, slow, who, when);
                            ++runs;
                            for (int w = 0; w < W; ++w)
                                if (at[w] != when) {
                                    ++bad;
                                    std::printf("%s, %d warps, %d rows, warp %d slow, warp %d gives up at %d: warp %d left at %d\n",
                                                reduce ? "slot_reduce" : "slot_meet", W, rows, slow, who, when, w, at[w]);
                                    break;
                                }
                        }
    std::printf("%d runs, %d wrong\n", runs, bad);
    return bad != 0;
}
