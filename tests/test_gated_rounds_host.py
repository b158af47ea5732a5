"""The exchange between the blocks of a cluster, with waits that give up, played through
on the CPU: the steps are the header's that the kernels take, on modelled barriers,
messages that arrive when they like, and warps that go on in any order."""
import subprocess

import pytest

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import build

PROGRAM = r"""
#include <ucontext.h>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>
#include <vector>
#include "mgs_rounds.h"

struct Barrier {  // one arrival a phase, and the messages that it is armed for
    int pending = 1, due = 0, done = 0;
};
struct Message {
    int to, from, round;
};
struct Block {
    Barrier bar[2];
    std::vector<int> slots[2];
    int gave_up[2] = {0, 0}, pushed = 0, told = 0, waiting = 0, generation = 0, warps = 0;
};
struct Warp {
    ucontext_t at;
    std::vector<char> stack;
    int block, warp;
    bool over = false;
};

struct Cluster {
    std::mt19937 rng;
    std::vector<Block> blocks;
    std::vector<Warp> warps;
    std::vector<Message> way;
    ucontext_t back;
    int running = 0, waiting = 0, generation = 0, rounds, give_ups = 0, from = -1, to = -1;  // a slow way
    bool patient;
    double haste;
    std::string wrong;

    int any(int n) { return int(rng() % unsigned(n)); }
    void fail(const std::string &what) {
        if (wrong.empty()) wrong = what;
    }
    void yield() { swapcontext(&warps[running].at, &back); }
    void settle(Barrier &b) {
        if (b.pending == 0 && b.due == 0) ++b.done, b.pending = 1;
    }
    void arm(Barrier &b, int n) {
        if (b.pending == 0) return fail("a barrier armed in an open phase");
        b.due += n, --b.pending;
        settle(b);
    }
    void deliver() {
        const int i = any(int(way.size()));
        const Message m = way[i];
        if (m.from == from && m.to == to && any(300) != 0) return;
        way.erase(way.begin() + i);
        Block &b = blocks[m.to];
        if (b.warps == 0) fail("a message to a block that has left");
        Barrier &bar = b.bar[m.round & 1];
        if (bar.done != m.round >> 1) fail("a message counted in another round's phase");
        b.slots[m.round & 1][m.from] = m.round;
        --bar.due;
        settle(bar);
    }
};
static Cluster *sim;

struct Ops {
    int block, warp, round;
    bool leaving = false;
    Block &me() const { return sim->blocks[block]; }
    bool gave_up(int turn) const { sim->yield(); return me().gave_up[turn]; }
    void stay_out(int turn) const { me().gave_up[turn] = 1; }
    void give_up(int turn) const { ++sim->give_ups, stay_out(turn); }
    void push(int turn) const {
        for (int r = warp; r < int(sim->blocks.size()); r += int(sim->warps.size() / sim->blocks.size())) {
            sim->way.push_back({r, block, round});
            sim->yield();
        }
        if ((round & 1) != turn) sim->fail("a turn of another round");
    }
    void count_and_arm(int turn) const {
        if (warp != 0) return;
        sim->arm(me().bar[turn], int(sim->blocks.size()));
        sim->yield();
        ++me().pushed;
    }
    bool wait(int turn, int phase) const {
        const int patience = sim->patient || leaving ? 100000 : 4 << sim->any(12);
        for (int polls = 0;; ++polls) {
            sim->yield();
            if ((me().bar[turn].done & 1) != phase) return true;
            if (polls > patience) return false;
            if (!leaving && sim->any(10000) < sim->haste * 10000) return false;
        }
    }
    void block_barrier() const {
        Block &b = me();
        const int g = b.generation;
        if (++b.waiting == b.warps) b.waiting = 0, ++b.generation;
        while (b.generation == g) sim->yield();
    }
    void cluster_barrier() const {
        const int g = sim->generation;
        if (++sim->waiting == int(sim->warps.size())) sim->waiting = 0, ++sim->generation;
        while (sim->generation == g) sim->yield();
    }
    void tell_all() const {
        for (Block &b : sim->blocks) b.told = 1, sim->yield();
    }
    bool told() const { return me().told; }
    bool first_warp() const { return warp == 0; }
    int rank() const { return block; }
    int pushed(int r) const {
        sim->yield();
        if (sim->blocks[r].warps == 0) sim->fail("the count of a block that has left");
        return sim->blocks[r].pushed;
    }
    void stand_in(int r, int turn) const { sim->way.push_back({block, r, round_of(turn)}); }
    void arm(int turn, int n) const { sim->arm(me().bar[turn], n); }
    void not_drained() const { sim->fail("messages that never came were waited for"); }
    int round_of(int turn) const { return me().pushed - 1 + ((me().pushed - 1 - turn) & 1); }
};

#ifdef PLANTED  // what must be seen: a block that gave up goes on without waiting, and leaves behind a cluster barrier
template <class O>
void exchange(O &op, int round) {
    const int turn = round & 1;
    op.push(turn), op.count_and_arm(turn);
    if (!op.gave_up(turn ^ 1) && op.wait(turn, (round >> 1) & 1)) return;
    op.give_up(turn);
}
template <class O>
void leave(O &op, int) { op.block_barrier(), op.cluster_barrier(); }
#else
template <class O>
void exchange(O &op, int round) { mgs::exchange_round(op, round); }
template <class O>
void leave(O &op, int n) { mgs::leave_rounds(op, n); }
#endif

static void play() {
    Warp &w = sim->warps[sim->running];
    Ops op{w.block, w.warp, 0};
    for (int n = 0; n < sim->rounds; ++n) {
        op.round = n;
        op.block_barrier();
        exchange(op, n);
        for (int m : sim->blocks[w.block].slots[n & 1]) {
            if (!sim->blocks[w.block].gave_up[n & 1] && m != n) sim->fail("a message of another round");
            sim->yield();
        }
    }
    op.leaving = true;
    leave(op, int(sim->blocks.size()));
    if (--sim->blocks[w.block].warps == 0)
        for (const Message &m : sim->way)
            if (m.to == w.block) sim->fail("a block left while a message was on its way to it");
    w.over = true;
    swapcontext(&w.at, &sim->back);
}

int main(int argc, char **argv) {
    long give_ups = 0, whole = 0;
    for (int seed = 0; seed < atoi(argv[1]); ++seed) {
        Cluster c;
        sim = &c;
        c.rng.seed(seed);
        const int blocks = 2 << (c.any(16) == 0 ? 3 : c.any(2)), warps = 1 + c.any(3);
        c.rounds = 1 + c.any(7), c.patient = c.any(2) == 0;
        c.haste = c.any(2) == 0 ? 0.0 : 0.1 / (1 << c.any(12));
        c.blocks.resize(blocks), c.warps.resize(blocks * warps);
        for (Block &b : c.blocks) b.warps = warps, b.slots[0].assign(blocks, -1), b.slots[1].assign(blocks, -1);
        std::vector<int> alive;
        for (int i = 0; i < blocks * warps; ++i) {
            Warp &w = c.warps[i];
            w.block = i / warps, w.warp = i % warps, w.stack.resize(65536);
            getcontext(&w.at);
            w.at.uc_stack.ss_sp = w.stack.data(), w.at.uc_stack.ss_size = w.stack.size(), w.at.uc_link = nullptr;
            makecontext(&w.at, play, 0);
            alive.push_back(i);
        }
        if (c.any(2) == 0) c.from = c.any(blocks), c.to = c.any(blocks);
        const int slow = c.any(3) == 0 ? c.any(blocks) : -1, net = 1 << c.any(6);  // one block behind the others, a slow network
        for (long step = 0; !alive.empty() && c.wrong.empty(); ++step) {
            if (step > 50000000) c.fail("no end");
            if (!c.way.empty() && c.any(net) == 0) {
                c.deliver();
                continue;
            }
            const int i = c.any(int(alive.size()));
            if (c.warps[alive[i]].block == slow && c.any(50) != 0) continue;
            c.running = alive[i];
            swapcontext(&c.back, &c.warps[c.running].at);
            if (c.warps[c.running].over) alive.erase(alive.begin() + i);
        }
        if (c.wrong.empty() && !c.way.empty()) c.fail("a message that nobody waited for");
        if (!c.wrong.empty())
            return printf("seed %d, %d blocks of %d warps, %d rounds: %s\n", seed, blocks, warps, c.rounds, c.wrong.c_str()), 1;
        give_ups += c.give_ups, whole += c.give_ups == 0;
    }
    return printf("%ld give-ups, %ld runs without\n", give_ups, whole), 0;
}
"""


def _play(tmp_path, runs, *flags):
    src, exe = tmp_path / "rounds.cpp", tmp_path / "rounds"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", *flags, "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe), str(runs)], capture_output=True, text=True, timeout=300)


def test_blocks_leave_with_nothing_on_its_way_to_them(tmp_path):
    run = _play(tmp_path, 300)
    assert run.returncode == 0, run.stdout
    give_ups, whole = (int(run.stdout.split()[i]) for i in (0, 2))
    assert give_ups > 100 and whole > 20


def test_going_on_without_waiting_is_seen(tmp_path):
    assert _play(tmp_path, 200, "-DPLANTED").returncode == 1


def test_refusals_of_the_diagnostic():
    build.build()
    fake = 1 << 40
    for args, status in (((-1, 0, 0, None, fake), b.MGS_ERR_INVALID_ARG), ((-1, 0, 0, fake, None), b.MGS_ERR_INVALID_ARG),
                         ((-1, 0, 1_000_000_001, fake, fake + 64), b.MGS_ERR_INVALID_ARG),
                         ((-1, 0, 0, fake, fake + 16), b.MGS_ERR_INVALID_ARG),  # over one another
                         ((-1, 0, 0, fake + 2, fake + 64), b.MGS_ERR_UNSUPPORTED)):
        with pytest.raises(b.MGSError) as e:
            b.mgs_debug_exchange(*args, stream=0)
        assert e.value.status == status
