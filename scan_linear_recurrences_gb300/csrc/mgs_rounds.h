// How the blocks of a cluster exchange one message each a round, and how they leave
// when a wait gives up.
//
// A block has two slots for each block's message, used in turn, with a barrier for each
// turn that counts the bytes of all of them.  In a round every block pushes its message
// to all (itself too), arms its barrier of that turn with what it expects and waits.
//   * A block pushes in round n + 1 when all its waits of round n are over, so it arms no
//     barrier whose last phase is open, and a peer's message of round n + 1 says that
//     the peer has read that of round n - 1: its slots and barrier are free again.
//   * A wait that gives up is known to the whole block behind its next block barrier,
//     and the block takes no part any more: it neither pushes, arms nor waits.  Its
//     peers' waits then give up in turn, and all run their rounds out.
//   * No block may leave while messages are on their way to it, and a cluster barrier
//     does not wait for them.  Without a give-up each block has waited for all there
//     are.  With one (blocks that gave up tell all others before the cluster's last
//     barrier) a block that has pushed in `mine` rounds has had all messages of
//     those before; of round mine - 1, armed for all blocks, some may never come (a block
//     that pushed in fewer rounds: it stands in for those itself), and peers that pushed
//     in more rounds, of which it can be one only, have sent that one's: it is armed for
//     those alone.  Both phases end then, and are waited for.
// The steps are Ops', the kernel's or a simulation's.
#pragma once

#ifdef __CUDACC__
#define MGS_ROUNDS_FN __device__ __forceinline__
#else
#define MGS_ROUNDS_FN inline
#endif

namespace mgs {

// A warp's part of a round, behind a block barrier.  (Whether its block takes part is the same for all its warps: what
// they read was written before that barrier, and is written for the round after this one in the other turn's place.)
template <class Ops>
MGS_ROUNDS_FN void exchange_round(const Ops &op, int round) {
    const int turn = round & 1;
    if (op.gave_up(turn ^ 1)) return op.stay_out(turn);
    op.push(turn);
    op.count_and_arm(turn);  // (by the first warp)
    if (!op.wait(turn, (round >> 1) & 1)) op.give_up(turn);
}

// Behind the last round; all warps
template <class Ops>
MGS_ROUNDS_FN void leave_rounds(const Ops &op, int cluster) {
    op.block_barrier();
    if (op.gave_up(0) || op.gave_up(1)) op.tell_all();
    op.cluster_barrier();
    if (!op.told()) return;
    if (op.first_warp()) {
        const int mine = op.pushed(op.rank());
        int more = 0;
        for (int r = 0; r < cluster; ++r) {
            const int theirs = op.pushed(r);
            if (theirs < mine) op.stand_in(r, (mine - 1) & 1);
            if (theirs > mine) ++more;
        }
        bool all = op.wait((mine - 1) & 1, ((mine - 1) >> 1) & 1);
        if (more > 0) {
            op.arm(mine & 1, more);
            if (!op.wait(mine & 1, (mine >> 1) & 1)) all = false;
        }
        if (!all) op.not_drained();
    }
    op.cluster_barrier();
}

}  // namespace mgs
