// Every order in which two copying warps, the issuing warp and the tensor cores can pass a ring's barriers, as the adapters' kernel for
// many rows uses them in its two products.  argv: stages of the first product, of the second, and optionally
//   two          a model with two barriers for finished products, by the parity of the stage, in place of a slot's own
//   lost N [on]  the products numbered N and later never finish: when nobody can go on, the waits run out.  Who waited leaves the loop and the
//                next one ("on": goes on in it).
// Prints "ok" or what went wrong.
#include <algorithm>
#include <array>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include <vector>

#include "ep_ring.h"

using namespace ep;

constexpr int kWarps = 2;
bool two = false, on = false;
int lost = 1 << 30;
int stages[2];

enum Kind { kFill, kWaitDone, kWaitFull, kWaitFree, kRead, kIssue, kTake, kWaitTaken, kSync };      // (the stage of the last but one: its chunk)
struct Op {
    Kind kind;
    int part, stage;
};
std::vector<Op> copier, issuer;

int done_bar(int stage) { return two ? stage & 1 : ring_slot(stage); }
int done_phase(int part, int stage) {
    if (!two) return ring_phase(stage, part ? stages[0] : 0);
    return (part ? (stages[0] + 1 - (stage & 1)) / 2 : 0) + (stage >> 1);
}
int full_phase(int part, int stage) { return ring_phase(stage, part ? stages[0] : 0); }

void programs() {
    for (int i = 0; i < kRing - 1 && i < stages[0]; ++i) copier.push_back({kFill, 0, i});
    for (int i = 0; i < stages[0]; ++i) {
        if (i > 0) copier.push_back({kWaitDone, 0, i - 1});
        if (i + kRing - 1 < stages[0]) copier.push_back({kFill, 0, i + kRing - 1});
        if (i > 0 && chunk_begins(i)) copier.push_back({kTake, 0, stage_chunk(i - 1)});
    }
    if (stages[0] > 0) {
        copier.push_back({kWaitDone, 0, stages[0] - 1});
        copier.push_back({kTake, 0, stage_chunk(stages[0] - 1)});
    }
    copier.push_back({kSync, 0, 0});
    for (int i = 0; i < kRing - 1 && i < stages[1]; ++i) copier.push_back({kFill, 1, i});
    for (int i = 0; i < stages[1]; ++i) {
        if (i > 0) copier.push_back({kWaitFree, 1, i - 1});
        if (i + kRing - 1 < stages[1]) copier.push_back({kFill, 1, i + kRing - 1});
        copier.push_back({kWaitFull, 1, i});
        copier.push_back({kWaitDone, 1, i});
        copier.push_back({kRead, 1, i});
    }
    for (int i = 0; i < stages[0]; ++i) {
        issuer.push_back({kWaitFull, 0, i});
        if (chunk_begins(i) && stage_chunk(i) >= 2) issuer.push_back({kWaitTaken, 0, stage_chunk(i) - 2});
        issuer.push_back({kIssue, 0, i});
    }
    issuer.push_back({kSync, 0, 0});
    for (int i = 0; i < stages[1]; ++i) {
        issuer.push_back({kWaitFull, 1, i});
        if (i >= 2) issuer.push_back({kWaitFree, 1, i - 2});
        issuer.push_back({kIssue, 1, i});
    }
}

// Where each warp and the issuer are, how many products have been finished, and who has had a wait run out.
using State = std::array<int, 2 * kWarps + 3>;
constexpr int kFailed = kWarps + 2;

int count(const std::vector<Op> &prog, int pc, Kind kind, int part, int stage_at_most, int (*key)(int), int k) {
    int n = 0;
    for (int i = 0; i < pc; ++i)
        if (prog[i].kind == kind && prog[i].part <= part && (prog[i].part < part || prog[i].stage <= stage_at_most) && key(prog[i].stage) == k) ++n;
    return n;
}
bool passed(const std::vector<Op> &prog, int pc, const Op &op) {
    for (int i = 0; i < pc; ++i)
        if (prog[i].kind == op.kind && prog[i].part == op.part && prog[i].stage == op.stage) return true;
    return false;
}

int ended(const State &s, Kind kind, int bar) {          // phases that a barrier has ended
    if (kind == kWaitDone) {
        int n = 0, at = 0;
        for (const Op &op : issuer)
            if (op.kind == kIssue && at++ < s[kWarps + 1] && done_bar(op.stage) == bar) ++n;
        return n;
    }
    int least = 1 << 30;
    if (kind == kWaitTaken) {
        for (int w = 0; w < kWarps; ++w) least = std::min(least, count(copier, s[w], kTake, 1, 1 << 30, chunk_buffer, bar));
        return least;
    }
    for (int w = 0; w < kWarps; ++w) least = std::min(least, count(copier, s[w], kind == kWaitFull ? kFill : kRead, 1, 1 << 30, ring_slot, bar));
    return least;
}

// 1: may go on, 0: has to wait, -1: goes on or waits wrongly
int wait(const State &s, const Op &op) {
    const int bar = op.kind == kWaitDone ? done_bar(op.stage) : op.kind == kWaitTaken ? chunk_buffer(op.stage) : ring_slot(op.stage);
    const int phase = op.kind == kWaitTaken ? chunk_phase(op.stage) : op.kind == kWaitDone ? done_phase(op.part, op.stage) : op.kind == kWaitFull ? full_phase(op.part, op.stage) : ring_phase(op.stage);
    const int n = ended(s, op.kind, bar);
    const bool sees = ((n ^ phase) & 1) != 0, is = n > phase;
    if (sees != is) return -1;
    return is;
}

std::string explore() {
    std::set<State> seen;
    std::vector<State> todo{State{}};
    seen.insert(todo[0]);
    while (!todo.empty()) {
        const State s = todo.back();
        todo.pop_back();
        bool moved = false, all = true;
        auto go = [&](int who) {
            State t = s;
            ++t[who];
            moved = true;
            if (seen.insert(t).second) todo.push_back(t);
        };
        for (int who = 0; who <= kWarps; ++who) {
            const std::vector<Op> &prog = who < kWarps ? copier : issuer;
            if (s[who] == (int)prog.size() || (s[kFailed + who] && !on)) continue;       // it has left its loops: done, and at the barrier between
            all = false;
            const Op op = prog[s[who]];
            if (op.kind == kFill) {
                // what the slot held before has been multiplied (and, of the second product, read by everyone)
                if (op.stage >= kRing) {
                    int at = 0, when = 0;
                    for (const Op &q : issuer)
                        if (q.kind == kIssue && ++at && q.part == op.part && q.stage == op.stage - kRing) when = at;
                    if (s[kWarps + 1] < when) return "a slot is filled before its products are done";
                    if (op.part == 1)
                        for (int w = 0; w < kWarps; ++w)
                            if (!passed(copier, s[w], {kRead, 1, op.stage - kRing})) return "a slot is filled before it has been read";
                }
                go(who);
            } else if (op.kind == kRead || op.kind == kIssue || op.kind == kTake) {
                // a chunk's buffer has been read by everyone before the next but one begins in it, and is read before that
                if (op.kind == kIssue && op.part == 0 && chunk_begins(op.stage) && stage_chunk(op.stage) >= 2)
                    for (int w = 0; w < kWarps; ++w)
                        if (!passed(copier, s[w], {kTake, 0, stage_chunk(op.stage) - 2})) return "a buffer of sums is written before it has been read";
                if (op.kind == kIssue && op.part == 1 && stages[0] > 0)
                    for (int w = 0; w < kWarps; ++w)
                        if (!passed(copier, s[w], {kTake, 0, stage_chunk(stages[0] - 1)}) && !s[kFailed + w]) return "sums are written over before they have been read";
                go(who);
            } else if (op.kind == kSync) {
                bool here = true;
                for (int o = 0; o <= kWarps; ++o) here = here && (s[kFailed + o] || passed(o < kWarps ? copier : issuer, s[o] + 1, {kSync, 0, 0}));
                if (here) go(who);
            } else {
                const int r = wait(s, op);
                if (r < 0) return "a wait sees the parity of another phase";
                if (r) go(who);
            }
        }
        int issued = 0;
        for (int i = 0; i < s[kWarps]; ++i) issued += issuer[i].kind == kIssue;
        if (s[kWarps + 1] < std::min(issued, lost)) all = false, go(kWarps + 1);
        if (!moved && !all) {
            if (lost == 1 << 30) return "nobody can go on";
            State t = s;
            bool waits = false;
            for (int who = 0; who <= kWarps; ++who) {
                const std::vector<Op> &prog = who < kWarps ? copier : issuer;
                if (s[who] == (int)prog.size() || (s[kFailed + who] && !on) || prog[s[who]].kind == kSync) continue;
                waits = true;
                t[kFailed + who] = 1;
                if (on) ++t[who];
            }
            if (!waits) return "nobody can go on";
            if (seen.insert(t).second) todo.push_back(t);
        }
    }
    return "ok";
}

int main(int argc, char **argv) {
    stages[0] = atoi(argv[1]);
    stages[1] = atoi(argv[2]);
    two = argc > 3 && !strcmp(argv[3], "two");
    if (argc > 4 && !strcmp(argv[3], "lost")) lost = atoi(argv[4]);
    on = argc > 5;
    programs();
    const std::string r = explore();
    printf("%s\n", r.c_str());
    return r == "ok" ? 0 : 1;
}
