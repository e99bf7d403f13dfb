"""Host model of the waits inside the 4-bit attention's tile kernel (no GPU).

A wait for an mbarrier names a phase by its parity alone: it is right only when
the phase before has completed already, and it ends only when the phase after
cannot complete first.  Both have to follow from the order of the kernel's own
waits and arrivals; that things usually land in time is not enough.  The model
runs the programs of the kernel's warps and keeps, for every step, the set of
steps that must have come before it: a product's commit arrives some time after
it was issued, in no order with other commits."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_aware_quantized_gb300", "csrc")
WARPS = 7


def mma(ng, tiles):
    """The issuing warp: ("wait", barrier, phase), ("commit", barrier)."""
    ops = [("wait", "KFull0", 0)] + [("commit", f"S{g}") for g in range(ng)] + [("commit", "KEmpty0")]
    for j in range(tiles):
        s, more = j & 1, j + 1 < tiles
        if ng == 2:
            ops.append(("wait", f"VFull{s}", j >> 1))
        if more:
            ops.append(("wait", f"KFull{s ^ 1}", j + 1 >> 1))
        if ng == 1:
            if more:
                ops.append(("commit", f"S{s ^ 1}"))
                if j:
                    ops.append(("wait", f"VEmpty{s ^ 1}", j - 1 >> 1))
                ops += [("wait", f"KEmpty{s}", j >> 1), ("commit", f"KEmpty{s ^ 1}")]
            ops += [("wait", f"P{s}", j >> 1), ("wait", f"VFull{s}", j >> 1), ("commit", f"VEmpty{s}")]
            if not more:
                ops.append(("commit", "O0"))
            continue
        for g in range(2):
            ops.append(("wait", f"P{g}", j))
            if g:
                ops.append(("commit", f"VEmpty{s}"))
            ops.append(("commit", f"S{g}" if more else f"O{g}"))
        if more:
            ops.append(("commit", f"KEmpty{s ^ 1}"))
    return ops


def decoder(w, per, tiles):
    """A decoding warp: keys, then values of a tile in pieces of `per` groups."""
    pieces, ops = 8 // per, []
    for u in range(w, 2 * pieces * tiles, WARPS):
        j, kind = u // (2 * pieces), "V" if u & pieces else "K"
        if j >= 2:
            ops.append(("wait", f"{kind}Empty{j & 1}", (j >> 1) - 1))
        ops.append(("arrive", f"{kind}Full{j & 1}"))
    return ops


def softmax(g, ng, tiles, raises):
    ops = []
    for j in range(tiles):
        at = j & 1 if ng == 1 else g
        ops.append(("wait", f"S{at}", j >> 1 if ng == 1 else j))
        if ng == 1 and j and raises and j % raises == 0:  # (a row's reference moves in every `raises`-th tile)
            ops.append(("wait", f"VEmpty{j - 1 & 1}", j - 1 >> 1))
        ops.append(("arrive", f"P{at}"))
    return ops + [("wait", f"O{g}", 0)]


def run(programs, counts):
    """Runs the programs; -> waits that their phase before, or the phase after, could be taken for."""
    past = {n: frozenset() for n in programs}       # steps before a program's next one
    landed = {}                                     # barrier -> arrivals, each the steps before it
    done, waits, at = {}, [], {n: 0 for n in programs}
    moved = True
    while moved:
        moved = False
        for n, ops in programs.items():
            while at[n] < len(ops):
                kind, bar, *phase = ops[at[n]]
                me = (n, at[n])
                if kind == "wait":
                    key = (bar, phase[0])
                    have, need = landed.get(bar, []), counts.get(bar[:-1], 1)
                    if len(have) < need * (phase[0] + 1):
                        break
                    if key not in done:
                        done[key] = frozenset().union(*have[need * phase[0]:need * (phase[0] + 1)]) | {("done", key)}
                    waits.append((me, key, past[n]))
                    past[n] |= done[key]
                else:
                    # (a commit's arrival is a step of its own, that its warp knows of by a wait alone)
                    landed.setdefault(bar, []).append(past[n] | ({me} if kind == "arrive" else {me, ("landed", me)}))
                past[n] |= {me}
                at[n] += 1
                moved = True
    assert all(at[n] == len(ops) for n, ops in programs.items()), "a wait without end"
    for bar, have in landed.items():
        need = counts.get(bar[:-1], 1)
        for i in range(len(have) // need):
            done.setdefault((bar, i), frozenset().union(*have[need * i:need * (i + 1)]) | {("done", (bar, i))})
    bad = []
    for me, (bar, i), before in waits:
        # all arrivals of the phase before came before this wait; the phase after needs this wait
        if i and not done[bar, i - 1] - {("done", (bar, i - 1))} <= before:
            bad.append(("before", me, bar, i))
        if (bar, i + 1) in done and me not in done[bar, i + 1]:
            bad.append(("after", me, bar, i))
    return bad


def programs(ng, per, tiles, raises, issue=mma, soft=softmax):
    p = {"mma": issue(ng, tiles)}
    p.update({f"decode{w}": decoder(w, per, tiles) for w in range(WARPS)})
    p.update({f"soft{g}": soft(g, ng, tiles, raises) for g in range(ng)})
    return p, {"KFull": 8 // per, "VFull": 8 // per}


@pytest.mark.parametrize("ng,per", [(1, 1), (1, 2), (2, 1)])
@pytest.mark.parametrize("raises", [0, 1, 3])
def test_no_wait_can_be_taken_for_another_phase(ng, per, raises):
    for tiles in (1, 2, 3, 4, 5, 22):
        assert run(*programs(ng, per, tiles, raises)) == []


def test_the_model_sees_a_phase_told_by_time_alone():
    """Buffers given back without a look at the ones before, and one barrier for both P."""
    def issue(ng, tiles):
        ops = mma(ng, tiles)
        return [(k, "P0", *p) if b in ("P0", "P1") else (k, b, *p) for k, b, *p in ops if not (k == "wait" and "Empty" in b)]

    def soft(g, ng, tiles, raises):
        return [(k, "P0", *p) if b in ("P0", "P1") else (k, b, *p) for k, b, *p in softmax(g, ng, tiles, raises)]

    def one_barrier(ops):
        n = iter(range(100))
        return [("wait", "P0", next(n)) if o[:2] == ("wait", "P0") else o for o in ops]

    found = set()
    for raises in (0, 1):
        p, counts = programs(1, 2, 22, raises, issue, soft)
        p["mma"] = one_barrier(p["mma"])
        found |= {(kind, bar) for kind, _, bar, _ in run(p, counts)}
    assert {bar[:-1] for kind, bar in found if kind == "before"} == {"KEmpty", "VEmpty"}
    assert {bar for kind, bar in found if kind == "after"} == {"P0"}


def test_the_kernel_has_these_waits():
    """The order of the waits and commits of the issuing warp, and the premises on the pieces, in the source."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "fp4_tiles.cu")).read())
    loop = src[src.index("for (int j = 0; ok && j < nkt; ++j)"):src.index("mma_commit_warp(BAR(kBarDrain))")]
    text = re.findall(r"wait\((kBar\w+)|BAR\((kBar\w+)|(issue_\w+)\(", loop)
    names = [a or b or c for a, b, c in text]
    assert names == ["kBarVFull", "kBarKFull",
                     "issue_s", "kBarVEmpty", "kBarKEmpty", "kBarKEmpty", "kBarP", "kBarVFull", "issue_pv", "kBarVEmpty", "kBarO",
                     "kBarP", "issue_pv", "kBarVEmpty", "issue_s", "kBarO", "kBarKEmpty"]
    assert "const int ng = kPer == 1 && " in src  # pieces of two groups: one row block
    assert f"kDqWarps = {WARPS}" in src and "static_assert(kDqWarps <= kTileGroups" in src
