"""The windowed backward's barriers, every order its roles can run in: a model of who waits for and arrives at what
(csrc/attn_bwd_window.cu), walked state by state.  A barrier has a phase, and a wait names the parity of the phase
it is for: it passes while the phase that is running has the other parity, so it fails where the barrier has moved
on by two.  No order may leave a role waiting for good, and no wait may pass before what it is for."""

import os
import re

import pytest

from tests._lib import ROOT

SOURCE = os.path.join(ROOT, "context_causal_attention_load_gb300", "csrc", "attn_bwd_window.cu")


def dq_tiles():
    """dQ tiles (each with a barrier of its own) of the head dim 64 kernel; 1 if the source gives one"""
    m = re.search(r"NDQ = APART \? (\d+) : 1;", open(SOURCE).read())
    return int(m.group(1)) if m else 1


def roles(n, apart, ndq):
    """The roles' programs for n steps of one unit: lists of ("wait", barrier, phase), ("arrive", barrier) and
    ("issue", [barriers that the tensor core arrives at once it is there])."""
    prod, mma, ew, read, red = [], [], [], [], []
    ring = lambda name, j: ("%s%d" % (name, j % 2), j // 2)  # noqa: E731
    dq = lambda j: ("dq_full%d" % (j % ndq), j // ndq)  # noqa: E731
    for j in range(n):
        if j >= 2:
            prod.append(("wait", *ring("q_empty", j - 2)))
        prod.append(("arrive", ring("q_full", j)[0]))
        if j >= 2:
            prod.append(("wait", *ring("do_empty", j - 2)))
        prod.append(("arrive", ring("do_full", j)[0]))

        more = j + 1 < n
        if j == 0:
            mma += [("wait", *ring("q_full", 0)), ("issue", ["s_full"]), ("wait", *ring("do_full", 0)), ("issue", ["dp_full"])]
        mma += [("wait", "p_full", j), ("issue", [ring("do_empty", j)[0]] if apart else [])]  # dV
        if more:
            mma += [("wait", *ring("q_full", j + 1)), ("issue", ["s_full"])]
        mma += [("wait", "dst_full", j), ("issue", [ring("q_empty", j)[0]])]  # dK
        if apart:
            if more:
                mma += [("wait", *ring("do_full", j + 1)), ("issue", ["dp_full"])]
            mma.append(("wait", "dss_full", j))
            if j >= 2:
                mma.append(("wait", *ring("dq_free", j - 2)))
            mma.append(("issue", [dq(j)[0]]))
        else:
            mma += [("wait", "dss_full", j), ("issue", [dq(j)[0]])]
            if more:
                mma += [("wait", "dq_free", j), ("wait", *ring("do_full", j + 1)), ("issue", ["dp_full"])]

        ew += [("wait", "s_full", j), ("arrive", "p_full"), ("wait", "dp_full", j), ("arrive", "dst_full")]
        if j:
            ew.append(("wait", *(dq(j - 1) if apart else ("ds_free", j - 1))))
        ew.append(("arrive", "dss_full"))

        read.append(("wait", *dq(j)))
        if apart:
            read.append(("arrive", ring("dq_free", j)[0]))
            if j >= 2:
                read.append(("wait", *ring("stg_empty", j - 2)))
            read.append(("arrive", ring("staged", j)[0]))
            red.append(("wait", *ring("staged", j)))
            if j:
                red.append(("arrive", ring("stg_empty", j - 1)[0]))  # the tile before is read
        else:
            read += [("arrive", "staged_ds"), ("arrive", "dq_free"), ("arrive", "staged")]
            red += [("wait", "staged_ds", j), ("wait", "staged", j), ("arrive", "ds_free"), ("arrive", ring("do_empty", j)[0])]
    return [prod, mma, ew, read, red]


def explore(programs):
    """(a state in which nobody can go on, or None; a wait that passed too early, or None)"""
    names = sorted({x for p in programs for op in p for x in (op[1] if op[0] == "issue" else [op[1]])})
    at = {x: i for i, x in enumerate(names)}
    mma = 1
    # the tensor core works off what was issued, in order: its program is the issuer's
    issues = [[at[b] for b in op[1]] for op in programs[mma] if op[0] == "issue"]
    start = ((0,) * len(programs), 0, (0,) * len(names))
    seen, todo = {start}, [start]
    early = None
    while todo:
        pcs, done, phases = todo.pop()
        nexts = []
        issued = sum(op[0] == "issue" for op in programs[mma][:pcs[mma]])
        if done < issued:
            ph = list(phases)
            for b in issues[done]:
                ph[b] += 1
            nexts.append((pcs, done + 1, tuple(ph)))
        for r, prog in enumerate(programs):
            if pcs[r] == len(prog):
                continue
            op = prog[pcs[r]]
            ph = phases
            if op[0] == "wait":
                if phases[at[op[1]]] % 2 == op[2] % 2:
                    continue
                if phases[at[op[1]]] <= op[2]:
                    early = op
            elif op[0] == "arrive":
                ph = list(phases)
                ph[at[op[1]]] += 1
                ph = tuple(ph)
            nexts.append((pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], done, ph))
        if not nexts and any(pc < len(p) for pc, p in zip(pcs, programs)):
            return [p[pc] if pc < len(p) else None for pc, p in zip(pcs, programs)], early
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None, early


@pytest.mark.parametrize("n", [1, 2, 3, 6])
@pytest.mark.parametrize("apart", [False, True])
def test_no_order_stops(apart, n):
    stuck, early = explore(roles(n, apart, dq_tiles() if apart else 1))
    assert stuck is None and early is None, (stuck, early)


def test_one_barrier_for_two_tiles_stops():
    """what the model is for: dQ of step j + 2 formed before the read-out looks for that of j + 1"""
    stuck, _ = explore(roles(6, True, 1))
    assert stuck is not None and stuck[3][:2] == ("wait", "dq_full0")
