"""The exchange between the slices of a row in the policy loss, checked on the
host in every order of its steps.

A small model of one row whose slices are worked on by a workgroup each, in
place, the label's score in one of them.  A workgroup
    reads its own scores and, wherever it lies, the label's score,
    publishes the pair of its scores,
    looks at every pair once (the last look of its wait);
where all are there, it uses them and overwrites its scores.  Else
    it waits until what it published has arrived; if it holds the label's score,
    it first publishes that, waits, and publishes its pair again with a mark;
    for each pair that is missing it reads the scores from memory and then looks
    once more, and takes the published pair if it is there by now.
Where the pair that it has of the label's slice is marked, it takes the published
score in place of the one it read.  What is published arrives at any later time;
words are looked at one by one.  Everything that a workgroup uses must come from
the scores, whatever the order.

The same model with one of the steps left out must find an order that goes wrong,
or it would show nothing."""
import pytest

SCORES, GRADIENT = "scores", "gradient"


def goes_wrong(slices, owner, mark=True, second_look=True, wait=True, score_first=True):
    """Whether some order lets a workgroup use what are no longer scores, or a
    published score that is not there."""
    nothing = (None,) * slices
    SCORE = slices  # the word of the label's score

    def program(j):
        p = [("own",), ("publish", j)] + [("look", i) for i in range(slices)] + [("through",)]
        if mark and j == owner:
            p += [("publish", SCORE), ("wait",)] if score_first else []
            p += [("mark",)]
            p += [] if score_first else [("wait",), ("publish", SCORE)]
        if wait:
            p += [("wait",)]
        for i in range(slices):
            p += [("read", i)] + [("again", i)] * second_look
        return p + [("score",), ("store",)]

    programs = [program(j) for j in range(slices)]
    # of every workgroup: step, the pairs it has, those read from memory, the label's
    # score, publications under way (in order)
    start = (((0, nothing, nothing, None, ()),) * slices, (SCORES,) * slices, (None,) * (slices + 1))
    seen, todo = {start}, [start]

    def put(t, i, v):
        return t[:i] + (v,) + t[i + 1:]

    while todo:
        groups, memory, words = todo.pop()
        after = []
        for j, (at, have, found, score, under_way) in enumerate(groups):
            for n, (w, v) in enumerate(under_way):  # something published arrives, in order at one address
                if all(u[0] != w for u in under_way[:n]):
                    rest = under_way[:n] + under_way[n + 1:]
                    after.append((put(groups, j, (at, have, found, score, rest)), memory, put(words, w, v)))
            if at == len(programs[j]):
                continue
            step, *w = programs[j][at]
            mem, to = memory, at + 1
            if step == "own":
                found, score = put(found, j, memory[j]), memory[owner]
            elif step == "publish":
                under_way += ((w[0], (score if w[0] == SCORE else found[j], False)),)
            elif step == "mark":
                under_way += ((j, (found[j], True)),)
            elif step == "look":
                have = put(have, w[0], words[w[0]])
            elif step == "through":
                if all(v is not None for v in have):
                    to = programs[j].index(("score",))
            elif step == "wait":
                if under_way:
                    continue  # not yet
            elif step == "read":
                if have[w[0]] is None:
                    found = put(found, w[0], memory[w[0]])
            elif step == "again":
                if have[w[0]] is None:
                    have = put(have, w[0], words[w[0]])
            elif step == "score":
                if have[owner] is not None and have[owner][1]:
                    score = words[SCORE][0] if words[SCORE] is not None else GRADIENT
            else:
                used = [v[0] if v is not None else f for v, f in zip(have, found)]
                if GRADIENT in used or score == GRADIENT:
                    return True
                mem = put(memory, j, GRADIENT)
            after.append((put(groups, j, (to, have, found, score, under_way)), mem, words))
        for state in after:
            if state not in seen:
                seen.add(state)
                todo.append(state)
    return False


@pytest.mark.parametrize("slices,owner", [(2, 0), (2, 1), (3, 1)])
def test_every_order_uses_the_scores(slices, owner):
    assert not goes_wrong(slices, owner)


@pytest.mark.parametrize("left_out", ["mark", "second_look", "wait", "score_first"])
@pytest.mark.parametrize("owner", [0, 1])
def test_the_model_finds_what_each_step_is_for(left_out, owner):
    assert goes_wrong(2, owner, **{left_out: False})
