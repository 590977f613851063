"""The barriers of the tiled 8-bit GEMM wait by count: a wave waits until at most
N of its memory instructions are on their way, N being what it has issued since
the token rows that the barrier stands for.  That holds only as long as the
compiler keeps every load that the count includes, in its place.  This test
compiles the kernel to gfx950 assembly and follows every path through it: at
each barrier of an item's loop, whatever the path, the rows of the next chunk
have to be among those waited for.

Memory instructions end in their order of issue, as far as the counter tells, so
after a wait for N the last N issued may be on their way and no others.  An item
issues (scales) (scales) (rows of chunk 0) .. (rows of chunk 2); its barrier number
b, from 0, is for the rows of chunk b.
"""

import os
import re
import subprocess

import pytest

from quantized_moe_amd import build as B

DEPTH = 64  # the counter holds 63 at most


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "f8_tile.s")
    cmd = [B.HIPCC, *B.COMMON, "--cuda-device-only", "-S", "-x", "hip", os.path.join(B.CSRC, "f8_tile.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        return f.read()


def kernels(text):
    """{name: [(label, events, successors)]}: an event is "X" (rows to LDS), "S"
    (scales to LDS), "W" (weights), "o" (other memory), ("wait", n) or "bar"."""
    found = {}
    for part in text.split("\t.globl\t")[1:]:
        name = part.split()[0].split(",")[0]
        if "f8_tile" not in name:
            continue
        blocks, label, events, to, open_ = [], "entry", [], [], True
        for line in part.split("\n"):
            t = line.split(";")[0].strip()
            m = re.match(r"^(\.LBB\w+):", t)
            if m:
                if open_:
                    to.append(m.group(1))
                blocks.append((label, events, to))
                label, events, to, open_ = m.group(1), [], [], True
                continue
            if not t or not open_:
                continue
            op = t.split()[0]
            if op == "s_endpgm" or op == "s_branch":
                if op == "s_branch":
                    to.append(t.split()[1])
                open_ = False
            elif op.startswith("s_cbranch"):
                # what follows in the text is a block of its own
                target, rest = t.split()[1], f"{label}+{len(blocks)}"
                blocks.append((label, events, to + [target, rest]))
                label, events, to = rest, [], []
            elif op.startswith("buffer_load") and t.endswith(" lds"):
                events.append("X" if op.endswith("dwordx4") else "S")
            elif op.startswith("buffer_load"):
                events.append("W")
            elif re.match(r"(global|flat|scratch|buffer)_(load|store|atomic)", op):
                events.append("o")
            elif op == "s_waitcnt":
                m = re.search(r"vmcnt\((\d+)\)", t)
                if m:
                    events.append(("wait", int(m.group(1))))
            elif op == "s_barrier":
                events.append("bar")
        blocks.append((label, events, to))
        found[name] = blocks
    return found


def faults(blocks):
    """What is wrong on some path, as texts, and the barriers looked at.

    A path's state: the memory instructions that may be on their way (oldest
    first), the groups of rows issued minus the barriers passed minus one (so the
    groups that may be on their way at a barrier), rows issued of a group not yet
    whole, and the loads of a group (0 in front of an item's first barrier)."""
    where = {b[0]: b for b in blocks}
    wrong, looked = set(), set()
    seen = set()
    todo = [(blocks[0][0], ("", -1, 0, 0))]
    while todo:
        label, state = todo.pop()
        if (label, state) in seen:
            continue
        seen.add((label, state))
        ops, slack, part, size = state
        last = ""
        for i, ev in enumerate(where[label][1]):
            if isinstance(ev, tuple):
                ops = ops[-ev[1]:] if ev[1] else ""
            elif ev == "bar":
                if size == 0 and part:  # an item's first: three groups were issued
                    if part % 3:
                        wrong.add(f"{label}: {part} loads of rows in front of the first barrier")
                    size, slack, part = max(1, part // 3), 2, 0
                flying = ops.count("X")
                if flying:
                    looked.add((label, i))
                if flying > max(slack, 0) * size:
                    wrong.add(f"{label}, barrier at {i}: {flying} loads of rows may be on their way, "
                              f"{max(slack, 0) * size} allowed")
                slack = max(slack - 1, -1)
            else:
                if ev == "S" and last == "S":  # a new item
                    slack, part, size = -1, 0, 0
                if ev == "S" and (part or last == "X"):
                    wrong.add(f"{label}: scales behind rows at {i}")
                if ev == "X":
                    part += 1
                    if size and part == size:
                        slack, part = slack + 1, 0
                ops = (ops + ev)[-DEPTH:]
            if ev != "W":
                last = ev
        for t in where[label][2]:
            todo.append((t, (ops, slack, part, size)))
    return wrong, looked


def test_rows_have_landed_at_every_barrier(assembly):
    found = kernels(assembly)
    assert len(found) == 7, sorted(found)
    for name, blocks in found.items():
        wrong, looked = faults(blocks)
        assert not wrong, (name, sorted(wrong)[:5])
        # an item's first barrier, four in the loop, for each height of tile
        assert len(looked) >= (5 if "ELi32E" in name else 35), (name, len(looked))


def loop_of(assembly, kernel):
    """(start, end) of the text of the first loop of four barriers of a kernel."""
    at = re.search(r"^\S*%s\S*:" % kernel, assembly, re.M).start()
    for m in re.finditer(r"^(\.LBB\w+):.*?s_cbranch_scc\d \1$", assembly[at:], re.M | re.S):
        body = assembly[at + m.start():at + m.end()]
        if body.count("s_barrier") == 4 and "\n.LBB" not in body:
            return at + m.start(), at + m.end()
    raise AssertionError("no loop found")


@pytest.mark.parametrize("kernel", ["f8_tileILi1ELi32ELi4ELi1", "f8_tileILi1ELi32ELi4ELi2"])
def test_a_lost_or_moved_load_is_noticed(assembly, kernel):
    """The same text with one load of weights taken out of the loop, with a larger
    count at a barrier, and with scales behind the rows.  (Weights three chunks ahead,
    and no wait of the compiler's own in the loop that would cover for it.)"""
    lo, hi = loop_of(assembly, kernel)
    body = assembly[lo:hi]

    def verdict(new):
        return faults([v for n, v in kernels(assembly[:lo] + new + assembly[hi:]).items() if kernel in n][0])[0]

    assert not verdict(body)
    loads = list(re.finditer(r"^\tbuffer_load_dwordx4 .*(?<! lds)\n", body, re.M))
    assert len(loads) == 16
    for m in loads[::5]:
        assert verdict(body[:m.start()] + body[m.end():])
    waits = [m for m in re.finditer(r"vmcnt\((\d+)\)(?=\n\ts_barrier)", body)]
    assert len(waits) == 4
    for m in waits:
        assert verdict(body[:m.start()] + f"vmcnt({int(m.group(1)) + 1})" + body[m.end():])
    lines = body.split("\n")
    scale = next(i for i, l in enumerate(lines) if l.strip().startswith("buffer_load_dword ") and l.endswith("lds"))
    rows = next(i for i in range(scale, len(lines)) if "buffer_load_dwordx4" in lines[i] and lines[i].endswith("lds"))
    lines.insert(rows + 1, lines[scale])
    del lines[scale]
    assert verdict("\n".join(lines))
