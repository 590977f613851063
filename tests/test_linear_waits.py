"""The 16-bit product waits by counts: a wave goes on when at most N of its loads to
LDS are on their way, N being those that it has issued since the ones it needs.  That
holds as long as the compiler leaves every load in its place.  This test compiles both
forms to gfx950 assembly and looks at the loops that wait so.

Tiled form, steady loop: the loads of x of a chunk, a wait, the barrier, the loads of
W.  The next chunk's x is older than XS - 2 chunks' loads, its W than W of WS - 2
chunks and x of WS - 1; the count has to be the smaller of the two.  Streaming form:
DEPTH groups of loads are on their way at each wait, of which DEPTH - 1 may be, and a
slot is loaded again only when its reads have arrived."""

import os
import re
import subprocess

import pytest

from quantized_moe_amd import build as B



def compiled(tmp_path_factory, name):
    out = str(tmp_path_factory.mktemp("asm") / (name + ".s"))
    cmd = [B.HIPCC, *B.COMMON, "--cuda-device-only", "-S", "-x", "hip", os.path.join(B.CSRC, name + ".hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        return f.read()


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    return compiled(tmp_path_factory, "linear_tile")


@pytest.fixture(scope="module")
def stream(tmp_path_factory):
    return compiled(tmp_path_factory, "linear")


def kernels(text, name):
    """{template arguments: [(label, events, last branch's target)]} of the kernels."""
    found = {}
    for part in text.split("\t.globl\t")[1:]:
        symbol = part.split()[0].split(",")[0]
        if name not in symbol:
            continue
        arguments = tuple(int(v) for v in re.findall(r"L[bi](\d+)E", symbol.split(name)[1]))
        blocks, label, events = [], "entry", []
        for line in part.split("\n"):
            t = line.split(";")[0].strip()
            m = re.match(r"^(\.LBB\w+):", t)
            op = t.split()[0] if t else ""
            if m or op.startswith(("s_branch", "s_cbranch", "s_endpgm")):
                blocks.append((label, events, "" if m or op == "s_endpgm" else t.split()[1]))
                label, events = m.group(1) if m else label + "+", []
            elif op.startswith("buffer_load") and t.endswith(" lds"):
                events.append("load")
            elif re.match(r"(global|flat|scratch|buffer)_(load|store|atomic)", op):
                events.append("other")
            elif op.startswith("ds_read"):
                events.append("read")
            elif op.startswith("v_mfma"):
                events.append("product")
            elif op == "s_barrier":
                events.append("barrier")
            elif op == "s_waitcnt":
                v, l = re.search(r"vmcnt\((\d+)\)", t), re.search(r"lgkmcnt\((\d+)\)", t)
                events.append(("wait", int(v.group(1)) if v else None, int(l.group(1)) if l else None))
            if op == "s_endpgm":
                break
        found[arguments] = blocks
    return found


def tile_faults(arguments, blocks):
    """(what is wrong, steady loops seen) of a kernel of the tiled form."""
    _, WM, WN, MG, NT, XS, WS, _, CUT = arguments
    waves, w = WM * WN, WN * NT * 2 // (WM * WN)  # loads of W in a chunk
    heights = {}  # products of a chunk: (loads of x, younger than a chunk's, younger than the first chunk's)
    for m in (MG, MG // 2) if CUT else (MG,):  # (a last round of half the height)
        x = WM * m * 2 // waves
        heights[2 * m * NT] = x, min((XS - 2) * (x + w), (WS - 1) * x + (WS - 2) * w), (XS - 2) * x + (WS - 1) * w
    wrong, steady = [], 0
    for label, events, to in blocks:
        if events.count("product") in heights and to == label and events.count("barrier") == 1:
            steady += 1
            x, count, _ = heights[events.count("product")]
            memory = [e for e in events if e in ("load", "other", "barrier")]
            if memory != ["load"] * x + ["barrier"] + ["load"] * w:
                wrong.append(f"{label}: {memory}")
            at = events.index("barrier")
            if events[at - 1] != ("wait", count, 0):
                wrong.append(f"{label}: {events[at - 1]} in front of the barrier, {count} loads are younger")
            continue
        for i, e in enumerate(events):  # elsewhere only the count in front of the first chunk
            if e == "barrier" and i and events[i - 1][0] == "wait" and \
                    events[i - 1][1] not in [None, 0] + [h[2] for h in heights.values()]:
                wrong.append(f"{label}: {events[i - 1]}")
    return wrong, steady


def test_tiles_have_landed(tile):
    found = kernels(tile, "linear_tile")
    assert len(found) == 8, sorted(found)
    for arguments, blocks in found.items():
        wrong, steady = tile_faults(arguments, blocks)
        assert not wrong, (arguments, wrong[:5])
        assert steady == 1 + arguments[-1], (arguments, steady)


def test_a_lost_or_moved_load_of_a_tile_is_noticed(tile):
    steady = [(arguments, blocks, n) for arguments, blocks in kernels(tile, "linear_tile").items()
              for n, (label, events, to) in enumerate(blocks)
              if to == label and events.count("barrier") == 1 and "product" in events]
    assert len(steady) == 10
    for arguments, blocks, n in steady:
        label, events, to = blocks[n]
        at = events.index("barrier")
        load = events.index("load")
        for changed in (events[:load] + events[load + 1:], events[:at] + ["load"] + events[at:],
                        events[:at - 1] + [("wait", events[at - 1][1] + 1, 0)] + events[at:], events + ["other"]):
            assert tile_faults(arguments, blocks[:n] + [(label, changed, to)] + blocks[n + 1:])[0]


def test_streamed_chunks_have_landed(stream):
    found = kernels(stream, "linear_stream")
    assert len(found) == 6, sorted(found)
    for (_, groups, depth), blocks in found.items():
        loads = 2 + groups
        products = [i for i, b in enumerate(blocks) if "product" in b[1]]
        assert len(products) == 1 and blocks[products[0]][1].count("product") == groups, products
        at = products[0]
        events = blocks[at][1]
        # the reads of a slot have arrived before anything is loaded again
        assert "load" not in events and "other" not in events
        behind = [e for e in events[len(events) - 1 - events[::-1].index("read"):] if e[0] == "wait"]
        assert any(e[2] == 0 for e in behind), events
        # every group of loads is whole
        for label, e, _ in blocks:
            assert e.count("load") in (0, loads), (label, e.count("load"))
        assert sum("load" in b[1] for b in blocks) == depth + 1
        # in front of the reads: all but depth - 1 groups, or all
        start = next(i for i, b in enumerate(blocks) if "load" in b[1])
        counts = {e[1] for b in blocks[start:at] for e in b[1] if e[0] == "wait" and e[1] is not None}
        assert counts == {0, (depth - 1) * loads}, counts
