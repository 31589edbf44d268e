"""The order of the softmax warps' accesses to what they share, read from the kernel's source (CPU).

Four warps hold a quarter of each head's scores and exchange two numbers through ``ms.red``: the maximum of a tile
whose reference moves, and at an item's end the sum.  Every warp writes its own entry and reads all four, so a group
barrier has to lie between a write and the reads, and between the reads and the next write, whichever branches a
tile takes.  The tile's code is walked for every course of tiles, events in the order of the source.
"""

import itertools
import os
import re

SOURCE = os.path.join(os.path.dirname(__file__), "..", "mqa_flash_attention_gb300", "csrc", "tree_attn.cu")
EVENTS = re.compile(r"(?P<write>ms\.red\[box\]\[h\] = )|(?P<read>ms\.red\[0\]\[h\])|(?P<barrier>bar_(?:red_or|sync_id)\(group)"
                    r"|(?P<skip>continue;)|(?P<leave>break;)")


def closing(text, at, pair):
    """Index behind the bracket that closes the one at ``at``."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("brackets do not match")


def tile_body():
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    role = text[text.index("void tree_softmax_role("):]
    loop = role[role.index("for (int g = 0; g < nt; ++g) {"):]
    return loop[loop.index("{") + 1:closing(loop, loop.index("{"), "{}") - 1]


def parse(text):
    """Nested list of event names and (condition, its events, branch, else branch); loops count as their body."""
    out, i = [], 0
    while i < len(text):
        m = re.compile(r"\b(if|for|while)\s*\(").search(text, i)
        e = EVENTS.search(text, i)
        if e and (not m or e.start() < m.start()):
            out.append(e.lastgroup)
            i = e.end()
            continue
        if not m:
            return out
        end = closing(text, m.end() - 1, "()")
        cond, head = text[m.end():end - 1], m.group(1)
        body, i = branch(text, end)
        other = []
        tail = re.compile(r"\s*else\b").match(text, i)
        if head == "if" and tail:
            other, i = branch(text, tail.end())
        if head != "if":
            out += body
        elif body or other or EVENTS.search(cond):
            out.append((cond, parse(cond), body, other))
    return out


def branch(text, at):
    at += len(text[at:]) - len(text[at:].lstrip())
    if text[at] == "{":
        end = closing(text, at, "{}")
        return parse(text[at + 1:end - 1]), end
    # A single statement, which may itself begin with a condition.
    m = re.compile(r"(if|for|while)\s*\(").match(text, at)
    end = closing(text, m.end() - 1, "()") if m else at
    if m:
        _, end = branch(text, end)
    else:
        end = text.index(";", at) + 1
    return parse(text[at:end]), end


def holds(cond, first, last, moved):
    if "top > m_lim" in cond:
        return moved
    if cond == "bad" or EVENTS.search(cond):
        return False  # a vote that some wait ran out
    code = re.sub(r"\(?flags & TF_(FIRST|LAST)\)?", lambda m: m.group(1).lower(), cond)
    code = code.replace("&&", " and ").replace("||", " or ").replace("!", " not ")
    return bool(eval(code.strip(), {"first": first, "last": last, "moved": moved}))  # NameError: a new condition


def walk(items, *tile):
    """Events of a tile; the last one is "skip" or "leave" if it ended early."""
    for x in items:
        if isinstance(x, str):
            yield x
            if x in ("skip", "leave"):
                return
            continue
        cond, in_cond, body, other = x
        yield from in_cond
        ended = False
        for e in walk(body if holds(cond, *tile) else other, *tile):
            yield e
            ended = e in ("skip", "leave")
        if ended:
            return


def courses():
    """Tiles (first, last, moved) of items of one to three tiles."""
    for lengths in itertools.product((1, 2, 3), repeat=2):
        flags = [(j == 0, j == n - 1) for n in lengths for j in range(n)]
        for moved in itertools.product((False, True), repeat=len(flags)):
            yield [(*f, m) for f, m in zip(flags, moved)]


def test_the_walk_finds_the_events():
    """One tile of one item whose reference moves: maxima, then the sum."""
    got = [e for e in walk(parse(tile_body()), True, True, True) if e != "skip"]
    assert [e for e in got if e != "barrier"] == ["write", "read", "write", "read"] and got.count("barrier") >= 4


def test_shared_numbers_are_read_before_they_are_written_again():
    body = parse(tile_body())
    for tiles in courses():
        unread, unmet = False, False  # written and not yet behind a barrier; read and not yet behind one
        for tile in tiles:
            for e in walk(body, *tile):
                if e == "barrier":
                    unread = unmet = False
                elif e == "write":
                    assert not unmet, f"a warp may write while another still reads: tiles (first, last, moved) {tiles}"
                    unread = True
                elif e == "read":
                    assert not unread, f"a warp may read what another has not written: {tiles}"
                    unmet = True
                assert e != "leave"


def test_threads_leave_the_tiles_together():
    """When a wait has run out in some threads, all of the group have to know before an output is taken behind the
    loop: those that did not would do so in steps that need whole warps, and wait there without end."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body, role = tile_body(), text[text.index("void tree_softmax_role("):]
    for m in re.finditer(r"\bbreak;", body):  # all leave the loop at once
        assert body[:m.start()].endswith("if (bar_red_or(group, 128, bad)) ")
    behind = role[role.index(body) + len(body):]
    assert re.match(r"\s*\}\s*if \(pending && !bar_red_or\(group, 128, bad\)\) drain\(nt\);\s*\}", behind)


def test_a_loader_leaves_with_all_its_lanes():
    """One lane of a loader waits for Q's buffer.  Its warp votes in every later wait: if that lane gave up alone, the
    others would wait for it without end."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    role = text[text.index("void tree_load_role("):text.index("void tree_widen_role(")]
    loop = role[role.index("for (int g = 0; g < nt && ok; ++g) {"):]
    alone = [m.start() for m in re.finditer(r"ok = false;", loop[:closing(loop, loop.index("{"), "{}")])]
    assert len(alone) == 2
    q_wait, kv_wait = alone
    assert re.match(r"[^$]*?if \(__any_sync\(0xffffffffu, !ok\)\) break;", loop[q_wait:loop.index("for (int c = 0;")])
    # Already a vote's result.
    assert re.search(r"if \(!__all_sync\(0xffffffffu, wait_phase\([^{]*\{\s*$", loop[:kv_wait])
