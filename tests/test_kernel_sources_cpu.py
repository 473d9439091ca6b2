"""Reads the kernels for what no run may show, because it would take a wait that runs out with copies or
products still on their way: every way out of a kernel waits for them first."""

import os
import re

import pytest

import ulysses_sequence_gb300 as U

CSRC = os.path.join(os.path.dirname(U.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def enclosing(text, at):
    """The heads (what stands between the last ;, { or } and the brace) of the blocks around position `at`, and of a
    statement's own condition, inside the kernel."""
    start = text.index("__global__")
    heads, last = [], start
    for i in range(start, at):
        if text[i] == "{":
            heads.append(text[last:i])
        elif text[i] == "}":
            heads.pop()
        if text[i] in "{};":
            last = i + 1
    return heads[1:] + [text[last:at]]


@pytest.mark.parametrize("name,waits", [("paged_decode.cu", 1), ("paged_chunk.cu", 4), ("attn_fwd.cu", 4), ("attn_bwd.cu", 4),
                                        ("proj.cu", 2)])
def test_kernels_wait_for_what_is_on_its_way_whatever_a_role_has_seen(name, waits):
    """A role that finished well does not know that another one has given up since: its copies (the producer) and
    products (the issuer) may still be on their way. So the wait depends on no role's own success."""
    text = source(name)
    found = [m.start() for m in re.finditer(r"\b(?:mbar|ring)_drain\b", text)]
    assert len(found) == waits
    for at in found:
        for head in enclosing(text, at):
            conditional = re.search(r"\bok\b", head) or ("else" in head and "warp ==" not in head)
            assert not conditional, head


ALIGNED = r"\btmem_(?:ld|st|wait|alloc)\w*\("
MEETS = re.compile(r"__syncwarp\(\)|__syncthreads\(\)|__all_sync\(|__any_sync\(|__ballot_sync\(")


@pytest.mark.parametrize("name", ["paged_chunk.cu"])
def test_warps_meet_before_instructions_for_whole_warps(name):
    """tcgen05.ld, .st, .wait and .alloc are for whole converged warps. Where rows leave a loop's turn early, clear their own
    values, or threads loop over their own requests, the warp meets again before the next of them."""
    text = source(name)
    turns = [m.start() for m in re.finditer(r"if \(!valid\) continue;", text)]
    apart = [m.end() for m in re.finditer(r"if \(key0 \+ row >= kv\)|paged_costs<", text)]
    assert turns
    for at in turns:  # the next turn begins at the head of the loop
        at = [m.end() for m in re.finditer(r"\bfor \([^{]*\{", text[:at])][-1]
        before = text[at:at + re.search(ALIGNED, text[at:]).start()]
        assert MEETS.search(before), before
    for at in apart:
        before = text[at:at + re.search(ALIGNED, text[at:]).start()]
        assert MEETS.search(before), before


@pytest.mark.parametrize("name", ["attn_fwd.cu", "attn_bwd.cu", "proj.cu"])
def test_rows_that_store_meet_the_others_before_the_next_columns(name):
    """Where only rows inside the tensor store, or leave the turn, the warp meets before the next columns are read."""
    text = source(name)
    loops = [m.end() for m in re.finditer(r"\bfor \([^{]*\{", text)]
    seen = 0
    for m in re.finditer(r"if \(!valid\) continue;|if \(valid\) \{|if \(row < p\.M\) \{", text):
        for at in (a for a in loops if a < m.start()):
            body = text[at:m.start()]
            inside = body.count("{") >= body.count("}") and all(body[:i].count("{") >= body[:i].count("}") for i in range(len(body)))
            load = re.search(ALIGNED, body)
            if inside and load and "mbar_wait" not in body:  # the loop whose turn reads the columns and stores them
                seen += 1
                assert MEETS.search(body[:load.start()]), body[:load.end()]
    assert seen


def test_the_lane_that_issued_a_reduction_is_back_before_the_next_columns():
    text = source("attn_bwd.cu")
    at = text.index("if (dq_lanes) stage_add(v, acc);")
    before = text[at:at + re.search(ALIGNED, text[at:]).start()]
    assert MEETS.search(before), before
