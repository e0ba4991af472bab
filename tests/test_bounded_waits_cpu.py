"""What follows a wait that gives up, read from the sources of the kernels over the 8-bit cache.

A bounded wait returns per lane.  If some lanes of a warp gave up and others went on, they would meet
at different warp-wide instructions; and a CTA that leaves, or uses its shared memory again, while a
copy is still on its way is written over.  (No wait is made to run out on a GPU for this.)"""
import os
import re

import pytest

import exact_attention_158_b200 as fa

CSRC = os.path.join(os.path.dirname(fa.__file__), "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def waits(text):
    """(statement up to the wait, headers of the blocks around it) of every mbar_wait call."""
    blocks, start = [], 0
    for m in re.finditer(r"[{};]|\bmbar_wait\(", text):
        if m.group() == "{":
            blocks.append(text[start:m.start()])
        elif m.group() == "}":
            blocks.pop()
        elif m.group() != ";":
            yield text[start:m.start()], list(blocks)
            continue
        start = m.end()


@pytest.mark.parametrize("name", ["fa_q8.cuh", "fa_q8_tile.cuh"])
def test_a_warp_agrees_on_its_waits(name):
    found = list(waits(source(name)))
    assert found
    for statement, blocks in found:
        one_thread = any("lane == 0" in b for b in blocks + [statement])
        assert one_thread or "__all_sync(0xffffffffu" in statement, statement.strip()


@pytest.mark.parametrize("name,first_use", [("fa_q8.cuh", "float *part ="), ("fa_q8_tile.cuh", None)])
def test_copies_land_before_shared_memory_is_used_again(name, first_use):
    text = source(name)
    if first_use is None:  # the loader stays until its copies have landed; nothing is written then
        assert re.search(r"if \(\*abort_flag\) \{\s*const uint64_t t0 = globaltimer_ns\(\);", text)
        return
    # a warp that leaves its loop early waits for the stages that it has asked for, the CTA joins, and
    # one that gave up leaves before the ring becomes the merge's memory
    before = text[:text.index(first_use)]
    loop = before.rindex("for (int i = 0; i < n_mine; ++i)")
    assert re.search(r"mbar_wait\([^;]*&never\)", before[loop:])
    joined = before.rindex("__syncthreads();")
    assert re.search(r"if \(.*\*gave_up\) \{.*return;", before[joined:], flags=re.S)
