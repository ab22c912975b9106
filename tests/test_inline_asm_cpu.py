"""Inline assembly of the kernels, read from their sources: what a block writes it names or puts back, so that the
compiler loses nothing of its own."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_diagonal_eigenbasis_amd", "csrc")


def blocks():
    """(file, instructions, [output, input and clobber sections]) of every asm statement."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))):
        for m in re.finditer(r"\basm\s+volatile\s*\(((?:[^;\"]|\"(?:[^\"\\]|\\.)*\")*)\)\s*;", open(path).read()):
            body = m.group(1)
            text = re.match(r"\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)+)", body).group(0)
            rest = re.sub(r"\"(?:[^\"\\]|\\.)*\"", lambda q: q.group(0).replace(":", "\0"), body[len(text):])
            ins = [i.strip() for i in re.sub(r"\"\s*\"", "", text).strip().strip('"').split("\\n\\t")]
            yield os.path.basename(path), ins, rest.split(":")[1:]


def test_the_reader_finds_every_block():
    n = sum(open(p).read().count("asm volatile") for e in ("*.h", "*.hip") for p in glob.glob(os.path.join(CSRC, e)))
    assert n == len(list(blocks())) > 10


@pytest.mark.parametrize("register,writes", [("scc", r"s_(cmp|add|sub|and|or|xor|lshl|lshr)\w* "), ("vcc", r"\w+ vcc\b"),
                                             ("exec", r"\w+ exec\b")])
def test_what_a_block_writes_is_named(register, writes):
    for path, ins, parts in blocks():
        if any(re.match(writes, i) for i in ins):
            assert len(parts) >= 3 and f'"{register}"' in parts[2], f"{path}: {ins}"


def test_a_block_leaves_m0_as_it_was():
    """(a reserved register: the compiler takes no statement that it is overwritten)"""
    found = 0
    for path, ins, parts in blocks():
        if any(re.match(r"s_\w+ m0\b", i) for i in ins):
            found += 1
            assert ins[0] == "s_mov_b32 %0, m0" and ins[-1] == "s_mov_b32 m0, %0", f"{path}: {ins}"
            assert parts[0].strip().startswith('"=&s"'), f"{path}: {parts}"
    assert found == 2


def test_a_wait_keeps_memory_in_order():
    for path, ins, parts in blocks():
        if any(i.startswith(("s_waitcnt", "s_barrier")) for i in ins):
            assert len(parts) >= 3 and '"memory"' in parts[2], f"{path}: {ins}"
