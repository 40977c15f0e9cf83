"""Rules of the kernel sources that no run shows while they happen to hold.
CPU only."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "pixel_aligned_image_amd", "csrc", "*")))


def statements(text):
    """The asm statements of a source: what stands in each one's brackets."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b\s*(?:volatile)?\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_assembly_names_the_registers_it_writes(path):
    """The compiler learns of a write to m0 from the list only; a load to LDS,
    which reads it, takes it as an operand, so that the compiler writes it."""
    for s in statements(open(path).read()):
        if re.search(r"\b[sv]_\w+\s+m0\b", s):
            assert re.search(r':[^:]*"m0"[^:]*$', s), s
        if "load_lds" in s:
            assert '"{m0}"(' in s, s


def test_the_rule_sees_a_write():
    writes = list(statements('asm volatile("s_mov_b32 m0, %0" :: "s"(f(x)) : "memory");'))
    assert len(writes) == 1 and re.search(r"\b[sv]_\w+\s+m0\b", writes[0])
    assert not re.search(r':[^:]*"m0"[^:]*$', writes[0])


def test_attention_tiles_start_on_whole_rows():
    """Fragments reach a chunk by an exclusive or on the byte address."""
    seen = 0
    for path in SOURCES:
        text = open(path).read()
        if '#include "attn_tile.h"' not in text:
            continue
        for line in re.findall(r"^.*__shared__.*\buint4\b.*$", text, re.M):
            assert "alignas(kTileAlign)" in line, (path, line)
            seen += 1
    assert seen >= 10
    text = open(os.path.join(ROOT, "pixel_aligned_image_amd", "csrc", "attn_tile.h")).read()
    assert int(re.search(r"kTileAlign = (\d+);", text).group(1)) == 256


def test_shared_arrays_are_aligned_as_they_are_read():
    """Scalars in LDS that are read or written as 16-byte vectors say so: what
    lies before them may have any size."""
    for path in SOURCES:
        text = open(path).read()
        for kind, name in re.findall(r"__shared__ ([^;\n]*\b(?:float|float2)) (\w+)\[", text):
            # the array itself, or a pointer set to a place in it
            names = [name] + re.findall(r"\bfloat\s*\*\s*(\w+) = %s\b" % name, text)
            wide = [n for n in names if re.search(
                r"reinterpret_cast<(?:const )?float4\*>\(&?%s\b|\bfactors<N>\(%s\b" % (n, n),
                text)]
            if wide:
                assert re.search(r"\balignas\(16\)|__align__\(16\)", kind), (path, name, wide)
