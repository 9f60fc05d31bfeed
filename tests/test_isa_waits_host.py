"""The built library's gfx950 code against the wait states that the instruction set leaves to software and
that the compiler cannot add inside inline assembly: one between a write of m0 and a load into LDS, which takes its LDS
address from there (the compiler leaves one between those it issues itself), and five between a vector instruction's
write of a scalar register and a memory instruction that reads it."""
import os
import re
import shutil
import subprocess

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_dispatch_grouped_amd", "librdg.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    """Instructions of every kernel, in order; None where another one may come from elsewhere (a kernel's start)."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump here")
    folder = tmp_path_factory.mktemp("isa")
    copy = shutil.copy(LIB, folder / "librdg.so")
    subprocess.run([OBJDUMP, "--offloading", copy], check=True, capture_output=True, cwd=folder)
    out = []
    for name in sorted(os.listdir(folder)):
        if not name.endswith("gfx950"):
            continue
        text = subprocess.run([OBJDUMP, "-d", str(folder / name)], check=True, capture_output=True, text=True).stdout
        for line in text.splitlines():
            line = line.split("//")[0].strip()
            if line.endswith(">:"):
                out.append(None)
            elif line and not line.endswith(":") and not line.startswith("Disassembly"):
                out.append(line)
    assert len(out) > 10000
    return out


def scalars(token):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", token)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", token)
    return {int(m[1])} if m else {"vcc"} if token == "vcc" else set()


def waits(line):
    return int(line.split()[1], 0) + 1 if line.startswith("s_nop") else 1


def test_m0_is_there_before_a_load_into_lds(listing):
    loads = [i for i, x in enumerate(listing) if x and re.match(r"(global|buffer|scratch)_load_lds_|buffer_load_\w+ .*\blds\b", x)]
    assert len(loads) > 100
    early = [(listing[i - 1], listing[i]) for i in loads if listing[i - 1] and re.match(r"s_\w+ m0,", listing[i - 1])]
    assert not early, (len(early), len(loads), early[0])


def test_scalars_that_memory_instructions_read_are_there(listing):
    early = []
    for i, x in enumerate(listing):
        if not x or not re.match(r"(global|buffer|scratch|flat)_", x):
            continue
        read = set().union(*(scalars(t) for t in re.split(r"[ ,]+", x)[1:]))
        gap, k = 0, i - 1
        while read and gap < 5 and listing[k]:
            token = re.split(r"[ ,]+", listing[k])
            written = scalars(token[1]) if token[0].startswith("v_") and len(token) > 1 else set()
            if "_co_" in token[0] or "div_scale" in token[0]:
                written |= scalars(token[2])
            if written & read:
                early.append((listing[k], x))
            gap, k = gap + waits(listing[k]), k - 1
    assert not early, (len(early), early[0])
