"""Wait states around the hand-written copies into LDS, read from the built library's gfx950 code.

The compiler adds the wait states that the hardware does not enforce itself, but does not look inside
inline assembly.  A vector memory instruction needs five after a vector instruction wrote a scalar
register that it reads, and a copy into LDS one after a scalar instruction wrote m0."""
import os
import re
import struct
import subprocess

import pytest

from orthogonalizing_polynomial_cascade_amd import anvil

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
AFTER_VECTOR, AFTER_M0 = 5, 1


def code_objects(path):
    """The gfx950 code objects bundled in a shared library."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + 24)
        entry = at + 32
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + name]
            entry += 24 + name
            if b"gfx950" in target and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 24)


def scalar_registers(operand):
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {int(m.group(1))}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    return set(range(int(m.group(1)), int(m.group(2)) + 1)) if m else set()


def hazards(lines):
    """(copies into LDS, the lines of those that lack a wait state) of one disassembly.  Code that is
    reached from elsewhere within the wait counts as lacking it."""
    code, copies, bad = [], 0, []
    for line in lines:
        text = line.split("//")[0].strip()
        if not text:
            continue
        if text.endswith(":"):
            code.append(("label", [], text))
            continue
        name, _, rest = text.partition(" ")
        code.append((name, [w for w in re.split(r"[,\s]+", rest) if w], text))
    for i, (name, words, text) in enumerate(code):
        if not (name.startswith("buffer_load") and "lds" in words):
            continue
        copies += 1
        reads = set().union(*(scalar_registers(w) for w in words))
        waited = 0
        for name, words, before in reversed(code[max(0, i - AFTER_VECTOR):i]):
            if waited >= AFTER_VECTOR:
                break
            writes = set().union(*(scalar_registers(w) for w in words[:2]))   # results come first
            if (name == "label" or name.startswith(("s_branch", "s_cbranch", "s_setpc"))
                    or name.startswith("v_") and writes & reads
                    or name.startswith("s_") and words[:1] == ["m0"] and waited < AFTER_M0):
                bad.append(f"{before} | {waited} | {text}")
                break
            waited += int(words[0], 0) + 1 if name == "s_nop" else 1
    return copies, bad


def test_scanner():
    copy = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds // 0000: E05D1000"
    assert hazards(["s_mov_b32 m0, s1", copy])[1]
    assert hazards(["v_readfirstlane_b32 s7, v3", "s_mov_b32 m0, s1", "s_nop 2", copy])[1]
    assert hazards(["v_readfirstlane_b32 s9, v3", "s_mov_b32 m0, s1", "s_nop 0", copy])[1]
    assert hazards(["v_add_co_u32 v1, s[6:7], v2, v3", "s_mov_b32 m0, s1", "s_nop 0", copy])[1]
    assert hazards(["<L1>:", "s_mov_b32 m0, s1", "s_nop 0", copy])[1]
    assert hazards(["v_readfirstlane_b32 s7, v3", "s_mov_b32 m0, s1", "s_nop 4", copy]) == (1, [])
    assert hazards(["v_readfirstlane_b32 s7, v3", "s_nop 4", "s_mov_b32 m0, s1", "s_nop 0", copy]) == (1, [])
    assert hazards(["s_mov_b32 m0, s1", "buffer_load_dwordx4 v[0:3], v9, s[4:7], s9 offen"]) == (0, [])


def test_copies_wait_for_their_registers(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    copies, bad = 0, []
    for i, blob in enumerate(code_objects(anvil.LIB_PATH)):
        path = tmp_path / f"code{i}.o"
        path.write_bytes(blob)
        out = subprocess.run([OBJDUMP, "-d", "--symbolize-operands", "--no-show-raw-insn", str(path)], check=True,
                             capture_output=True, text=True).stdout
        n, b = hazards(out.splitlines())
        copies += n
        bad += b
    assert copies > 0, "no copy into LDS found in the library"
    assert not bad, f"{len(bad)} of {copies} copies lack a wait state, for instance {bad[:3]}"
