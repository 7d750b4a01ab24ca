"""Static check of the room in front of the inline matrix instructions along
every way that leads to them: through labels by falling in, and by jumps."""
import os
import re
import subprocess
import tempfile

import lossless_compression_float_amd.build as b
from test_asm_products import SRC, regs

JUMP = re.compile(r"s_c?branch\S*\s+(\.LBB\S+)")


def kernels(text):
    """(name, instruction lines and labels) of every tiled product whose matrix instructions come from asm."""
    name, lines, asm, inline = None, [], False, False
    for raw in text.splitlines():
        m = re.match(r"^(_ZN\S*k_gemm\S*):", raw)
        if m:
            name, lines, asm, inline = m.group(1), [], False, False
        elif name:
            asm = "#ASMSTART" in raw or (asm and "#ASMEND" not in raw)
            inline = inline or (asm and "v_mfma" in raw)
            s = raw.split(";")[0].strip()
            if s.startswith("s_endpgm") and raw.startswith("\t"):
                lines.append(s)
            elif s.startswith(".Lfunc_end"):
                if inline:
                    yield name, lines
                name = None
            elif s and (s.startswith(".LBB") or not s.startswith(".")):
                lines.append(s)


def check(lines):
    """Vector registers written less than two slots ahead of a matrix instruction that reads them, over all ways."""
    jumps = {}
    for i, s in enumerate(lines):
        m = JUMP.match(s)
        if m:
            jumps.setdefault(m.group(1), []).append(i)
    bad, products, through = [], 0, 0
    for i, s in enumerate(lines):
        if not s.startswith("v_mfma"):
            continue
        products += 1
        ops = [o.strip() for o in s.split(None, 1)[1].split(",")]
        need = regs(ops[1], "v") | regs(ops[2], "v")
        todo, seen = [(i - 1, 0)], set()
        while todo:
            j, slots = todo.pop()
            if j < 0 or slots >= 2 or (j, slots) in seen:
                continue
            seen.add((j, slots))
            p = lines[j]
            if p.endswith(":"):
                through += 1
                todo += [(k, slots) for k in jumps.get(p[:-1], [])]
                if not re.match(r"s_branch|s_setpc|s_endpgm", lines[j - 1]):  # (behind those only a jump leads here)
                    todo.append((j - 1, slots))
                continue
            if p.startswith("v_") and not p.startswith("v_mfma") and regs(p.split(",")[0], "v") & need:
                bad.append("%s right before %s" % (p, s))
            m = re.match(r"s_nop (\d+)", p)
            todo.append((j - 1, slots + (int(m.group(1)) + 1 if m else 1)))
    return bad, products, through


PRODUCT = "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]"


def test_the_walk_finds_planted_writes():
    write = "v_mov_b32_e32 v5, 0"
    assert check([write, ".LBB0_1:", PRODUCT])[0]                                     # by falling in
    assert check([write, "s_cbranch_scc1 .LBB0_1", "s_nop 7", ".LBB0_1:", PRODUCT])[0]  # by a jump over the room
    assert check([".LBB0_1:", PRODUCT, write, "s_cbranch_scc1 .LBB0_1"])[0]           # round a loop
    assert not check([write, "s_branch .LBB0_2", ".LBB0_1:", PRODUCT])[0]             # not reached from the write
    assert not check([write, "s_nop 1", ".LBB0_1:", PRODUCT])[0]
    assert not check([write.replace("v5", "v12"), ".LBB0_1:", PRODUCT])[0]


def test_asm_products_have_room_on_every_way():
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        flags = [f for f in b.HIPCC_FLAGS if f not in ("-shared",)]
        subprocess.check_call([hipcc] + flags + ["--cuda-device-only", "-S", "-o", out, SRC], stderr=subprocess.DEVNULL)
        text = open(out).read()
    seen = through = 0
    for name, lines in kernels(text):
        bad, products, labels = check(lines)
        assert not bad, (name, bad[:5])
        assert products >= 16, name
        seen, through = seen + 1, through + labels
    assert seen >= 9 and through > 0
