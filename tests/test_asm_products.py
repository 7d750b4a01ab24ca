"""Static check of the matrix instructions that the tiled products issue in
inline asm, so as to keep their accumulators in place.

The compiler does not know that these are matrix instructions, so it leaves no
room where one needs it: an instruction that writes a vector register has to be
two slots ahead of a matrix instruction that reads it, and nothing else may
touch the accumulators between the first of them and the wait behind the last.
This test compiles the kernels for gfx950 and walks the generated code of the
main loops.
"""
import os
import re
import subprocess
import tempfile

import lossless_compression_float_amd.build as b

SRC = os.path.join(b.CSRC, "uzip_linear.hip")
REG = re.compile(r"\b([va])(\d+)\b|\b([va])\[(\d+):(\d+)\]")


def regs(text, kind):
    out = set()
    for k1, one, k2, lo, hi in REG.findall(text):
        if k1 == kind:
            out.add(int(one))
        elif k2 == kind:
            out.update(range(int(lo), int(hi) + 1))
    return out


def kernels(text):
    """(name, its instruction lines; None for a label) of every tiled product whose matrix instructions come from asm."""
    name, lines, asm, inline = None, [], False, False
    for raw in text.splitlines():
        m = re.match(r"^(_ZN\S*k_gemm\S*):", raw)
        if m:
            name, lines, asm, inline = m.group(1), [], False, False
        elif name:
            asm = "#ASMSTART" in raw or (asm and "#ASMEND" not in raw)
            inline = inline or (asm and "v_mfma" in raw)
            s = raw.split(";")[0].strip()
            if re.match(r"^\.LBB\S*:", s):
                lines.append(None)
            elif s.startswith("s_endpgm"):
                if inline:
                    yield name, lines
                name = None
            elif s and not s.startswith("."):
                lines.append(s)


def check(lines):
    bad, products = [], 0
    first = next(i for i, s in enumerate(lines) if s and s.startswith("v_mfma"))
    last = max(i for i, s in enumerate(lines) if s and s.startswith("v_mfma"))
    for i, s in enumerate(lines):
        if s is None or not s.startswith("v_mfma"):
            continue
        products += 1
        ops = [o.strip() for o in s.split(None, 1)[1].split(",")]
        if ops[0] != ops[3] or not ops[0].startswith("a"):
            bad.append("not in place: " + s)
        need = regs(ops[1], "v") | regs(ops[2], "v")
        slots = 0
        for p in reversed(lines[:i]):
            if slots >= 2:
                break
            if p is None:  # a label: what comes before is not known, but a jump takes longer than two slots
                break
            if p.startswith("v_") and not p.startswith("v_mfma") and regs(p.split(",")[0], "v") & need:
                bad.append("%s right before %s" % (p, s))
            m = re.match(r"s_nop (\d+)", p)
            slots += int(m.group(1)) + 1 if m else 1
    inner = lines[first:last]
    bad += ["accumulator touched in the loop: " + s for s in inner if s and not s.startswith("v_mfma") and regs(s, "a")]
    return bad, products


def test_asm_products_have_room():
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        flags = [f for f in b.HIPCC_FLAGS if f not in ("-shared",)]
        subprocess.check_call([hipcc] + flags + ["--cuda-device-only", "-S", "-o", out, SRC], stderr=subprocess.DEVNULL)
        text = open(out).read()
    seen = 0
    for name, lines in kernels(text):
        bad, products = check(lines)
        assert not bad, (name, bad[:5])
        assert products >= 16, name
        seen += 1
    assert seen >= 9
    # (the check itself: a planted write right before a product is found)
    assert check(["v_mov_b32_e32 v5, 0", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]", "s_nop 0",
                  "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]"])[0]
