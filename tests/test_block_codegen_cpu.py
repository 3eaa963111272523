"""What the compiler is held to in the kernels between the products (CPU only:
their gfx950 code is compiled here and read, not run).

Conversions to 8-bit floats saturate while a bit of the MODE register is set,
and BF16 conversions must not run while it is.  Both are pure to the compiler,
so the source ties them to the register writes by empty volatile asm; that it
does is read from the intermediate code, and that the instructions come out in
that order from the assembly.

The fused epilogue hands values between a wave's lanes through LDS without a
barrier; that every such hand-over crosses a wave fence is read from the
intermediate code."""
import os
import re
import subprocess

import pytest

from microscaled_block_scaled_amd import build as B

CVT8 = ("llvm.amdgcn.cvt.scalef32.pk.fp8.f32", "llvm.amdgcn.cvt.scalef32.pk.bf8.f32")


def compiled(source, out, *more):
    """Text of a source's gfx950 code: intermediate code or assembly."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    cmd = [B.HIPCC] + [f for f in B.FLAGS if f != "-shared"] + ["--cuda-device-only", "-S"]
    r = subprocess.run(cmd + list(more) + [source, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return open(out).read()


def functions(ir):
    """{name: lines} of the kernels of intermediate code."""
    found = {}
    for m in re.finditer(r"^define [^\n]*@(\S+?)\(([^\n]*)\{\n(.*?)^\}", ir, re.M | re.S):
        found[m.group(1)] = m.group(3).splitlines()
        parameters[m.group(1)] = re.split(r", (?=ptr|i\d|%)", m.group(2))
    return found


parameters = {}                         # of the functions found: text of each


def mode_problems(lines):
    """Conversions of one function that the intermediate code does not hold to
    their side of the MODE writes: (8-bit windows, problems)."""
    defs, uses, where = {}, {}, {}
    windows, problems, window, block = 0, [], 0, 0
    for n, line in enumerate(lines):
        if re.match(r"\S+:", line):
            block += 1
        m = re.match(r"\s*(%\S+) = ", line)
        if m:
            defs[m.group(1)] = n
        for v in re.findall(r"%[\w.]+", line.split(" = ", 1)[-1]):
            uses.setdefault(v, []).append(n)
        if "llvm.amdgcn.s.setreg" in line and line.lstrip().split()[0] != "declare":
            window = n if re.search(r"i32 1\)", line) else 0
            windows += bool(window)
        where[n] = (block, window)

    def held(v):
        """Whether v comes out of volatile asm: the line of that asm."""
        n = defs.get(v)
        if n is None or "asm sideeffect" in lines[n]:
            return n
        m = re.search(r"= (?:extractvalue|bitcast|insertelement|extractelement|shufflevector)(.*)",
                      lines[n])
        inner = [held(x) for x in re.findall(r"%[\w.]+", m.group(1))] if m else []
        return next((at for at in inner if at is not None), None)

    def goes_to(v, allowed):
        """Whether every use of v is volatile asm or an `allowed` line."""
        for n in uses.get(v, []):
            if "asm sideeffect" in lines[n] or any(a in lines[n] for a in allowed):
                continue
            m = re.match(r"\s*(%\S+) = (bitcast|insertelement|extractelement|shufflevector)", lines[n])
            if not m or not goes_to(m.group(1), allowed):
                return False
        return True

    for n, line in enumerate(lines):
        eight = any(c in line for c in CVT8)
        if not eight and " to <2 x bfloat>" not in line:
            continue
        v = re.match(r"\s*(%\S+) = ", line).group(1)
        if eight:
            s = re.findall(r"float (?:noundef )?(%[\w.]+)", line)[2]      # the scale
        else:
            s = re.search(r"<2 x float> (%[\w.]+)", line).group(1)
        at = held(s)
        if at is None or where[at] != where[n] or bool(where[n][1]) != eight:
            problems.append("operand: " + line.strip())
        if not goes_to(v, CVT8 if eight else ()):
            problems.append("result: " + line.strip())
    return windows, problems


def test_conversions_are_tied_to_the_mode_register(tmp_path):
    ir = compiled(os.path.join(B.CSRC, "mxblock.hip"), str(tmp_path / "block.ll"), "-emit-llvm")
    seen = 0
    for name, lines in functions(ir).items():
        windows, problems = mode_problems(lines)
        if windows:
            seen += 1
            assert not problems, (name, problems[:4])
    assert seen >= 16                       # norm and gated activation, two types, two 8-bit formats


def test_conversions_come_out_in_their_window(tmp_path):
    asm = compiled(os.path.join(B.CSRC, "mxblock.hip"), str(tmp_path / "block.s"))
    eight = wide = 0
    for kernel in re.split(r"\n\t\.globl\t", asm)[1:]:
        on = False
        if "s_setreg" not in kernel:
            continue
        for line in kernel.splitlines():
            if re.match(r"\.?\w+:", line) or re.match(r"\ts_c?branch", line):
                assert not on, kernel[:80]            # a window lies within a block
            m = re.match(r"\ts_setreg_imm32_b32 hwreg\(HW_REG_MODE, 23, 1\), (\d)", line)
            if m:
                assert on != (m.group(1) == "1"), kernel[:80]
                on = m.group(1) == "1"
            if re.search(r"\tv_cvt_scalef32_pk_(fp8|bf8)_f32", line):
                eight += 1
                assert on, kernel[:80]
            if "v_cvt_pk_bf16_f32" in line:
                wide += 1
                assert not on, kernel[:80]
        assert not on
    assert eight >= 64 and wide >= 64, (eight, wide)


FUSED = """
#include <hip/hip_runtime.h>
#include "mx_epilogue.h"
void use(const uint8_t *p, void *c, mx::Epilogue ep)
{
    hipLaunchKernelGGL((mx::tile_kernel<mx::FP8, mx::FP8, mx::OBF16, 128, 128, 2, 2, 3, mx::NoGroups,
                                        mx::Epilogue>),
                       dim3(1), dim3(256), 0, 0, p, p, p, p, c, 1, 1, 512, 1, 1, 4, 512, (int64_t)0,
                       mx::NoGroups{}, ep);
    hipLaunchKernelGGL((mx::tile_kernel<mx::FP8, mx::FP8, mx::OBF16, 128, 128, 2, 2, 3>),
                       dim3(1), dim3(256), 0, 0, p, p, p, p, c, 1, 1, 512, 1, 1, 4, 512, (int64_t)0,
                       mx::NoGroups{}, mx::NoEpilogue{});
}
"""


@pytest.fixture(scope="module")
def fused_ir(tmp_path_factory):
    """Intermediate code of a tile kernel with the fused epilogue (two bands and
    two activation turns a wave) and of one without."""
    at = tmp_path_factory.mktemp("fused")
    (at / "fused.hip").write_text(FUSED)
    return functions(compiled(str(at / "fused.hip"), str(at / "fused.ll"), "-emit-llvm"))


def unfenced(lines):
    """(LDS stores, pairs of LDS accesses that different lanes' copies of can
    meet without a wave fence between).  A band's sums are staged; reads by
    other lanes follow, by way of an activation that rewrites each value in the
    lane that read it; then the next band."""
    blocks, name = {None: []}, None
    for line in lines:
        m = re.match(r"(\S+):", line)
        if m:
            name = m.group(1)
            blocks[name] = []
        else:
            blocks[name].append(line)
    text = {b: "\n".join(ls) for b, ls in blocks.items()}
    nexts = {b: re.findall(r"label %(\S+?)(?:[,\s\]]|$)", t) for b, t in text.items()}

    def access(line):
        if "addrspace(3)" not in line or " = getelementptr" in line:
            return None
        if re.search(r"\bstore .*ptr addrspace\(3\)", line):
            return "store"
        if re.search(r"= load .*ptr addrspace\(3\)", line):
            return "load"
        return None

    def reach(block, at):
        """The LDS accesses after line `at` of a block up to a fence."""
        found, seen, todo = set(), set(), [(block, at + 1)]
        while todo:
            b, i = todo.pop()
            if (b, i) in seen:
                continue
            seen.add((b, i))
            for n in range(i, len(blocks[b])):
                if 'fence syncscope("wavefront")' in blocks[b][n] or "s_barrier" in blocks[b][n]:
                    break
                if access(blocks[b][n]):
                    found.add((b, n))
            else:
                todo += [(x, 0) for x in nexts[b]]
        return found

    kind = {(b, n): access(line) for b, ls in blocks.items() for n, line in enumerate(ls) if access(line)}
    to = {p: reach(*p) for p in kind}
    # a value's own rewriting in a loop reaches back to where it was read
    bad = [(p, q) for p in kind for q in to[p] if {kind[p], kind[q]} == {"load", "store"} and p not in to[q]]
    return sum(k == "store" for k in kind.values()), bad


def test_staged_sums_are_fenced_between_lanes(fused_ir):
    (lines,) = [ls for n, ls in fused_ir.items() if "Epilogue" in n and "NoEpilogue" not in n]
    stores, bad = unfenced(lines)
    assert stores >= 64
    assert not bad, (len(bad), bad[:4])


def test_c_may_be_the_residual(fused_ir):
    """The compiler is told that nothing else addresses C in the kernels
    without an epilogue, and is not told so where C may be the residual."""
    told = {"noalias" in parameters[n][4] for n in fused_ir if "NoEpilogue" in n}
    assert told == {True}
    told = {"noalias" in parameters[n][4] for n in fused_ir if "NoEpilogue" not in n and "Epilogue" in n}
    assert told == {False}
