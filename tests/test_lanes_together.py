"""Matrix instructions write all lanes of their result, also those that are switched off, so no wave may be
at one while some of its lanes wait elsewhere (their registers would be overwritten).  What the compiler makes
of the adapters' kernels is walked along every branch, with the masks that lanes are switched off by."""
import os
import re
import subprocess

import pytest

from epilogue_scaled_gemm_amd import build

MATRIX_OR_BARRIER = re.compile(r"v_mfma|s_barrier|; wave barrier")


def kernels(text):
    name, body = None, []
    for line in text.splitlines():
        start = re.match(r"(\w+):", line)
        if start and not line.startswith(".L"):
            name, body = start.group(1), []
        elif line.startswith(".Lfunc_end"):
            if name:
                yield name, body
            name = None
        elif name:
            body.append(line.strip())


def step(t, off, saved):
    """(masks whose lanes are off, register that last took a copy of exec) behind an instruction."""
    if m := re.match(r"s_\w+_saveexec_b64 (s\[[\d:]+\])", t):
        return tuple(r for r in off if r != m[1]) + (m[1],), saved
    if m := re.match(r"s_mov_b64 (s\[[\d:]+\]), exec$", t):
        return off, m[1]
    if m := re.match(r"s_mov_b64 exec, (\S+)$", t):
        if m[1] == "-1":
            return (), saved
        return (off[:off.index(m[1])] if m[1] in off else off + (saved,)), saved
    if m := re.match(r"s_or_b64 exec, exec, (\S+)$", t):  # (a mask kept elsewhere comes back under another name)
        return (off[:off.index(m[1])] if m[1] in off else off[:-1]), saved
    if m := re.match(r"s_(?:andn2|xor|and)_b64 exec, exec, (\S+)$", t):
        return (off if m[1] in off else off + (m[1],)), saved
    if m := re.match(r"s_xor_b64 (s\[[\d:]+\]), exec, (s\[[\d:]+\])$", t):
        return tuple(m[1] if r == m[2] else r for r in off), saved
    return off, saved


def behind_masks(body):
    """Instructions of MATRIX_OR_BARRIER that are reached with lanes off."""
    code, at = [], {}
    for line in body:
        if m := re.match(r"(\.L\w+):", line):
            at[m[1]] = len(code)
        elif "; wave barrier" in line:
            code.append("; wave barrier")
        elif line and line[0] not in ".;":
            code.append(line.split(";")[0].strip())
    found, seen, todo = set(), set(), [(0, (), "")]
    while todo:
        i, off, saved = todo.pop()
        while i < len(code) and (i, off) not in seen:
            seen.add((i, off))
            t = code[i]
            if off and MATRIX_OR_BARRIER.match(t):
                found.add((i, t))
            off, saved = step(t, off, saved)
            if t.startswith("s_endpgm"):
                break
            if m := re.match(r"s_(c?)branch\w* (\.L\w+)", t):
                if not m[1]:
                    i = at[m[2]]
                    continue
                todo.append((at[m[2]], off, saved))
            i += 1
    return sorted(found)


LOOP = """
k:
 s_mov_b64 s[2:3], 0
.L1:
 {}
 s_or_b64 s[2:3], vcc, s[2:3]
 s_andn2_b64 exec, exec, s[2:3]
 s_cbranch_execnz .L1
 s_or_b64 exec, exec, s[2:3]
 {}
 s_and_saveexec_b64 s[4:5], vcc
 s_cbranch_execz .L2
 {}
.L2:
 s_or_b64 exec, exec, s[4:5]
 {}
 s_endpgm
.Lfunc_end0:
"""


@pytest.mark.parametrize("place,bad", [(0, True), (1, False), (2, True), (3, False)])
@pytest.mark.parametrize("what", ["v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], 0", "; wave barrier"])
def test_the_walk_finds_what_stands_behind_a_mask(place, bad, what):
    (name, body), = kernels(LOOP.format(*[what if i == place else "v_nop" for i in range(4)]))
    assert name == "k" and bool(behind_masks(body)) == bad


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")
def test_adapters_waves_stay_together(tmp_path):
    out = tmp_path / "lora.s"
    subprocess.run([build.HIPCC, *build.FLAGS, "-w", "-x", "hip", "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "kernels_lora.hip"), "-o", str(out)], check=True, capture_output=True)
    walked = 0
    for name, body in kernels(out.read_text()):
        if any("v_mfma" in line for line in body):
            assert not behind_masks(body), name
            walked += 1
    assert walked >= 8
