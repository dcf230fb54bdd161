"""The assembly of the kernels that run with nearly all registers in use, compiled here,
searched for two mistakes that no result of an ordinary size would show:

- a vector instruction between the label where lanes join again and the instruction
  that switches them on: lanes that had skipped the block never execute it.  The compiler
  has placed a live register's copy there;
- a scalar register that a vector instruction wrote, read by a load of inline assembly
  less than five wait states later: the compiler inserts waits for its own loads only.
"""
import os
import re
import shutil
import subprocess

import pytest

from parameter_layout_collectives_amd import build

FILES = ["ortho.hip", "fp4_mm.hip", "block_mm.hip"]


def functions(text):
    """{name: [(label, [(instruction, in inline assembly)])]}: basic blocks in order."""
    out, blocks, asm = {}, None, False
    for line in text.split("\n"):
        t = line.strip()
        m = re.match(r"(_Z\w+):", line)
        if m:
            blocks = out.setdefault(m[1], [("entry", [])])
        elif line.startswith(".Lfunc_end"):
            blocks = None
        if blocks is None or m:
            continue
        m = re.match(r"(\.LBB\d+_\d+):", line)
        if m:
            blocks.append((m[1], []))
        elif "ASMSTART" in t or "ASMEND" in t:
            asm = "ASMSTART" in t
        elif t and t[0] not in ";.":
            blocks[-1][1].append((t, asm))
            if re.match(r"s_(cbranch|branch)", t):
                blocks.append((f"{len(blocks)}", []))
    return out


def before_lanes_join(blocks):
    """Vector instructions at the head of a block that a branch over masked lanes
    targets, before the lanes are switched on again."""
    targets = {m[1] for _, b in blocks for t, _ in b for m in [re.match(r"s_cbranch_execz (\S+)", t)] if m}
    bad = []
    for label, b in blocks:
        if label not in targets:
            continue
        seen = []
        for t, _ in b:
            if t.startswith("s_or_b64 exec, exec"):
                bad += seen
                break
            if re.match(r"s_(cbranch|branch|\w+_saveexec|\w+ exec)", t):
                break
            if re.match(r"(v|ds|global|buffer|flat|scratch)_", t):
                seen.append(f"{label}: {t}")
    return bad


def scalars(t):
    out = set()
    for a, b, c in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", t):
        out |= {int(c)} if c else set(range(int(a), int(b) + 1))
    return out


def loads_too_soon(blocks):
    """Loads of inline assembly within five wait states of a vector instruction that
    wrote one of their scalar registers, on any path."""
    before = [set() for _ in blocks]
    at = {label: i for i, (label, _) in enumerate(blocks)}
    for i, (_, b) in enumerate(blocks):
        last = b[-1][0] if b else ""
        m = re.match(r"s_(?:cbranch_\w+|branch) (\.LBB\S+)", last)
        if m and m[1] in at:
            before[at[m[1]]].add(i)
        if not last.startswith(("s_branch", "s_endpgm")) and i + 1 < len(blocks):
            before[i + 1].add(i)

    def back(i, k, waited, used, depth):
        while k >= 0:
            t = blocks[i][1][k][0]
            if re.match(r"v_(readlane|readfirstlane|cmp)", t) and scalars(t.split(",")[0]) & used:
                return t
            waited += int(t.split()[1]) + 1 if t.startswith("s_nop") else 1
            if waited >= 5:
                return None
            k -= 1
        if depth:
            for p in before[i]:
                found = back(p, len(blocks[p][1]) - 1, waited, used, depth - 1)
                if found:
                    return found
        return None

    bad, n = [], 0
    for i, (label, b) in enumerate(blocks):
        for k, (t, asm) in enumerate(b):
            if asm and t.startswith("buffer_load"):
                n += 1
                found = back(i, k - 1, 0, scalars(t), 6)
                if found:
                    bad.append(f"{label}: {found} -> {t}")
    return bad, n


def test_the_search_finds_both():
    text = "\n".join(["_Zk:", "s_and_saveexec_b64 s[4:5], vcc", "s_cbranch_execz .LBB0_2",
                      "global_load_dword v1, v[2:3], off", ".LBB0_2:", "v_mov_b32_e32 v7, v8",
                      "s_or_b64 exec, exec, s[4:5]", "v_readfirstlane_b32 s9, v1", "s_branch .LBB0_3",
                      ".LBB0_3:", ";ASMSTART", "s_mov_b32 m0, s2", "s_nop 0",
                      "buffer_load_dwordx4 v4, s[8:11], s3 offen lds", ";ASMEND", "s_endpgm",
                      ".Lfunc_end0:"])
    blocks = functions(text)["_Zk"]
    assert before_lanes_join(blocks) == [".LBB0_2: v_mov_b32_e32 v7, v8"]
    bad, n = loads_too_soon(blocks)
    assert n == 1 and len(bad) == 1
    late = functions(text.replace("s_nop 0", "s_nop 2"))["_Zk"]
    assert loads_too_soon(late) == ([], 1)


def test_no_kernel_has_either(tmp_path):
    hipcc = build.HIPCC if os.path.exists(build.HIPCC) else shutil.which("hipcc")
    if hipcc is None:
        pytest.skip("needs hipcc")
    flags = [f for f in build.FLAGS if f != "-shared"]
    jobs = [subprocess.Popen([hipcc, *flags, "-w", "-I", build.INCLUDE, "-S", "--offload-device-only",
                              os.path.join(build.CSRC, f), "-o", str(tmp_path / (f + ".s"))])
            for f in FILES]
    assert [j.wait(timeout=600) for j in jobs] == [0] * len(jobs)
    loads = 0
    for f in FILES:
        kernels = functions((tmp_path / (f + ".s")).read_text())
        assert len(kernels) > 3
        for name, blocks in kernels.items():
            assert before_lanes_join(blocks) == [], name
            bad, n = loads_too_soon(blocks)
            assert bad == [], name
            loads += n
    assert loads > 100
