"""The machine code of the built kernels: wait states that gfx9 does not insert by
itself.  Direct global -> LDS loads are issued from inline assembly, into which the
compiler does not look, so what it would keep apart elsewhere is checked here, on the
disassembly of the objects of the last build:

  - a scalar write of m0 and an LDS load, which takes its LDS address from m0: one
    instruction (or s_nop) between them;
  - a vector instruction that writes an SGPR (v_readlane, v_readfirstlane, a compare)
    and a vector memory instruction that reads it: five between them.

Every path to a load is followed, backwards through branches and labels."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJS = os.path.join(ROOT, "newton_schulz_gram_amd", "_build")
LLVM = "/opt/rocm/llvm/bin"
TARGET = "hipv4-amdgcn-amd-amdhsa--gfx950"
NEEDS = {"m0": 1, "sgpr": 5}

LINE = re.compile(r"^\s+(\S+)\s*(.*?)\s*//\s*([0-9A-F]+):")
BRANCH = re.compile(r"^s_(c?branch\w*|call_b64|setpc_b64|endpgm\w*)$")


def parse(text):
    """Functions of a disassembly: lists of (mnemonic, operands, address)."""
    functions, now = [], None
    for line in text.splitlines():
        if line.endswith(">:"):
            now = []
            functions.append(now)
            continue
        m = LINE.match(line)
        if m and now is not None:
            now.append((m.group(1), m.group(2), int(m.group(3), 16)))
    return functions


def registers(operand):
    """The SGPR numbers of s7 or s[4:5]."""
    m = re.fullmatch(r"s(\d+)", operand) or re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    lo = int(m.group(1))
    return set(range(lo, int(m.group(m.lastindex)) + 1))


def operands(text):
    return [o.strip() for o in re.split(r",(?![^\[]*\])", text) if o.strip()]


def predecessors(code):
    """Indices of the instructions that may run right before each one."""
    at = {a: i for i, (_, _, a) in enumerate(code)}
    before = [[] for _ in code]
    for i, (name, args, addr) in enumerate(code):
        b = BRANCH.match(name)
        if b and b.group(1).startswith(("branch", "cbranch")):
            offset = int(args.split()[0], 0)
            to = at.get(addr + 4 + 4 * (offset - 65536 if offset >= 32768 else offset))
            if to is not None:
                before[to].append(i)
        if i + 1 < len(code) and not (b and not b.group(1).startswith("cbranch")):
            before[i + 1].append(i)
    return before


def hazards(code):
    """(address, what) of every load that follows a write too closely."""
    before, found = predecessors(code), []

    def written_within(i, states, writes, over=lambda name, args: False):
        """Whether `writes` holds for an instruction less than `states` wait states
        before i, on a path on which `over` holds for none behind it."""
        todo, seen = [(p, 0) for p in before[i]], {}
        while todo:
            j, passed = todo.pop()
            if passed >= states or seen.get(j, states) <= passed:
                continue
            seen[j] = passed
            name, args, _ = code[j]
            if writes(name, args):
                return True
            if over(name, args):
                continue
            step = int(args, 0) + 1 if name == "s_nop" else 1
            todo += [(p, passed + step) for p in before[j]]
        return False

    for i, (name, args, addr) in enumerate(code):
        if not name.startswith(("global_", "buffer_", "flat_", "scratch_")):
            continue
        ops = operands(args)
        if "_lds_" in name or "lds" in args.split():
            if written_within(i, NEEDS["m0"], lambda n, a: n.startswith("s_") and operands(a)[:1] == ["m0"]):
                found.append((addr, "m0"))
        for r in set().union(*(registers(o.split()[0]) for o in ops)) if ops else ():
            # (a scalar instruction that writes the register again has waited for the vector one)
            if written_within(i, NEEDS["sgpr"],
                              lambda n, a: n.startswith("v_") and any(r in registers(o) for o in operands(a)[:2 if "_co_" in n else 1]),
                              lambda n, a: n.startswith("s_") and any(r in registers(o) for o in operands(a)[:1])):
                found.append((addr, "sgpr"))
                break
    return found


def listing(lines):
    """A function's disassembly with four-byte instructions."""
    return "0 <f>:\n" + "\n".join(f"\t{l}  // {4 * i:012X}: 00000000" for i, l in enumerate(lines))


@pytest.mark.parametrize("lines,what", [
    (["s_mov_b32 m0, s7", "global_load_lds_dwordx4 v5, s[0:1]"], ["m0"]),
    (["s_mov_b32 m0, s7", "s_nop 0", "global_load_lds_dwordx4 v5, s[0:1]"], []),
    (["s_mov_b32 m0, s7", "global_load_dwordx4 v[4:7], v5, s[0:1]"], []),
    (["s_nop 0", "global_load_lds_dword v5, s[2:3]", "v_readlane_b32 s3, v9, 0", "s_cbranch_scc1 65533", "s_endpgm"], ["sgpr"]),
    (["v_readlane_b32 s3, v9, 0", "s_endpgm", "global_load_lds_dword v5, s[2:3]"], []),
    (["v_readlane_b32 s1, v9, 3", "s_mov_b32 m0, s7", "s_nop 0", "global_load_lds_dwordx4 v5, s[0:1]"], ["sgpr"]),
    (["v_readlane_b32 s1, v9, 3", "s_mov_b32 m0, s7", "s_nop 3", "global_load_lds_dwordx4 v5, s[0:1]"], []),
    (["v_readlane_b32 s1, v9, 3", "s_addc_u32 s1, s5, s1", "global_load_dword v5, v4, s[0:1]"], []),
    (["v_readlane_b32 s2, v9, 3", "global_load_dword v5, v4, s[0:1]"], []),
    (["v_readfirstlane_b32 s0, v9", "s_nop 3", "global_store_dword v5, v4, s[0:1]"], ["sgpr"]),
    (["v_readfirstlane_b32 s0, v9", "s_nop 4", "global_store_dword v5, v4, s[0:1]"], []),
])
def test_the_check_itself(lines, what):
    code, = parse(listing(lines))
    assert [w for _, w in hazards(code)] == what


def disassembly(source, tmp_path):
    """The functions of a source's built device code."""
    obj = os.path.join(OBJS, source + ".o")
    tools = [os.path.join(LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump")]
    if not (os.path.exists(obj) and all(map(os.path.exists, tools))):
        pytest.skip("needs the objects of a build and the ROCm LLVM tools")
    fat, device = str(tmp_path / "fat"), str(tmp_path / "device")
    subprocess.run([tools[0], "--dump-section", f".hip_fatbin={fat}", obj, os.devnull], check=True)
    subprocess.run([tools[1], "--unbundle", "--type=o", f"--targets={TARGET}", f"--input={fat}", f"--output={device}"], check=True)
    text = subprocess.run([tools[2], "-d", device], check=True, stdout=subprocess.PIPE, text=True).stdout
    functions = parse(text)
    assert sum(len(f) for f in functions) > 100
    return functions


@pytest.mark.parametrize("source", ["nsg_kernels.hip", "nsg_select.hip", "nsg_muon.hip", "nsg_expert.hip", "nsg_fp8.hip",
                                    "nsg_fp8_gemm.hip"])
def test_wait_states(source, tmp_path):
    functions = disassembly(source, tmp_path)
    found = [(f"{a:x}", w) for f in functions for a, w in hazards(f)]
    assert not found, (len(found), found[:10])


@pytest.mark.parametrize("source", ["nsg_expert.hip", "nsg_fp8.hip", "nsg_fp8_gemm.hip"])
def test_no_scratch_memory(source, tmp_path):
    """The expert layer's kernels keep what they hold in registers and LDS."""
    names = {name for f in disassembly(source, tmp_path) for name, _, _ in f}
    assert not [n for n in names if n.startswith("scratch_")]
