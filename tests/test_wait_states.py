"""The built library's machine code keeps the distance the hardware asks for
between a vector instruction that writes a scalar register and a memory
instruction that reads it: 5 wait states, which nothing but the code provides.
The compiler keeps it for its own memory instructions; loads written as inline
assembly have to bring it along."""
import os
import re
import subprocess

import pytest

from combine_moe_layout_05_amd._paths import LIB_PATH

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
NEEDED = 5
LINE = re.compile(r"^\s+(\S+)(.*?)\s*//\s*([0-9A-F]+):[^<]*(?:<[^>]*\+0x([0-9a-f]+)>)?")
SYMBOL = re.compile(r"^([0-9a-f]+) <(.+)>:")
SCALAR = re.compile(r"\b(?:s(\d+)\b|s\[(\d+):(\d+)\]|(vcc)\b)")
MEMORY = ("global_", "buffer_", "flat_", "scratch_")


def _registers(text):
    found = set()
    for one, lo, hi, vcc in SCALAR.findall(text):
        if vcc:
            found.add("vcc")
        elif one:
            found.add(int(one))
        else:
            found.update(range(int(lo), int(hi) + 1))
    return found


def _functions(text):
    """Name -> [(address, mnemonic, operands, branch target)]."""
    out, code, start = {}, None, 0
    for line in text.splitlines():
        m = SYMBOL.match(line)
        if m:
            start, code = int(m[1], 16), out.setdefault(m[2], [])
            continue
        m = LINE.match(line)
        if m and code is not None:
            target = start + int(m[4], 16) if m[4] and "branch" in m[1] else None
            code.append((int(m[3], 16), m[1], m[2], target))
    return out


def _violations(code):
    """Memory instructions too close behind a vector write of a scalar
    register they read, along every path that leads to them."""
    index = {ins[0]: n for n, ins in enumerate(code)}
    jumps = {}
    for n, ins in enumerate(code):
        if ins[3] in index:
            jumps.setdefault(index[ins[3]], []).append(n)

    def close(n, regs, states, seen):
        """Whether a path to instruction n, `states` wait states ahead of the
        load, holds such a write."""
        before = list(jumps.get(n, []))
        if n > 0 and code[n - 1][1] not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            before.append(n - 1)
        for p in before:
            _, op, args, _ = code[p]
            if states >= NEEDED or (p, states) in seen:
                continue
            seen.add((p, states))
            if op.startswith("v_"):
                # Destinations: the first operand, with a carry the second.
                wide = any(k in op for k in ("_co_", "div_scale", "mad_u64", "mad_i64"))
                dests = _registers(",".join(args.split(",")[:2 if wide else 1]))
                if dests & regs:
                    return True
            passed = int(args, 0) + 1 if op == "s_nop" else 1
            if close(p, regs, states + passed, seen):
                return True
        return False

    bad = []
    for n, (at, op, args, _) in enumerate(code):
        if op.startswith(MEMORY):
            regs = _registers(args)
            if regs and close(n, regs, 0, set()):
                bad.append((hex(at), op + args))
    return bad


def test_the_check_sees_a_violation():
    """On two lines as the disassembler prints them, one state short, then not."""
    text = ("0000000000001000 <k>:\n"
            "\tv_readfirstlane_b32 s8, v1    // 000000001000: 7E100501\n"
            "\ts_nop {}                      // 000000001004: BF800003\n"
            "\tglobal_load_dword v2, v0, s[8:9] // 000000001008: DC508000 02080000\n")
    assert _violations(_functions(text.format(3))["k"])
    assert not _violations(_functions(text.format(4))["k"])


def test_the_check_follows_jumps_and_carries():
    text = ("0000000000001000 <k>:\n"
            "\tv_mad_u64_u32 v[2:3], s[8:9], v4, v5, 0 // 000000001000: D1E80802 02020904\n"
            "\ts_cbranch_scc1 2                // 000000001008: BF850002 <k+0x14>\n"
            "\ts_nop 7                         // 00000000100C: BF800007\n"
            "\ts_endpgm                        // 000000001010: BF810000\n"
            "\tglobal_load_dword v2, v0, s[{}] // 000000001014: DC508000 02080000\n")
    assert _violations(_functions(text.format("8:9"))["k"])
    assert not _violations(_functions(text.format("6:7"))["k"])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not available")
def test_memory_instructions_wait_for_scalar_registers(tmp_path):
    lib = tmp_path / "lib.so"
    lib.symlink_to(LIB_PATH)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True,
                   cwd=tmp_path)
    objects = sorted(p for p in tmp_path.iterdir() if "gfx950" in p.name)
    assert objects
    loads, bad = 0, {}
    for obj in objects:
        text = subprocess.run([OBJDUMP, "-d", str(obj)], check=True, capture_output=True,
                              text=True).stdout
        for name, code in _functions(text).items():
            loads += sum(ins[1].startswith("global_load_lds") for ins in code)
            found = _violations(code)
            if found:
                bad[name] = found
    assert loads > 0
    assert not bad, {name: (len(v), v[:3]) for name, v in bad.items()}
