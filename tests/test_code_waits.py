"""Wait states around hand-written loads, read off the library's own machine code (CPU).

The compiler puts the wait states that an instruction needs between the instructions that it
issues itself; inside an asm statement it does not look.  A vector memory instruction reads an
SGPR that a vector instruction wrote no sooner than five wait states later, and a load into LDS
reads M0 no sooner than one after it was written.  Here every path of every kernel
with loads into LDS is followed, through its branches, and each of its vector memory instructions
is held against both."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_amd", "libuep.so")
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
VALU_TO_VMEM, M0_TO_LDS = 5, 1

_LINE = re.compile(r"^\t(\S+) *(.*?) *// ([0-9A-F]+):(?:.*<(\S+?)(?:\+0x([0-9a-f]+))?>)?")
_HEAD = re.compile(r"^([0-9a-f]+) <(\S+)>:$")
_SGPR = re.compile(r"(?<![\w.])s(?:(\d+)|\[(\d+):(\d+)\])(?!\w)")


def sgprs(text):
    """Numbers of the SGPRs that an operand names (vcc as 106 and 107)."""
    out = {106, 107} if "vcc" in text else set()
    for one, a, b in _SGPR.findall(text):
        out.update([int(one)] if one else range(int(a), int(b) + 1))
    return out


def effects(op, args):
    """What an instruction's waits depend on: SGPRs that a vector instruction writes, whether
    M0 is written, SGPRs that a vector memory instruction reads, whether it reads M0, and the
    wait states that it makes."""
    part = [a.strip() for a in args.split(",")]
    wrote, needs = set(), set()
    if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
        wrote = sgprs(part[0])
    elif op.startswith("v_") and ("_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64"))):
        wrote = sgprs(part[1])
    elif op.startswith(("buffer_", "global_", "scratch_", "flat_", "tbuffer_")):
        needs = sgprs(args)
    m0 = part[0] == "m0"
    to_lds = op.startswith(("buffer_load", "global_load")) and " lds" in " " + args
    return wrote, m0, needs, to_lds, int(args) + 1 if op == "s_nop" else 1


def kernels(text):
    """(name, [(address, op, args, branch target or None)]) of a disassembly."""
    name, base, body = None, 0, []
    for line in text.splitlines():
        h = _HEAD.match(line)
        if h:
            if name:
                yield name, body
            base, name, body = int(h[1], 16), h[2], []
            continue
        m = _LINE.match(line)
        if m and name:
            to = None
            if m[1].startswith(("s_branch", "s_cbranch")):
                assert m[4] == name, line
                to = base + int(m[5] or "0", 16)
            body.append((int(m[3], 16), m[1], m[2], to))
    if name:
        yield name, body


def too_soon(body):
    """The instructions that come sooner than they may behind what they read.  `into` holds, for
    every place that a branch reaches, the fewest wait states since each write, over all ways there."""
    rows = [(at, op, args, to, *effects(op, args)) for at, op, args, to in body]
    into, found = {r[3]: None for r in rows if r[3] is not None}, {}

    def merge(at, state):
        old = into[at]
        new = dict(state) if old is None else {
            k: min(old.get(k, 99), state.get(k, 99)) for k in old.keys() | state.keys()}
        if new != old:
            into[at] = new
            return True
        return False

    again = True
    while again:
        again, state = False, {}
        for at, op, args, to, wrote, m0, needs, to_lds, waits in rows:
            if at in into:
                if state is not None:
                    merge(at, state)
                state = dict(into[at]) if into[at] is not None else state
            if state is None:
                continue                                  # only a branch from below comes here
            for r in needs:
                if state.get(r, 99) < VALU_TO_VMEM:
                    found[at] = f"{op} {args}: s{r} after {state[r]} wait states"
            if to_lds and state.get("m0", 99) < M0_TO_LDS:
                found[at] = f"{op} {args}: m0 after {state['m0']} wait states"
            state = {k: v + waits for k, v in state.items() if v + waits < VALU_TO_VMEM}
            for r in wrote:
                state[r] = 0
            if m0:
                state["m0"] = 0
            if to is not None and merge(to, state):
                again = again or to <= at
            if op in ("s_branch", "s_endpgm", "s_setpc_b64"):
                state = None
    return found


def test_the_reader_itself():
    """By hand: a read right behind the write, one behind enough waits, one over a loop's back edge."""
    text = "\n".join([
        "0000000000000100 <k>:",
        "\tv_readlane_b32 s22, v253, 1 // 000000000100: 0",
        "\ts_mov_b32 m0, s4 // 000000000108: 0",
        "\ts_nop 0 // 00000000010C: 0",
        "\tbuffer_load_dword v1, s[20:23], s6 offen lds // 000000000110: 0",
        "\ts_nop 4 // 000000000118: 0",
        "\tbuffer_load_dword v1, s[20:23], s6 offen lds // 00000000011C: 0",
        "\tv_cmp_lt_i32_e64 s[6:7], v1, v2 // 000000000124: 0",
        "\ts_cbranch_scc1 65523 // 00000000012C: 0 <k+0x1c>",
        "\ts_mov_b32 m0, s5 // 000000000130: 0",
        "\tbuffer_load_dword v1, s[8:11], 0 offen lds // 000000000134: 0",
        "\ts_endpgm // 00000000013C: 0"])
    (name, body), = kernels(text)
    assert name == "k" and len(body) == 11
    found = too_soon(body)
    assert sorted(found) == [0x110, 0x11C, 0x134]
    assert "s22 after 2" in found[0x110] and "s6 after 1" in found[0x11C] and "m0 after 0" in found[0x134]


def test_loads_into_lds_wait_for_their_scalars(tmp_path):
    if not os.path.exists(LIB):
        pytest.fail("libuep.so is not built (run __graft_entry__.build())")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    shutil.copy(LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    seen, bad = 0, []
    for f in sorted(tmp_path.glob("*gfx950*")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], check=True,
                              capture_output=True, text=True).stdout
        if " lds " not in text:
            continue
        for name, body in kernels(text):
            if any(" lds" in args for _, op, args, _ in body if op.startswith("buffer_load")):
                seen += 1
                bad += [f"{name}+{at:x}: {what}" for at, what in too_soon(body).items()]
    assert seen >= 20                                     # the expert product's kernels
    assert not bad, f"{len(bad)}: " + "; ".join(bad[:5])
