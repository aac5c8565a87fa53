"""The machine code of the built library keeps the wait states that gfx9 does not enforce itself.

The compiler puts them between the instructions it schedules, but not into or
around inline assembly, where the direct loads to LDS are written.  Two rules
concern those loads:

* a load to LDS stands at least one wait state behind the scalar instruction
  that wrote M0;
* a memory instruction stands at least five wait states behind a vector
  instruction that wrote a scalar register it reads (v_readfirstlane and the
  like).

An instruction is one wait state, s_nop N is N + 1.
"""
import os
import re
import struct
import subprocess

import pytest

from mixture_experts_layer_03_amd import abi

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
LINE = re.compile(r"^\t(\S.*?)\s*// ([0-9A-F]{12}):")


def code_objects(data):
    """The gfx950 code objects of a library's offload bundles."""
    at = data.find(MAGIC)
    while at >= 0:
        n, p = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            if size and b"gfx950" in data[p + 24:p + 24 + length]:
                yield data[at + off:at + off + size]
            p += 24 + length
        at = data.find(MAGIC, at + 24)


def scalars(text):
    """Numbers of the scalar registers that an operand names."""
    out = set()
    for a, b, c in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(c)} if c else set(range(int(a), int(b) + 1))
    return out


class Instr:
    def __init__(self, text, at):
        self.at = at
        self.op, _, rest = text.partition(" ")
        args = rest.split(", ")
        self.waits = int(args[0], 0) + 1 if self.op == "s_nop" else 1
        self.memory = self.op.startswith(("buffer_", "global_", "flat_", "scratch_"))
        self.to_lds = self.memory and (" lds" in rest or "_lds_" in self.op)
        self.reads = scalars(rest) if self.memory else set()
        self.writes_m0 = self.op.startswith("s_") and args[0] == "m0"
        self.vector_writes = set()
        if self.op.startswith("v_"):
            self.vector_writes = scalars(args[0]) | (scalars(args[1]) if "_co_" in self.op else set())
        self.target = None
        if self.op == "s_branch" or self.op.startswith("s_cbranch"):
            jump = int(args[0].split()[0], 0)
            self.target = at + 4 + 4 * (jump - 65536 if jump >= 32768 else jump)
        self.falls = self.op not in ("s_branch", "s_endpgm", "s_setpc_b64", "s_trap")


def parse(listing):
    """[(kernel, [Instr])] of a disassembly."""
    out = []
    for line in listing.splitlines():
        head = re.match(r"(?:[0-9a-f]+ )?<(\S+)>:$", line)
        if head:
            out.append((head.group(1), []))
            continue
        m = LINE.match(line)
        if m:
            out[-1][1].append(Instr(m.group(1), int(m.group(2), 16)))
    return out


def violations(code):
    """(address, rule) of each memory instruction that stands too near."""
    place = {x.at: i for i, x in enumerate(code)}
    before = [[i - 1] if i and code[i - 1].falls else [] for i in range(len(code))]
    for i, x in enumerate(code):
        if x.target in place:
            before[place[x.target]].append(i)

    def near(i, left, hit):   # whether `hit` is fewer than `left` wait states before i
        for j in before[i]:
            if hit(code[j]):
                return True
            rest = left - code[j].waits
            if rest > 0 and near(j, rest, hit):
                return True
        return False

    for i, x in enumerate(code):
        if x.to_lds and near(i, 1, lambda y: y.writes_m0):
            yield x.at, "m0"
        if x.reads and near(i, 5, lambda y: y.vector_writes & x.reads):
            yield x.at, "sgpr"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    with open(abi.LIB_PATH, "rb") as f:
        data = f.read()
    path = str(tmp_path_factory.mktemp("code") / "object")
    out = []
    for obj in code_objects(data):
        with open(path, "wb") as f:
            f.write(obj)
        out += parse(subprocess.run([OBJDUMP, "-d", path], check=True, capture_output=True, text=True).stdout)
    return out


def test_the_rules_are_found_in_a_listing():
    def run(*lines):
        body = "".join("\t%s    // %012X: 00000000\n" % (t, 256 + 4 * i) for i, t in enumerate(lines))
        return [rule for _, rule in violations(parse("<k>:\n" + body)[0][1])]
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    assert run("s_mov_b32 m0, s1", load) == ["m0"]
    assert run("s_mov_b32 m0, s1", "s_nop 0", load) == []
    assert run("s_add_i32 m0, s1, s2", "v_mov_b32_e32 v1, v2", load) == []
    assert run("v_readfirstlane_b32 s6, v1", "s_nop 3", load) == ["sgpr"]
    assert run("v_readfirstlane_b32 s6, v1", "s_nop 4", load) == []
    assert run("v_readfirstlane_b32 s8, v1", load) == []
    assert run("v_cmp_lt_u32_e64 s[6:7], s1, v1", "s_mov_b32 m0, s1", "s_nop 0", load) == ["sgpr"]
    # over a branch back: the load is the first instruction of the loop
    assert run(load, "v_readlane_b32 s4, v1, 3", "s_cbranch_scc1 65533", "s_endpgm") == ["sgpr"]
    assert run(load, "v_readlane_b32 s4, v1, 3", "s_branch 0", "s_endpgm") == []


@pytest.mark.parametrize("rule", ["m0", "sgpr"])
def test_the_library_keeps_the_wait_states(kernels, rule):
    loads, bad = 0, {}
    for name, code in kernels:
        loads += sum(x.to_lds for x in code)
        for at, r in violations(code):
            if r == rule:
                bad.setdefault(name, []).append(hex(at))
    assert loads > 0
    assert not bad, {k: len(v) for k, v in bad.items()}
