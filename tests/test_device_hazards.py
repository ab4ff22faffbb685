"""Wait states that the hardware asks of the program, checked in the built library's own code.

The compiler keeps them for the instructions that it emits itself, but it does not look into
inline assembly, through which the kernels issue their direct-to-LDS loads.  On gfx9

* an instruction that writes M0 and a load into LDS, which takes its LDS address from M0, need
  one wait state between them;
* a vector instruction that writes a scalar register and a memory instruction that reads it (as
  its base address) need five.

An instruction between the two is one wait state, s_nop n is n + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

LLVM = "/opt/rocm/llvm/bin"
OBJDUMP = next((p for p in (os.path.join(LLVM, "llvm-objdump"), shutil.which("llvm-objdump")) if p and os.path.exists(p)), None)


class Instruction:
    def __init__(self, addr, text, target):
        self.addr, self.target = addr, target
        self.name, _, rest = text.partition(" ")
        self.args = [a.strip() for a in rest.split(",")] if rest.strip() else []
        self.states = int(self.args[0], 0) + 1 if self.name == "s_nop" else 1

    def into_lds(self):
        return "_load_lds_" in self.name or (self.name.startswith("buffer_load") and any(a.split()[-1:] == ["lds"] for a in self.args))

    def memory(self):
        return self.name.startswith(("global_", "buffer_", "flat_", "scratch_"))

    def ends(self):
        return self.name in ("s_branch", "s_endpgm", "s_setpc_b64")


def scalars(arg):
    """The scalar registers that an operand names."""
    m = re.match(r"s\[(\d+):(\d+)\]", arg)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)\b", arg)
    return {int(m[1])} if m else set()


def parse(listing):
    """llvm-objdump -d --no-show-raw-insn of a code object -> functions, each a list of instructions."""
    out = []
    base = 0
    for line in listing.splitlines():
        m = re.match(r"([0-9a-f]{16}) <(.+)>:$", line)
        if m:
            base = int(m[1], 16)
            out.append((m[2], []))
            continue
        m = re.match(r"\t(\S.*?)\s*// ([0-9A-F]+):?(.*)$", line)
        if m and out:
            t = re.search(r"<[^>]*?(?:\+0x([0-9a-f]+))?>\s*$", m[3])
            target = base + int(t[1] or "0", 16) if t else None
            out[-1][1].append(Instruction(int(m[2], 16), m[1].strip(), target))
    return out


def violations(code):
    """(what, first, second) of every pair of instructions that is too close on some path."""
    at = {x.addr: i for i, x in enumerate(code)}
    jumps = {}
    for i, x in enumerate(code):
        if x.target in at and x.name.startswith(("s_branch", "s_cbranch")):
            jumps.setdefault(at[x.target], []).append(i)
    before = lambda i: ([i - 1] if i and not code[i - 1].ends() else []) + jumps.get(i, [])
    found = []
    for i, x in enumerate(code):
        if not x.memory():
            continue
        reads = set().union(*(scalars(a) for a in x.args)) if x.args else set()
        todo, seen = [(p, 0) for p in before(i)], {}
        while todo:
            p, gap = todo.pop()
            if gap >= 5 or seen.get(p, 9) <= gap:
                continue
            seen[p] = gap
            y = code[p]
            if gap < 1 and x.into_lds() and y.args[:1] == ["m0"]:
                found.append(("M0", y, x))
            if y.name.startswith("v_") and y.args and scalars(y.args[0]) & reads:
                found.append(("scalar base", y, x))
            todo += [(q, gap + y.states) for q in before(p)]
    return found


@pytest.fixture(scope="module")
def code(lib, tmp_path_factory):
    if OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    import precision_moe_gemm_amd as pmg
    d = tmp_path_factory.mktemp("code")
    so = shutil.copy(pmg.library_path(), d / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(so)], check=True, capture_output=True)
    functions = []
    for f in sorted(os.listdir(d)):
        if "gfx950" in f:
            r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(d / f)], check=True, capture_output=True, text=True)
            functions += parse(r.stdout)
    return functions


def test_the_listing_is_understood(code):
    loads = sum(x.into_lds() for _, c in code for x in c)
    assert len(code) > 20 and loads > 100
    for name, c in code:
        at = {x.addr for x in c}
        assert all(x.target in at for x in c if x.name.startswith(("s_branch", "s_cbranch"))), name


def test_the_check_finds_what_it_looks_for():
    def fn(*lines):
        body = "".join(f"\t{t} // {4 * i:012X}:{j}\n" for i, (t, j) in enumerate((l, "") if isinstance(l, str) else l for l in lines))
        return parse("0000000000000000 <f>:\n" + body)[0][1]
    load = "global_load_lds_dwordx4 v1, s[4:5]"
    assert [w for w, *_ in violations(fn("s_mov_b32 m0, s3", load))] == ["M0"]
    assert not violations(fn("s_mov_b32 m0, s3", "s_nop 0", load))
    assert [w for w, *_ in violations(fn("v_readfirstlane_b32 s5, v2", "s_mov_b32 m0, s3", "s_nop 0", load))] == ["scalar base"]
    assert not violations(fn("v_readfirstlane_b32 s5, v2", "s_mov_b32 m0, s3", "s_nop 3", load))
    # through a branch: the write is far away in the listing and next to the load on the path
    far = fn("s_nop 0", load, "s_endpgm", "s_mov_b32 m0, s3", ("s_branch 65532", " <f+0x4>"))
    assert not violations(far)   # the branch itself is a wait state
    assert violations(fn("s_nop 0", load, "s_endpgm", "v_cmp_eq_u32_e64 s[4:5], v0, v1", ("s_branch 65532", " <f+0x4>")))


def _bad(code, kind):
    return [f"{name}: {a.name} {', '.join(a.args)} -> {b.name} {', '.join(b.args)} at {b.addr:#x}"
            for name, c in code for what, a, b in violations(c) if what == kind]


def test_loads_into_lds_wait_for_m0(code):
    bad = _bad(code, "M0")
    assert not bad, f"{len(bad)} pairs too close, e.g.\n" + "\n".join(bad[:10])


def test_memory_instructions_wait_for_scalars_of_vector_instructions(code):
    bad = _bad(code, "scalar base")
    assert not bad, f"{len(bad)} pairs too close, e.g.\n" + "\n".join(bad[:10])
