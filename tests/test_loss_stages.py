"""The order of the vocabulary loss' LDS stages in the built library (no GPU).

The matrix kernels load a stage of LDS again behind the second barrier after
its reads: reads from before the previous barrier have to have come back by
then, whatever the compiler did with the instructions that use them.  The
machine code built for gfx950 is followed instruction by instruction: LDS
operations answer in order, so `s_waitcnt lgkmcnt(n)` leaves the n youngest
outstanding (scalar loads share the counter, which only makes n smaller for
LDS), and at every barrier none may be older than the barrier before."""
import os
import re
import shutil
import subprocess

import pytest

from collective_communication_primitives_amd import _lib

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
LINE = re.compile(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):[^<]*(?:<.*\+0x([0-9a-f]+)>)?")


def functions(listing):
    """name -> [(address, mnemonic, operands, branch target or None)]"""
    found, name, start = {}, None, 0
    for line in listing.splitlines():
        head = re.match(r"^([0-9a-f]+) <(.*)>:$", line)
        if head:
            name, start = head.group(2), int(head.group(1), 16)
            found[name] = []
        elif name is not None:
            m = LINE.match(line)
            if m:
                target = start + int(m.group(4), 16) if m.group(4) and "branch" in m.group(1) else None
                found[name].append((int(m.group(3), 16), m.group(1), m.group(2), target))
    return found


def stale_reads(code):
    """Addresses of the barriers at which an LDS operation from before the previous barrier may be outstanding.  State: the
    barriers passed since each outstanding operation was issued, oldest first; two ways that meet give the worse of both."""
    at = {address: i for i, (address, *_) in enumerate(code)}
    states, todo, bad = {0: ()}, [0], set()

    def reach(i, state):
        old = states.get(i)
        if old is None:
            new = state
        else:
            n = max(len(old), len(state))
            pad = lambda s: (-1,) * (n - len(s)) + s
            new = tuple(max(a, b) for a, b in zip(pad(old), pad(state)))
        if old != new:
            states[i] = new
            todo.append(i)

    while todo:
        i = todo.pop()
        state = states[i]
        address, op, operands, target = code[i]
        if op.startswith("ds_"):
            state = (state + (0,))[-64:]
        elif op == "s_waitcnt":
            m = re.search(r"lgkmcnt\((\d+)\)", operands)
            if m:
                state = state[max(0, len(state) - int(m.group(1))):]
        elif op == "s_barrier":
            if any(age >= 1 for age in state):
                bad.add(address)
            state = tuple(min(age + 1, 2) for age in state)
        if op == "s_endpgm":
            continue
        if target is not None:
            reach(at[target], state)
        if op != "s_branch" and i + 1 < len(code):
            reach(i + 1, state)
    return sorted(bad)


def program(text):
    return functions("0000000000000000 <f>:\n" + "".join(
        "\t%s // %012X: 0%s\n" % (op, 4 * i, " <f+0x%x>" % (4 * int(op.split()[1])) if "branch" in op else "") for i, op in enumerate(text)))["f"]


def test_the_check_itself():
    turn = ["s_barrier", "ds_read_b128 v[0:3], v4", "ds_read_b128 v[4:7], v4"]
    assert stale_reads(program(turn + ["s_waitcnt lgkmcnt(0)", "s_cbranch_scc0 0", "s_endpgm"])) == []
    # both reads of the turn before may be outstanding at the barrier, none of an earlier one
    assert stale_reads(program(["s_waitcnt vmcnt(2) lgkmcnt(2)"] + turn + ["s_cbranch_scc0 0", "s_endpgm"])) == []
    assert stale_reads(program(["s_waitcnt vmcnt(2) lgkmcnt(3)"] + turn + ["s_cbranch_scc0 0", "s_endpgm"])) == [4]
    assert stale_reads(program(turn + ["s_cbranch_scc0 0", "s_endpgm"])) == [0]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    where = tmp_path_factory.mktemp("code")
    shutil.copy(_lib.LIBRARY, where / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=where, check=True, capture_output=True)
    found = {}
    for name in sorted(os.listdir(where)):
        if "gfx950" in name:
            with open(where / name, "rb") as f:
                if b"k_loss_stats" not in f.read():
                    continue
            out = subprocess.run([OBJDUMP, "-d", name], cwd=where, check=True, capture_output=True, text=True).stdout
            found.update({k: v for k, v in functions(out).items() if "k_loss" in k and "Shape" in k})
    return found


def test_no_stage_is_loaded_over_outstanding_reads(kernels):
    tiled = {k: v for k, v in kernels.items() if any(op == "s_barrier" for _, op, *_ in v)}
    assert len(tiled) > 20 and any("k_loss_dweight" in k for k in tiled)  # the library's matrix kernels are all here
    bad = {k: ["%x" % a for a in at] for k, v in tiled.items() if (at := stale_reads(v))}
    assert bad == {}
