"""Reads the GPU code of the library that is built here: which barriers a wave may reach with LDS operations of its own
that it has not waited for. Other waves may read before such a write, or write before such a read."""
from __future__ import annotations

import os
import re
import subprocess

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def code_objects(lib, folder):
    """The gfx950 code objects inside the library, as files in `folder`."""
    link = os.path.join(folder, "lib.so")
    os.symlink(lib, link)
    subprocess.run([OBJDUMP, "--offloading", link], cwd=folder, check=True, capture_output=True)
    return sorted(os.path.join(folder, f) for f in os.listdir(folder) if f.endswith("gfx950"))


def functions(path):
    """(name, [(address, mnemonic, operands, branch target or None)]) of a code object."""
    text = subprocess.run([OBJDUMP, "-d", path], check=True, capture_output=True, text=True).stdout
    name, base, body = None, 0, []
    for line in text.splitlines():
        head = re.match(r"^([0-9a-f]+) <(.+)>:$", line)
        if head:
            if name is not None:
                yield name, body
            base, name, body = int(head.group(1), 16), head.group(2), []
            continue
        code, _, rest = line.partition("//")
        code = code.strip()
        if name is None or not code or not rest:
            continue
        op, _, operands = code.partition(" ")
        address = int(rest.strip().split(":")[0], 16)
        target = None
        if op.startswith(("s_branch", "s_cbranch")):
            at = re.search(r"<.*?(?:\+0x([0-9a-f]+))?>\s*$", rest)
            target = base + int(at.group(1) or "0", 16)
        body.append((address, op, operands, target))
    if name is not None:
        yield name, body


def _after(pending, op, operands):
    """Operations of the wave's LDS counter still on the way, oldest first, after one more instruction."""
    if op.startswith(("ds_bpermute", "ds_permute", "ds_swizzle")):
        return pending + ("lane",)  # counted, touches no memory
    if op.startswith("ds_"):
        return (pending + ("read" if op.startswith("ds_read") else "write",))[-64:]
    if op.startswith(("s_load", "s_buffer_load")):
        return pending + ("scalar",)
    if op == "s_waitcnt":
        n = re.search(r"lgkmcnt\((\d+)\)", operands)
        if n and int(n.group(1)) == 0:
            return ()
        if n and "scalar" not in pending:  # scalar loads return in any order
            return pending[-int(n.group(1)):] if len(pending) > int(n.group(1)) else pending
    return pending


def _either(a, b):
    """What may be on the way where two paths meet."""
    if a is None or a == b:
        return b
    if len(a) < len(b):
        a, b = b, a
    out, off = list(a), len(a) - len(b)
    for i, x in enumerate(b):
        if x != out[off + i]:
            out[off + i] = next(k for k in ("write", "read", "scalar", "lane") if k in (x, out[off + i]))
    return tuple(out)


def open_barriers(body):
    """(number of barriers, addresses of those that an unfinished LDS read or write may reach) of a function."""
    starts = {t for _, _, _, t in body if t is not None} | {body[0][0]}
    blocks, cut = {}, True
    for i, (address, op, operands, target) in enumerate(body):
        if cut or address in starts:
            at = address
            blocks[at] = [[], []]
            if not cut and i:
                blocks[before][1].append(at)
        blocks[at][0].append((address, op, operands))
        before, cut = at, False
        if target is not None:
            blocks[at][1].append(target)
        if op in ("s_endpgm", "s_branch", "s_setpc_b64"):
            cut = True
        elif target is not None and i + 1 < len(body):  # falls through to a block of its own
            starts.add(body[i + 1][0])
    entry, work, found = {body[0][0]: ()}, [body[0][0]], set()
    barriers = sum(op == "s_barrier" for _, op, _, _ in body)
    for _ in range(1000 * len(blocks)):
        if not work:
            break
        at = work.pop()
        pending = entry[at]
        for address, op, operands in blocks[at][0]:
            if op == "s_barrier" and ("read" in pending or "write" in pending):
                found.add(address)
            pending = _after(pending, op, operands)
        for t in blocks[at][1]:
            met = _either(entry.get(t), pending)
            if t in blocks and met != entry.get(t):
                entry[t] = met
                work.append(t)
    assert not work, "the paths of a function have not settled"
    return barriers, sorted(found)
