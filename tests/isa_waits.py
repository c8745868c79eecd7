"""Reads the gfx950 machine code of the built library (this repository's own build) and lists the memory
instructions that follow too closely on the instruction that wrote a scalar register they read.

The hardware does not wait there by itself: an instruction of the vector unit that writes a scalar register
(v_readfirstlane_b32, v_readlane_b32, a compare's mask) has to be five wait states before a vector-memory instruction
that reads it, and a scalar write of M0 one before a load to LDS (CDNA ISA, "Manually Inserted Wait States"). The
compiler keeps these distances between its own instructions, not into inline assembly.
"""
import re

SGPR_WAIT, M0_WAIT = 5, 1
_MEM = ("buffer_", "global_", "flat_", "scratch_")
# vector instructions with a second, scalar destination
_TWO = re.compile(r"^v_(add_co|addc_co|sub_co|subb_co|subrev_co|subbrev_co|mad_u64_u32|mad_i64_i32|div_scale)")


def instructions(text):
    """{symbol: [(address, mnemonic, [operands])]} from llvm-objdump output."""
    funcs, cur = {}, None
    for line in text.splitlines():
        h = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if h:
            cur = funcs.setdefault(h.group(1), [])
            continue
        m = re.match(r"^\s+(\S[^/]*?)\s*// ([0-9A-Fa-f]+):", line)
        if cur is None or not m:
            continue
        parts = m.group(1).split(None, 1)
        ops = [o.strip() for o in parts[1].split(",")] if len(parts) > 1 else []
        cur.append((int(m.group(2), 16), parts[0], ops))
    return funcs


def _scalars(text):
    """Scalar registers named anywhere in an operand."""
    out = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    out |= {int(a) for a in re.findall(r"\bs(\d+)\b", text)}
    return out


def _vector_writes(mn, ops):
    if not mn.startswith("v_") or not ops:
        return set()
    out = _scalars(ops[0]) if ops[0].startswith("s") else set()
    if _TWO.match(mn) and len(ops) > 1 and ops[1].startswith("s"):
        out |= _scalars(ops[1])
    return out


def _to_lds(mn, ops):
    return mn.startswith("global_load_lds") or (mn.startswith(_MEM) and bool(ops) and " lds" in " " + ops[-1])


def close_pairs(insts):
    """(address of the memory instruction, its mnemonic, the writer's mnemonic, wait states between them) of every
    pair that is too close on any path through the branches."""
    at = {a: i for i, (a, _, _) in enumerate(insts)}
    before = [[] for _ in insts]
    for i, (a, mn, ops) in enumerate(insts):
        if mn.startswith(("s_branch", "s_cbranch")):
            off = int(ops[0].split()[0])
            to = at.get(a + 4 + 4 * (off - 65536 if off >= 32768 else off))
            if to is not None:
                before[to].append(i)
        if i + 1 < len(insts) and not mn.startswith(("s_branch", "s_endpgm", "s_setpc")):
            before[i + 1].append(i)
    found = set()
    for i, (a, mn, ops) in enumerate(insts):
        if not mn.startswith(_MEM):
            continue
        reads, lds = _scalars(" ".join(ops)), _to_lds(mn, ops)
        todo = [(p, 0) for p in before[i]]
        seen = set()
        while todo:
            k, states = todo.pop()
            if (k, states) in seen or states >= SGPR_WAIT:
                continue
            seen.add((k, states))
            _, wmn, wops = insts[k]
            if _vector_writes(wmn, wops) & reads:
                found.add((a, mn, wmn, states))
            if lds and states < M0_WAIT and wmn.startswith("s_") and wops and wops[0] == "m0":
                found.add((a, mn, wmn, states))
            states += int(wops[0], 0) + 1 if wmn == "s_nop" else 1
            todo += [(p, states) for p in before[k]]
    return sorted(found)
