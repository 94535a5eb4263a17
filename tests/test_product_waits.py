"""The built code of the dense product: its matrix instructions stand in inline assembly,
for whose operands the compiler inserts no wait states. Every path from the last of
them to a read of their sums has to hold the waits, and no vector instruction may
write an operand within two wait states before one."""
import os
import re
import struct
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
RESULT_WAITS = 18  # wait states (the longest instruction's; these are among the shortest)
OPERAND_WAITS = 2
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(lib):
    """The gfx950 code objects of a library's bundles."""
    data = open(lib, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        p = at + len(MAGIC)
        (n,) = struct.unpack_from("<Q", data, p)
        p += 8
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            p += 24
            if data[p:p + length].endswith(b"gfx950") and size:
                yield data[at + off:at + off + size]
            p += length
        at = data.find(MAGIC, at + 1)


def listing(path):
    """{kernel: [(address, mnemonic, operands)]}"""
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], check=True,
                          capture_output=True, text=True).stdout
    out, cur = {}, None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            cur = out.setdefault(m.group(1), [])
            continue
        m = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if m and cur is not None:
            ops = m.group(2)
            if m.group(1).startswith(("s_branch", "s_cbranch")):
                ops = re.search(r"\+0x([0-9a-f]+)>", m.group(4)).group(1)
            cur.append((int(m.group(3), 16), m.group(1), ops))
    return out


def registers(ops):
    out = set()
    for f, a, b, g, c in re.findall(r"\b([av])\[(\d+):(\d+)\]|\b([av])(\d+)\b", ops):
        if f:
            out |= {(f, i) for i in range(int(a), int(b) + 1)}
        else:
            out.add((g, int(c)))
    return out


def operands(ops):
    return [registers(o) for o in re.split(r",(?![^\[]*\])", ops)]


def successors(code):
    """Indices that may run after each instruction."""
    index = {a - code[0][0]: i for i, (a, _, _) in enumerate(code)}
    out = []
    for i, (_, op, ops) in enumerate(code):
        if op == "s_endpgm":
            out.append([])
        elif op == "s_branch":
            out.append([index[int(ops, 16)]])
        elif op.startswith("s_cbranch"):
            out.append([i + 1, index[int(ops, 16)]])
        else:
            out.append([i + 1] if i + 1 < len(code) else [])
    return out


def states(op, ops):
    return int(ops) + 1 if op == "s_nop" else 1


def faults(code):
    """What reads or overwrites a sum too early, and operands written too late."""
    nxt, found = successors(code), []
    before = [[] for _ in code]
    for i, js in enumerate(nxt):
        for j in js:
            before[j].append(i)
    for i, (_, op, ops) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        sides = operands(ops)
        result, sources = sides[0], sides[1] | sides[2] | sides[3]
        todo, seen = [(j, 0) for j in nxt[i]], {}
        while todo:
            j, n = todo.pop()
            if n >= RESULT_WAITS or seen.get(j, RESULT_WAITS) <= n:
                continue
            seen[j] = n
            _, o, s = code[j]
            if o.startswith("v_mfma"):  # the same sum again is the hardware's to order
                other = operands(s)
                if result & (other[1] | other[2]) or (result & other[0] and result != other[0]):
                    found.append((code[i], code[j]))
            elif registers(s) & result:
                found.append((code[i], code[j]))
            todo += [(k, n + states(o, s)) for k in nxt[j]]
        todo = [(j, 0) for j in before[i]]
        while todo:
            j, n = todo.pop()
            if n >= OPERAND_WAITS:
                continue
            _, o, s = code[j]
            if o.startswith("v_") and not o.startswith("v_mfma") and operands(s)[0] & sources:
                found.append((code[j], code[i]))
            todo += [(k, n + states(o, s)) for k in before[j]]
    return found


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    from combine_moe_layout_03_amd import build

    if not os.path.exists(build.LIB) or not os.path.exists(OBJDUMP):
        pytest.skip("no built library, or no disassembler")
    out = {}
    for i, obj in enumerate(code_objects(build.LIB)):
        if b"product_kernel" in obj:
            path = tmp_path_factory.mktemp("code") / f"{i}.o"
            path.write_bytes(obj)
            out.update({k: c for k, c in listing(str(path)).items() if "product_kernel" in k})
    return out


def test_waits(kernels):
    assert len(kernels) >= 20
    for name, code in kernels.items():
        assert sum(op.startswith("v_mfma") for _, op, _ in code) >= 32
        assert not faults(code), (name, faults(code)[:3])


def test_the_check_sees_a_missing_wait():
    """Made listings: a sum stored at once, one behind the waits, an operand just moved."""
    mfma = "v_mfma_f32_16x16x32_bf16", "a[0:3], v[4:7], v[8:11], a[0:3]"
    end = "s_endpgm", ""
    store = "ds_write_b128", "v0, a[0:3]"

    def made(*ins):
        return [(4 * i, op, ops) for i, (op, ops) in enumerate(ins)]

    assert faults(made(mfma, store, end))
    assert faults(made(mfma, ("v_accvgpr_read_b32", "v1, a2"), ("s_nop", "15"), end))
    assert not faults(made(mfma, ("s_nop", "15"), ("s_nop", "15"), store, end))
    assert faults(made(("v_mov_b32_e32", "v5, v1"), mfma, end))
    assert faults(made(("v_mov_b32_e32", "v5, v1"), ("s_nop", "0"), mfma, end))
    assert not faults(made(("v_mov_b32_e32", "v5, v1"), ("s_nop", "1"), mfma, end))
    # through a branch: the sum's read stands ahead of the product in the listing
    assert faults(made(("s_branch", "8"), store, mfma, ("s_cbranch_scc1", "4"), end))
    assert not faults(made(mfma, mfma, end))
