"""Waits behind matrix instructions in the built library, without a GPU.

A matrix instruction's result must not be read, nor its registers written by another vector instruction, before it is done: the
hardware does not wait by itself, the compiler puts instructions or s_nop in between.  It has left them out where a
branch skips a block (before_branch in csrc/mfma_util.h).  Here every path behind every matrix instruction is followed through the
library's own code, the waits on it counted."""

import os
import re
import shutil
import subprocess

import pytest

import kernelized_psd_feature_amd as K

LLVM = "/opt/rocm/llvm/bin/llvm-objdump"
# slots between the instruction and a reader, by its passes (4, 8, and 8 of the fp32 form); each other instruction is one
WAITS = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x16_bf16": 8, "v_mfma_f32_32x32x16_bf16": 12, "v_mfma_f32_16x16x4_f32": 10}
TAKEN = 4                                            # a taken branch fetches anew: four slots at least


def _registers(text):
    out = set()
    for kind, lo, hi, kind1, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        out.update((kind, i) for i in range(int(lo), int(hi) + 1)) if kind else out.add((kind1, int(one)))
    return out


def _decode(text):
    """(operation, registers written, registers read) of one instruction; loads' results arrive late, and count as neither."""
    op, _, rest = text.partition(" ")
    ops = [x.strip() for x in re.split(r",(?![^\[]*\])", rest)]
    if not op.startswith("v_"):
        if op.startswith("s_"):
            return op, set(), set()
        stores = any(x in op for x in ("store", "write", "atomic", "add"))
        return op, set(), _registers(rest) if stores else _registers(",".join(ops[1:]))
    if op.startswith("v_cmp"):
        return op, set(), _registers(rest)
    wrote, read = _registers(ops[0]), _registers(",".join(ops[1:]))
    if "swap" in op:
        return op, wrote | _registers(ops[1]), read | wrote
    if op.startswith(("v_fmac", "v_mac", "v_dot2c", "v_writelane")) or "dpp" in op or "row_" in rest:
        read = read | wrote
    return op, wrote, read


def missing_waits(code):
    """Of [(address, instruction, branch target or None)]: [(address, slots, instruction, its first reader)] of those whose
    reader is early."""
    at = {a: i for i, (a, _, _) in enumerate(code)}
    decoded = [_decode(t) for _, t, _ in code]
    out = []
    for i, (op, result, _) in enumerate(decoded):
        if not op.startswith("v_mfma"):
            continue
        need, todo, seen = WAITS[op], [(i + 1, 0, frozenset(result))], {}
        while todo:
            j, slots, live = todo.pop()
            if j >= len(code) or slots >= need or not live or seen.get((j, live), need) <= slots:
                continue
            seen[j, live] = slots
            other, wrote, read = decoded[j]
            text, target = code[j][1:]
            if other.startswith("v_mfma"):           # an addend may follow at once: the matrix unit holds it back until it is done
                ops = [x.strip() for x in re.split(r",(?![^\[]*\])", text.partition(" ")[2])]
                if live & (_registers(ops[1]) | _registers(ops[2])):
                    out.append((hex(code[i][0]), slots, code[i][1], text))
                    continue
                live = live - wrote - _registers(ops[3])
            elif live & (wrote | read):
                out.append((hex(code[i][0]), slots, code[i][1], text))
                continue
            if other == "s_endpgm":
                continue
            nop = re.match(r"s_nop (\w+)", text)
            if target is not None:
                todo.append((at[target], slots + TAKEN, live))
            if other != "s_branch":
                todo.append((j + 1, slots + (int(nop.group(1), 0) + 1 if nop else 1), live))
    return out


def _functions(listing):
    """{function: its code} of a disassembly."""
    out, code = {}, None
    for line in listing.split("\n"):
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            code = out.setdefault(m.group(1), [])
            continue
        m = re.match(r"^\s+(\S.*?)\s*// ([0-9A-F]+): ([0-9A-F ]+)", line)
        if m and code is not None:
            address, text = int(m.group(2), 16), m.group(1)
            target = None
            if re.match(r"s_(c?branch)", text):
                step = int(m.group(3).split()[0][-4:], 16)
                target = address + 4 + 4 * (step - (1 << 16) if step & 0x8000 else step)
            code.append((address, text, target))
    return out


def test_waits_are_counted_along_every_path():
    mfma = "v_mfma_f32_16x16x4_f32 v[0:3], v8, v9, v[0:3]"
    body = [(16 + 4 * i, "v_mov_b32_e32 v20, 0", None) for i in range(10)]
    late = [(56, "v_add_f32_e32 v4, v3, v4", None), (60, "s_endpgm", None)]
    straight = [(8, mfma, None), *body, *late]
    assert not missing_waits(straight)
    skipping = [(8, mfma, None), (12, "s_cbranch_vccnz 10", 56), *body, *late]
    assert [x[1] for x in missing_waits(skipping)] == [TAKEN]
    waits = [(56, "s_nop 5", None), (60, "v_add_f32_e32 v4, v3, v4", None), (64, "s_endpgm", None)]
    assert not missing_waits([*skipping[:-2], *waits])
    assert len(missing_waits([(8, mfma, None), (12, "s_nop 8", None), (16, "v_mov_b32_e32 v2, 0", None)])) == 1
    assert not missing_waits([(8, mfma, None), (12, "s_nop 9", None), (16, "v_mov_b32_e32 v2, 0", None)])
    assert not missing_waits([(8, mfma, None), (12, mfma, None), (16, "s_nop 9", None), (20, "ds_write_b32 v3, v4", None)])
    assert len(missing_waits([(8, mfma, None), (12, "global_store_dword v[12:13], v1, off", None)])) == 1
    assert len(missing_waits([(8, mfma, None), (12, "v_mfma_f32_16x16x4_f32 v[12:15], v2, v9, v[12:15]", None)])) == 1


def test_the_library_waits_for_its_matrix_products(tmp_path):
    if not os.path.exists(LLVM) or not os.path.exists(K.library_path()):
        pytest.skip("needs llvm-objdump and the built library")
    lib = shutil.copy(K.library_path(), tmp_path)
    subprocess.run([LLVM, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True, timeout=120)
    objects = [x for x in os.listdir(tmp_path) if "gfx950" in x]
    assert objects
    products, early = 0, []
    for x in objects:
        listing = subprocess.run([LLVM, "-d", x], cwd=tmp_path, check=True, capture_output=True, text=True, timeout=300).stdout
        for name, code in _functions(listing).items():
            products += sum(t.startswith("v_mfma") for _, t, _ in code)
            early += [(name, *m) for m in missing_waits(code)]
    assert products > 1000
    assert not early, early[:10]
