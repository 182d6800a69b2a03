"""The machine code of the gradient's products (CPU only: it is compiled, not run).

Their matrix instructions are inline assembly, of which the compiler does not know
the waits that they need. What mfma_tiles.hpp relies on is checked in the assembly
of every kernel of theirs:
  - an accumulator is a matrix instruction's source and destination at once
  - they all stand between the two waits of a sum, and nothing else there touches an
    accumulator register or memory of its own
  - none of the two instructions in front of one, on any way to it, is a vector
    instruction that writes one of its operands (2 wait states; LDS reads are waited for
    by the counters)
  - nothing spills
"""
import os
import re
import subprocess

import pytest

from invariant_token_log_fp32_amd import build

pytestmark = pytest.mark.slow


def registers(operand):
    m = re.fullmatch(r"([av])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m.group(1), k) for k in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.fullmatch(r"([av])(\d+)", operand)
    return {(m.group(1), int(m.group(2)))} if m else set()


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "products.s")
    flags = [f for f in build.HIP_FLAGS if f not in ("-shared", "-fPIC")]
    src = os.path.join(build.PKG, "csrc", "rlk_linear_grad.hip")
    res = subprocess.run([build.hipcc(), *flags, "-I", build.INCLUDE, "-I", os.path.dirname(src), "-S",
                          "--cuda-device-only", "-o", out, src], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    found, labels, name, text = {}, {}, None, open(out).read()
    for line in text.splitlines():
        m = re.match(r"(_ZN\S*(?:k_product|k_weight)\S*):", line)
        if m:
            name = m.group(1)
            found[name], labels[name] = [], {}
        elif name and re.match(r"\.LBB\S+:", line):
            labels[name][line.split(":")[0]] = len(found[name])
        elif name and line.startswith("\t") and not line.strip().startswith((";", ".")):
            op, _, rest = line.split(";")[0].strip().partition(" ")
            op, _, more = op.partition("\t")
            found[name].append((op, [a.strip() for a in (more + " " + rest).split(",")]))
        elif line.startswith(".Lfunc_end"):
            name = None
    return found, labels, text


def ways_to(code, labels):
    """For each instruction those that may run just before it."""
    before = [[] for _ in code]
    for k, (op, a) in enumerate(code):
        if op.startswith(("s_cbranch", "s_branch")):
            before[labels[a[0]]].append(k)
        if op not in ("s_branch", "s_endpgm") and k + 1 < len(code):
            before[k + 1].append(k)
    return before


def test_products_have_their_waits(kernels):
    found, labels, _ = kernels
    assert len(found) >= 9
    for name, code in found.items():
        waits = [k for k, (op, a) in enumerate(code) if op == "s_nop" and a == ["15"]]
        products = [k for k, (op, _) in enumerate(code) if op.startswith("v_mfma")]
        assert len(waits) == (16 if "k_product" in name else 4), (name, waits)  # one sum for each kind of tile
        inside = []
        for k in range(0, len(waits), 4):
            first, last, after, end = waits[k:k + 4]
            assert last == first + 1 and end == after + 1, (name, waits)
            inside += range(last + 1, after)
        assert products and set(products) <= set(inside), name
        before = ways_to(code, labels[name])
        for k in products:
            op, a = code[k]
            assert a[0] == a[3] and a[0].startswith("a["), (name, a)
            needed = registers(a[1]) | registers(a[2])
            for near in set(before[k]) | {q for p in before[k] for q in before[p]}:
                what, b = code[near]
                if what.startswith("v_") and not what.startswith("v_mfma"):
                    assert not registers(b[0]) & needed, (name, what, b, a)
        for k in inside:
            op, a = code[k]
            if not op.startswith("v_mfma"):
                assert not any(r[0] == "a" for x in a for r in registers(x)), (name, op, a)
                assert not op.startswith("scratch_"), (name, op, a)


def test_products_do_not_spill(kernels):
    found, _, text = kernels
    blocks = re.split(r"\n  - \.", text[text.index("amdhsa.kernels:"):])
    seen = 0
    for b in blocks:
        if "k_product" in b or "k_weight" in b:
            seen += 1
            for what in ("private_segment_fixed_size", "vgpr_spill_count"):
                assert re.search(rf"\.{what}:\s+0\b", b), (what, b[:300])
    assert seen == len(found)
