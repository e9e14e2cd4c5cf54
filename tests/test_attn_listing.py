"""Checks of the attention kernels' assembly, as it is built (no GPU): what the compiler does
not see to around the loads that attn.h writes out.

Their m0 has no other use, as they overwrite it unnamed; and a load is at least five
instructions behind any vector instruction that wrote a scalar register of its address."""
import os
import re
import subprocess

import pytest

from gated_delta_rule_77_amd import build

WAIT = 5
LOAD = "global_load_lds"
# vector instructions whose second operand is a scalar result (a carry or a flag)
SECOND = re.compile(r"v_(mad_[ui]64_[ui]32|(add|sub|subrev|addc|subb|subbrev)_co|div_scale)")


def scalars(operand):
    """The scalar registers that an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return range(int(m[1]), int(m[2]) + 1)
    m = re.fullmatch(r"s(\d+)", operand)
    return [int(m[1])] if m else []


def parse(text):
    """(instructions as (operation, operands, within a written-out block, line), labels)."""
    code, labels, ours = [], {}, False
    for line in text.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            ours = "#ASMSTART" in line
            continue
        line = re.split(r";|//", line)[0].strip()
        m = re.fullmatch(r"([\w.$]+):", line)
        if m:
            labels[m[1]] = len(code)
        elif line and not line.startswith("."):
            op, _, rest = line.partition(" ")
            # an offset or a modifier behind the last operand is no part of it
            code.append((op, [x.strip().split(" ")[0] for x in re.split(r",(?![^\[]*\])", rest)] if rest else [], ours, line))
    return code, labels


def faults(text):
    """(loads found, complaints) of a listing."""
    code, labels = parse(text)
    bad = ["m0 outside of the loads' blocks: " + line for _, _, ours, line in code if not ours and re.search(r"\bm0\b", line)]
    # scalar registers that a vector instruction wrote, and how many instructions ago at the least, on any path
    before, work = {}, []

    def reach(i, ages):
        old = before.get(i)
        new = dict(ages) if old is None else {**old, **{r: a for r, a in ages.items() if a < old.get(r, WAIT)}}
        if new != old and i < len(code):
            before[i] = new
            work.append(i)

    for i in (0, *labels.values()):
        reach(i, {})
    while work:
        i = work.pop()
        op, operands, _, line = code[i]
        passed = int(operands[0]) + 1 if op == "s_nop" else 1
        ages = {r: a + passed for r, a in before[i].items() if a + passed < WAIT}
        if op.startswith("v_"):
            for x in operands[:2 if SECOND.match(op) else 1]:
                ages.update((r, 0) for r in scalars(x))
        if op.startswith("s_cbranch") or op == "s_branch":
            reach(labels[operands[0]], ages)
        if op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            reach(i + 1, ages)
    loads = 0
    for i, (op, operands, _, line) in enumerate(code):
        if op.startswith(LOAD):
            loads += 1
            if any(r in before.get(i, {}) for x in operands for r in scalars(x)):
                bad.append("too close behind a vector instruction that writes its address: " + line)
    return loads, bad


@pytest.mark.parametrize("source", ["attn_fwd.hip", "attn_bwd.hip"])
def test_written_out_loads(source, tmp_path):
    out = tmp_path / "listing.s"
    subprocess.run([build._hipcc(), *build.COMMON, *build.EXTRA.get(source, []), "--offload-device-only", "-S", os.path.join(build.CSRC, source),
                    "-o", str(out)], check=True, capture_output=True)
    loads, bad = faults(out.read_text())
    assert loads > 100 and not bad, "\n".join(bad[:20])


BLOCK = "\t;;#ASMSTART\n\ts_mov_b32 m0, s9\n\ts_nop 0\n\tglobal_load_lds_dwordx4 v1, s[4:5]%s\n\t;;#ASMEND\n"
LISTINGS = [
    (True, "k:\n\tv_readfirstlane_b32 s4, v0\n\ts_nop 2\n" + BLOCK % "" + "\ts_endpgm\n"),
    (False, "k:\n\tv_readfirstlane_b32 s4, v0\n\ts_nop 1\n" + BLOCK % "" + "\ts_endpgm\n"),
    (False, "k:\n\tv_readlane_b32 s5, v0, 3\n" + BLOCK % " offset:16" + "\ts_endpgm\n"),
    (True, "k:\n\tv_readlane_b32 s6, v0, 3\n" + BLOCK % "" + "\ts_endpgm\n"),
    (False, "k:\n\tv_cmp_lt_i32_e64 s[4:5], v0, v1\n\ts_nop 0\n" + BLOCK % "" + "\ts_endpgm\n"),
    (False, "k:\n\tv_mad_u64_u32 v[0:1], s[4:5], v2, v3, 0\n" + BLOCK % "" + "\ts_endpgm\n"),
    (True, "k:\n\tv_cndmask_b32_e64 v0, v1, v2, s[4:5]\n" + BLOCK % "" + "\ts_endpgm\n"),
    # around a loop's end
    (False, "k:\n.L1:\n" + BLOCK % "" + "\ts_nop 7\n\tv_readfirstlane_b32 s4, v0\n\ts_cbranch_scc1 .L1\n\ts_endpgm\n"),
    (False, "k:\n\ts_mov_b32 m0, s3\n" + BLOCK % "" + "\ts_endpgm\n"),
]


@pytest.mark.parametrize("n", range(len(LISTINGS)))
def test_the_checks_see_what_they_are_for(n):
    fine, text = LISTINGS[n]
    loads, bad = faults(text)
    assert loads == 1 and fine == (not bad)
