"""Waits of the chunk-attention kernel's converged warps. Each lane polls a
barrier, the abort flag and its own timer, so that lanes can disagree on giving
up; whoever then goes on alone would meet the others' full-mask votes at another
place. Every such decision has to be voted on. Read from the source, as a wait
that gives up cannot be brought about without a stuck kernel. No GPU."""
import os
import re

import global_soft_capped_b200 as g2

SOURCE = os.path.join(os.path.dirname(g2.__file__), "csrc", "extend.cuh")


def code():
    with open(SOURCE) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def call_around(text, at):
    """Names of the calls whose parentheses enclose position `at`, inner to outer."""
    names, depth = [], 0
    for i in range(at, -1, -1):
        if text[i] == ")":
            depth += 1
        elif text[i] == "(":
            if depth:
                depth -= 1
            else:
                names.append(re.search(r"(\w*)\s*$", text[:i]).group(1))
        elif text[i] in ";{}" and not depth:
            break
    return names


def test_polled_conditions_are_voted():
    text = code()
    kernel = text[text.index("extend_sm100("):]
    poll = r"\*abort_flag(?!\s*=\s*0;)|mbar_test_wait\(|globaltimer_ns\(\) -"
    polls = [m.start() for m in re.finditer(poll, kernel)]
    assert len(polls) >= 5
    for at in polls:
        assert {"__all_sync", "__any_sync"} & set(call_around(kernel, at)), kernel[at - 80:at + 80]


def test_results_of_waits_are_voted():
    text = code()
    kernel = text[text.index("extend_sm100("):]
    args = r"(?:[^()]|\((?:[^()]|\([^()]*\))*\))*"
    waits = list(re.finditer(r"(\w+) = mbar_wait\(" + args + r"\);\s*", kernel))
    assert len(waits) == kernel.count("mbar_wait(") and len(waits) >= 10
    for m in waits:
        vote = f"{m.group(1)} = __all_sync(0xffffffffu, {m.group(1)});"
        assert kernel[m.end():].startswith(vote), m.group(0) + kernel[m.end():m.end() + 60]
