"""What is read from tensor memory is named by the wait for it (on the host, from the source).

A load of tensor memory gives its registers to the compiler before their values
are there. Only a wait that takes each register as an operand keeps what reads
it behind the wait; without, a compiler may put it in front. Such a build would
have to read registers too early to be tried, so the source is looked at.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_get_dispatch_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def waits(text):
    """(name, {array: registers}, body) of each function that waits for loads of tensor memory."""
    found = []
    for m in re.finditer(r"void (\w+)\(([^)]*(?:\(&\w+\)[^)]*)*)\) \{", text):
        body = text[m.end():text.index("\n}", m.end())] if "\n" in text[m.end():m.end() + 1] else \
            text[m.end():text.index("\n", m.end())]
        if "tcgen05.wait::ld" in body:
            found.append((m.group(1), {a: int(n) for a, n in re.findall(r"\(&(\w+)\)\[(\d+)\]", m.group(2))}, body))
    return found


@pytest.mark.parametrize("name", ["expert_linear_fp8.cu", "tensor.cuh"])
def test_a_wait_names_every_register_that_it_waits_for(name):
    found = waits(source(name))
    assert found
    for function, arrays, body in found:
        assert arrays, function
        for array, n in arrays.items():
            tied = {int(i) for i in re.findall(r'"\+[rf]"\(%s\[(\d+)\]\)' % array, body)}
            assert tied == set(range(n)), (function, array, set(range(n)) - tied)


@pytest.mark.parametrize("name", ["expert_linear.cu", "expert_linear_fp8.cu"])
def test_what_is_loaded_is_waited_for_before_it_is_read(name):
    text = source(name)
    names = {f for n in ("tensor.cuh", name) for f, _, _ in waits(source(n))}
    loads = list(re.finditer(r"tmem_load\d+\((\w+),", text))
    assert names and loads
    for m in loads:
        after = text[m.end():]
        use = re.search(r"\b%s\b" % m.group(1), after)
        assert re.search(r"\b(%s)\((\w+, )?$" % "|".join(names), after[:use.start()]), text[m.start():m.end() + use.end()]
