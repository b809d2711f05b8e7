"""A kernel whose wait gave up may not leave before the copies and products that it has in
flight are done: they would write into shared or tensor memory of the next block.  Those last
waits have a limit of their own and must not end early because the abort flag is set, which it
then is.  Read from the sources: to make a kernel give up a wait would take a kernel that hangs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_exact_attention_ra_gb300",
                    "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def _calls(text, name):
    """The argument lists of the calls of `name`, split at their commas."""
    for m in re.finditer(r"\b" + name + r"\(", text):
        depth, args, start = 1, [], m.end()
        for i in range(m.end(), len(text)):
            c = text[i]
            depth += (c in "([{") - (c in ")]}")
            if depth == 0 or (depth == 1 and c == ","):
                args.append(text[start:i].strip())
                start = i + 1
            if depth == 0:
                break
        yield args


@pytest.mark.parametrize("name", FILES)
def test_waits_for_work_in_flight_do_not_end_at_the_abort_flag(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    for args in _calls(text, "mbar_wait"):
        assert len(args) == 5 and args[3] != "nullptr", f"{name}: mbar_wait({', '.join(args)})"


def test_every_kernel_with_tensor_memory_drains():
    text = {f: open(os.path.join(CSRC, f)).read() for f in FILES}
    for name in ("ra_fwd_tc.cu", "ra_bwd_tc.cu", "ra_gemm_tc.cu", "ra_pair.cuh"):
        assert len(list(_calls(text[name], "mbar_drain"))) >= 2, name
    body = text["ra_device.cuh"].split("void mbar_drain(")[1].split("\n}\n")[0]
    assert "abort" not in body and "globaltimer_ns()" in body
