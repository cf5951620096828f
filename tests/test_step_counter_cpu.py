"""The optimizer's step counter is written by a kernel whose threads all read it first: what orders the
write behind the reads is checked on the source, since a thread that comes late does so too rarely for a
run to show it."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "linear_cross_entropy_forward_gb300", "csrc", "flce_adamw.cu")


def _body(name):
    """A kernel's body without its comments."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    start = text.index("{", text.index(name + "("))
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]


def test_a_blocks_ticket_comes_behind_all_of_its_reads():
    body = _body("adamw_kernel")
    read, ticket = body.index("*a.step + 1"), body.index("atomicAdd(a.ticket")
    write = body.index("*a.step = step")
    assert read < ticket < write
    # a barrier of the whole block lies between, under conditions that are the same for all of its threads
    barrier = body.index("__syncthreads()", read)
    assert barrier < ticket
    guard = body.rindex("if (", 0, barrier)
    assert body[guard:body.index("{", guard)].split() == ["if", "(a.last", "&&", "!skip)"]


def test_the_norms_ticket_comes_behind_its_sum():
    body = _body("norm_kernel")
    assert body.index("a.partial[a.base + blockIdx.x] = total") < body.index("__threadfence()") \
        < body.index("atomicAdd(a.ticket")
