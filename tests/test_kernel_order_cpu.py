"""Orders that the kernels' sources have to keep and that no run would show for certain: read from the sources, with
the calls of a kernel replaced by what they do, in the order of the text."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_quantized_moe_b200", "csrc")


def body_at(text, at):
    """The braces' contents of the definition that follows position `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def load(name):
    """(kernels, device functions) of a source and the headers beside it: name -> body."""
    def read(path):
        return re.sub(r"//[^\n]*", "", open(path).read())
    text = read(os.path.join(CSRC, name))
    kernels = {}
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(", text):
        kernels[m.group(1)] = body_at(text, m.end())
    functions = {}
    for t in [text] + [read(p) for p in glob.glob(os.path.join(CSRC, "*.cuh"))]:
        for m in re.finditer(r"__device__[^;{()]*?\b(\w+)\(", t):
            end = t.index(")", m.end())
            if re.match(r"\s*(const)?\s*\{", t[end + 1:]):
                functions.setdefault(m.group(1), body_at(t, end))
    return kernels, functions


def steps(body, functions, words, inside=()):
    """The words of a body in order, its calls expanded."""
    out = []
    for m in re.finditer(r"\b(\w+)\b(?=\s*(?:<[\w, ]*>)?\s*\()|tcgen05\.alloc", body):
        w = m.group(1) or "tcgen05.alloc"
        if w == "sync" and body[:m.start()].endswith("cl."):
            out.append("cluster_sync_all")
        elif w in words:
            out.append(w)
        elif w in functions and w not in inside:
            out += steps(functions[w], functions, words, inside + (w,))
    return out


REMOTE = ("map_shared_rank", "leader_addr", "mma_commit_pair")
BARRIERS = ("cluster_sync_all", "cluster_started", "cluster_wait")


@pytest.mark.parametrize("name", ["kernels_sample.cu", "kernels_linear.cu", "kernels_tc.cu"])
def test_other_blocks_memory_after_a_cluster_barrier(name):
    """A block may reach into another one's shared memory only when that one is known to have started: a whole cluster
    barrier lies before the first such access."""
    kernels, functions = load(name)
    seen = 0
    for kernel, body in kernels.items():
        order = steps(body, functions, REMOTE + BARRIERS)
        first = next((i for i, w in enumerate(order) if w in REMOTE), None)
        if first is None:
            continue
        seen += 1
        before = order[:first]
        whole = "cluster_sync_all" in before or (
            "cluster_started" in before and "cluster_wait" in before[before.index("cluster_started"):])
        assert whole, (kernel, order[:first + 1])
    assert seen > 0


@pytest.mark.parametrize("name", ["kernels_linear.cu", "kernels_tc.cu"])
def test_dependents_start_after_tensor_memory_is_held(name):
    """A block lets the next kernel start only when it holds its tensor memory (a barrier lies between): blocks of the
    next kernel that took what it waits for would not give it back before it ends."""
    kernels, functions = load(name)
    seen = 0
    for kernel, body in kernels.items():
        order = steps(body, functions, ("tcgen05.alloc", "pdl_trigger", "__syncthreads", "cluster_sync_all"))
        if "tcgen05.alloc" not in order or "pdl_trigger" not in order:
            continue
        seen += 1
        between = order[order.index("tcgen05.alloc"):order.index("pdl_trigger")]
        assert "__syncthreads" in between or "cluster_sync_all" in between, (kernel, order)
    assert seen > 0
