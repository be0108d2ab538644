"""The kernels' source texts, for tests of an order that no run on a GPU shows reliably."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_b200", "csrc")


def text(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        s = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)


def _block(s, at):
    """The text between the brace at s[at] and its partner."""
    depth = 0
    for i in range(at, len(s)):
        depth += (s[i] == "{") - (s[i] == "}")
        if depth == 0:
            return s[at + 1:i]
    raise AssertionError("unbalanced braces")


def kernels():
    """{kernel name: body} of every __global__ function under csrc/."""
    found = {}
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        s = text(name)
        for m in re.finditer(r"__global__\s+void\s", s):
            # past __launch_bounds__(...), whose arguments may nest parentheses
            at = m.end()
            bounds = re.compile(r"\s*__launch_bounds__\s*\(").match(s, at)
            if bounds:
                at, depth = bounds.end(), 1
                while depth:
                    depth += (s[at] == "(") - (s[at] == ")")
                    at += 1
            kernel = re.compile(r"\s*(\w+)\s*\(").match(s, at)
            found[kernel.group(1)] = _block(s, s.index("{", kernel.end()))
    return found


def roles(body):
    """The branches of a kernel's outermost `if (warp ...) {} else if ... {} else {}` chain, as texts."""
    out = []
    start = re.search(r"\n    if \(warp == 0\) \{", body).start()
    at = body.index("{", start)
    while True:
        part = _block(body, at)
        out.append(part)
        rest = body[at + len(part) + 2:]
        follow = re.match(r"\s*else[^{;]*\{", rest)
        if not follow:
            return out
        at += len(part) + 2 + follow.end() - 1
