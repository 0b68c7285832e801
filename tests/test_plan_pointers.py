"""A kernel launched behind its plan is resident while the plan still writes, so nothing that reaches it may be
declared read-only or unaliased for its whole life: the compiler might then load it ahead of the wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_verification_gdn_gb300",
                    "csrc")


def kernels(text):
    """(name, parameters, body) of every kernel: parameters up to the body's brace, the body up to a brace in column 0."""
    for m in re.finditer(r"__global__ void", text):
        head, rest = text[m.start():].split("{\n", 1)
        names = re.findall(r"(\w+_kernel)\(", head)
        if names:
            yield names[0], head[head.index(names[0]):], rest.split("\n}\n", 1)[0]


def test_kernels_behind_a_plan_declare_nothing_read_only():
    seen, wrong = [], []
    for name in sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))):
        with open(os.path.join(CSRC, name)) as f:
            for kernel, parameters, body in kernels(f.read()):
                if "wait_for_plan()" in body:
                    seen.append(kernel)
                    if "__restrict__" in parameters:
                        wrong.append(kernel)
    assert {"qk_rope_kernel", "window_rows_kernel", "window_tiles_kernel"} <= set(seen)
    assert not wrong
