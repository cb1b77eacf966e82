"""The kernels' sources (no GPU needed)."""
import collections
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiered_sparse_mla_gb300", "csrc")


def device_functions(text):
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__device__ (?:__forceinline__|__noinline__) [\w:<> ]*?\b(\w+)\(", text):
        i = text.index("{", m.end())
        depth = 0
        for j in range(i, len(text)):
            depth += (text[j] == "{") - (text[j] == "}")
            if depth == 0:
                break
        yield m.group(1), " ".join(text[i:j + 1].split())


def test_no_device_function_is_written_twice():
    """What two kernels have to do alike (a query row's codes, say) is one function in a header."""
    where = collections.defaultdict(set)
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                for function, body in device_functions(f.read()):
                    where[body].add(f"{name}: {function}")
    assert len(where) > 50
    assert not [sorted(x) for x in where.values() if len(x) > 1]
