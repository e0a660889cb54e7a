"""Every host function that the library's parts declare for one another (csrc/kernels.h) has a caller."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_gemm_mma_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_every_declared_function_is_called():
    declared = set(re.findall(r"^(?:cudaError_t|int|size_t|bool|void) (\w+)\(", code("kernels.h"), re.M))
    assert len(declared) > 30
    sources = "\n".join(code(n) for n in sorted(os.listdir(CSRC)) if n != "kernels.h")
    # one mention is the definition
    alone = [n for n in sorted(declared) if len(re.findall(rf"\b{n}\b", sources)) < 2]
    assert not alone, alone
