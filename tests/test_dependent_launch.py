"""How kernels that start before the work ahead of them ends may read memory (by reading their source, no GPU).

Such a kernel (programmatic dependent launch) is resident while the kernels ahead still write what it will
read.  The non-coherent load (ld.global.nc, __ldg, and what the compiler may make of a read through a const
__restrict__ pointer) is defined for memory that nothing writes for the whole length of the kernel, so it
has no place there: a line that an earlier reader left in the SM's read-only path may be old.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q4_quantized_matmul_gb300", "csrc")
NON_COHERENT = re.compile(r"ld\.global[a-z.]*\.nc\b|__ldg\s*\(|const\s+[\w:]+\s*\*\s*__restrict__")


def code(name, csrc=CSRC):
    """A source file without its comments."""
    with open(os.path.join(csrc, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def mx_sources(csrc=CSRC):
    return [n for n in sorted(os.listdir(csrc)) if n.startswith(("q4q_mx", "q4q_moe")) and n.endswith((".cu", ".cuh"))]


def test_mxfp4_and_expert_kernels_read_coherently():
    names = mx_sources()
    assert {"q4q_mx.cuh", "q4q_mxfp4.cu", "q4q_mxmm.cu", "q4q_moe.cu"} <= set(names)
    for name in names:
        assert NON_COHERENT.findall(code(name)) == [], name


def test_projections_read_their_activations_coherently():
    """Weights and biases are resident by contract and may be read any way; the activations may not."""
    for name, kernels in (("q4q_gemv.cuh", ("quantize_acts",)), ("q4q_rmma.cu", ("act_to_rmma_kernel", "rmma_reduce_kernel"))):
        text = code(name)
        for kernel in kernels:
            body = text[text.index(" %s(" % kernel if kernel == "quantize_acts" else "\n%s(" % kernel):]
            body = body[:body.index("\n}\n")]
            assert ("__ldcg(" in body or "ld_behind_wait(" in body) and "__ldg(" not in body, kernel
    # whatever else these files read through the read-only path are biases
    for name in ("q4q_gemv.cuh", "q4q_rmma.cu"):
        assert all(a.startswith("p.bias") for a in re.findall(r"__ldg\s*\(([^)]*)\)", code(name))), name
