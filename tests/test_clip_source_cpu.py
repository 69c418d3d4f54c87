"""The list kernels clip in place, one of them in the launch that also sums the squares.  Loads on the read-only
path (__ldg) need memory that nothing writes while the kernel runs: the source takes it only where the
launch does not write the gradients."""
import os
import re

from learnable_channel_permutation_b200 import build


def test_gradients_that_the_launch_clips_are_not_read_as_constants():
    text = open(os.path.join(build.CSRC, "clip.cu")).read()
    loads = re.findall(r"[^;\n]*(?:__ldg\(|ld\.global\.nc)", text)
    assert loads and all("CONST ? " in x for x in loads)
    kernels = re.findall(r"\n(small|squares|apply)_kernel\((.*?)\n}\n", text, flags=re.S)
    assert [k for k, _ in kernels] == ["squares", "apply", "small"]
    reads = {k: re.findall(r"squares_of<\w+, ([^>]*)>", body) for k, body in kernels}
    assert reads == dict(squares=["true"], apply=[], small=["!APPLY"])
    assert "apply<" in dict(kernels)["small"] and "apply<" not in dict(kernels)["squares"]
