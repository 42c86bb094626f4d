"""CPU: the library holds every kernel once.  A kernel defined in a header with internal linkage is compiled
into each source file that includes it, also where nothing launches it."""
import collections
import re
import subprocess


def test_no_kernel_is_compiled_twice(cuda_lib):
    from hstu_pointwise_attention_jagged_b200 import binding
    names = subprocess.run(["nm", "-C", binding.library_path()], check=True, capture_output=True, text=True).stdout
    kernels = collections.Counter(m.group(1) for m in re.finditer(r"^\S+ [tTwW] (?:void )?(hstu::\w*_kernel\b.*)$", names, re.M))
    assert len(kernels) > 20
    assert {k: n for k, n in kernels.items() if n > 1} == {}
