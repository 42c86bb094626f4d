"""CPU: the digest by which bench.py tells whether recorded DRAM counters are current covers every source of the
kernel they were recorded of."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hstu_pointwise_attention_jagged_b200", "csrc")
sys.path.insert(0, ROOT)


def included(name, seen):
    """The project's files that `name` includes, itself among them."""
    if name not in seen:
        seen.add(name)
        with open(os.path.join(CSRC, name)) as f:
            for other in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                if os.path.exists(os.path.join(CSRC, other)):
                    included(other, seen)
    return seen


def test_digest_covers_the_kernel_and_its_plan():
    import bench
    needed = included("hstu_fwd_sm100.cuh", set()) | included("schedule_kernel.cuh", set()) | {"hstu_attn.cu"}
    assert needed <= set(bench.KERNEL_SOURCES), needed - set(bench.KERNEL_SOURCES)


def test_digest_changes_with_every_source(tmp_path, monkeypatch):
    import bench
    where = tmp_path / "hstu_pointwise_attention_jagged_b200" / "csrc"
    where.mkdir(parents=True)
    for name in bench.KERNEL_SOURCES:
        with open(os.path.join(CSRC, name)) as f:
            (where / name).write_text(f.read())
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    digests = [bench.kernel_source_digest()]
    for name in bench.KERNEL_SOURCES:
        (where / name).write_text((where / name).read_text() + "// changed\n")
        digests.append(bench.kernel_source_digest())
    assert len(set(digests)) == len(digests)
