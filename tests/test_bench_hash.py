"""What the hash behind the stored DRAM traffic covers (CPU): every source that
the benchmarked kernels are made of, or that chooses their grids."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "diffusion_transformer_elementwise_gb300", "csrc")
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def sources():
    import bench
    out = {}
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            out[name] = bench._code_only(f.read())
    return bench, out


def test_left_out_sources_define_nothing_of_the_benchmarked_kernels():
    bench, text = sources()
    assert bench.OTHER_SOURCES <= set(text)
    # what the kernels' host interface declares
    names = set(re.findall(r"^(?:inline )?(?:cudaError_t|int) (\w+)\(", text["dit_internal.h"], re.M))
    assert {"current_device", "resident_ctas", "launch_modulate", "launch_rga_full"} <= names
    for name in names:
        defined = re.compile(rf"^[a-z][\w:<> ]*\b{name}\([^;{{]*\)\s*{{", re.M)
        where = {f for f, t in text.items() if defined.search(t)}
        assert where and not where & bench.OTHER_SOURCES, (name, where)


def test_hashed_sources_include_no_left_out_one():
    bench, text = sources()
    for f, t in text.items():
        if f not in bench.OTHER_SOURCES:
            used = set(re.findall(r'#include "([^"]+)"', t))
            assert not used & bench.OTHER_SOURCES, f


def test_the_hash_follows_the_launch_limits(tmp_path, monkeypatch):
    """An edit of the file that holds resident_ctas changes it."""
    bench, text = sources()
    pkg = tmp_path / "diffusion_transformer_elementwise_gb300" / "csrc"
    pkg.mkdir(parents=True)
    for f, t in text.items():
        (pkg / f).write_text(t, encoding="utf-8")
    real = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == real
    (where,) = [f for f, t in text.items() if "int resident_ctas(const DeviceInfo& dev, const void* fn, int block, size_t smem) {" in t]
    (pkg / where).write_text(text[where].replace("n = 1;", "n = 2;"), encoding="utf-8")
    assert bench.kernel_source_hash() != real
