"""The experts' kernels count vector-memory operations in explicit waits: the
loads into LDS, which the compiler does not see, and, of a whole tile, the stores
of the tile before.  Two properties of the compiled code carry that: a wave stores a
whole tile in exactly the stores that the waits allow for, and nothing else of
vector memory (spilled registers) lies between the loads.  This test compiles
experts.hip for gfx950 to assembly, as the library build does, and looks."""
import os
import re
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "fine_grained_sparse_amd", "csrc", "experts.hip")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# kinds as in experts.hpp: stores of 16 bytes per wave and tile (kStores; EXP_UP does not count its own)
STORES = {1: 16, 2: 32, 3: 16, 4: 16, 5: 16}


def test_stores_and_no_scratch():
    with tempfile.TemporaryDirectory() as tmp:
        out = os.path.join(tmp, "experts.s")
        subprocess.run([HIPCC, "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-x", "hip", "--offload-device-only",
                        "-S", SRC, "-o", out], check=True, capture_output=True)
        text = open(out).read()
    found = {}
    for m in re.finditer(r"^(_ZN3moe\S*k_expertsILi(\d)ELi(n?\d)E\S*):(.*?)\.Lfunc_end", text, re.S | re.M):
        ops = [l.split()[0] for l in m.group(4).split("\n") if l.startswith("\t") and not l.strip().startswith((".", ";"))]
        found[m.group(2), m.group(3)] = ops
    assert set(found) == {("0", "n1"), ("1", "n1"), ("2", "n1"), ("3", "n1"), ("4", "n1"), ("5", "n1"), ("2", "4"), ("3", "5")}
    for (a, b), ops in found.items():
        assert not any(o.startswith(("scratch_", "buffer_", "flat_")) for o in ops), (a, b)
        if a != "0":
            want = STORES[int(a)] + (STORES[int(b)] if b != "n1" else 0)
            assert ops.count("global_store_dwordx4") == want, (a, b)
            assert sum(o.startswith("global_store") for o in ops) == want, (a, b)
        assert sum(o.startswith("v_mfma_f32_16x16x32_bf16") for o in ops) > 0
