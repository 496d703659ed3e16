"""CPU check of the registers of the norm's backward in the built library (what the compiler
notes beside each kernel). Results do not depend on them, but speed does: a row is held in
registers from its loads to its stores, and where a second way of loading in the same kernel
had raised them, rows of 8200 to 32768 bf16 took up to 1.4 times as long (3000 x 12289
without ds and dw 60 us, then 82; 4096 x 4095 with both 54, then 69), and float32 rows of
4096 to 16384 with both up to 1.2 times (4096 x 8192 127 us, then 141)."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from lm_head_linear_amd import _lib

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
READELF = os.path.join(ROCM, "llvm", "bin", "llvm-readelf")

pytestmark = pytest.mark.skipif(not os.path.exists(READELF) or shutil.which("c++filt") is None,
                                reason="no llvm-readelf or c++filt")


def code_objects(path):
    """The gfx950 code objects in a library's bundles, one a source file."""
    data, magic = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length] and size:
                yield data[at + off:at + off + size]
            p += 24 + length
        at = data.find(magic, at + 24)


def notes(needle, folder):
    """{name: {noted: value}} of the kernels in the code objects that hold `needle`."""
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__ as g
        g.build()
    path, out = str(folder / "k.co"), {}
    for code in code_objects(_lib.LIB_PATH):
        if needle.encode() not in code:
            continue
        with open(path, "wb") as f:
            f.write(code)
        text = subprocess.run([READELF, "--notes", path], capture_output=True, text=True).stdout
        cur = {}
        for line in text.split("\n"):
            m = re.match(r"\s+(?:- )?\.(name|private_segment_fixed_size|vgpr_count|vgpr_spill_count):\s+(\S+)",
                         line)
            if m:
                cur[m.group(1)] = m.group(2)
                if m.group(1) == "vgpr_spill_count":       # a kernel's keys are in order: the last
                    name = cur.pop("name")
                    out[name] = {k: int(v) for k, v in cur.items()}
    plain = subprocess.run(["c++filt"], input="\n".join(out), capture_output=True, text=True).stdout
    return dict(zip((n.replace("flce::(anonymous namespace)::", "") for n in plain.split("\n")), out.values()))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    return notes("k_rms_norm_bwd", tmp_path_factory.mktemp("co"))


# (rows' type, threads, chunks a thread): registers and spilled ones with neither, dw, ds, both
BF, F32 = "unsigned short", "float"
MOST = {
    (BF, 256, 2): [(78, 0), (113, 0), (97, 0), (127, 0)],
    (BF, 256, 4): [(149, 0), (214, 0), (179, 0), (236, 0)],
    (BF, 1024, 4): [(128, 6), (128, 118), (128, 34), (128, 176)],
    (F32, 256, 4): [(75, 0), (117, 0), (97, 0), (134, 0)],
    (F32, 1024, 4): [(70, 0), (120, 0), (86, 0), (128, 0)],
}


@pytest.mark.parametrize("which", sorted(MOST))
def test_registers(kernels, which):
    t, lanes, chunks = which
    for i, most in enumerate(MOST[which]):
        ds, dw = ("false", "true")[i >> 1], ("false", "true")[i & 1]
        pre = f"void k_rms_norm_bwd<{t}, {t}, {lanes}, {chunks}, {ds}, {dw}, false"
        found = {n: v for n, v in kernels.items() if n.startswith(pre)}
        assert found
        for name, got in found.items():
            got = got["vgpr_count"], got["vgpr_spill_count"]
            assert got[0] <= most[0] and got[1] <= most[1], (name.split("(")[0], got, most)
