"""What the compiler gave each kernel of a built library: registers and
scratch, from the metadata of the gfx950 code objects that it carries."""
import os
import re
import shutil
import struct
import subprocess

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
CXXFILT = "c++filt"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def available() -> bool:
    return all(shutil.which(p) for p in (READELF, CXXFILT))


def code_objects(path):
    with open(path, "rb") as f:
        blob = f.read()
    at = blob.find(MAGIC)
    while at >= 0:
        entries, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        o = at + len(MAGIC) + 8
        for _ in range(entries):
            off, size, n = struct.unpack_from("<QQQ", blob, o)
            triple = blob[o + 24:o + 24 + n].decode()
            o += 24 + n
            if size and triple.endswith("gfx950"):
                yield blob[at + off:at + off + size]
        at = blob.find(MAGIC, at + len(MAGIC))


def kernels(path, tmp):
    """{demangled name: {"vgpr", "sgpr", "scratch"}}; the vector count is the
    whole allocation, accumulation registers included."""
    out = {}
    for i, obj in enumerate(code_objects(path)):
        name = os.path.join(str(tmp), f"code{i}.o")
        with open(name, "wb") as f:
            f.write(obj)
        text = subprocess.run([READELF, "--notes", name], capture_output=True, text=True, check=True).stdout
        found = []
        for part in re.split(r"\n  - \.a", text)[1:]:
            field = lambda k: re.search(r"\." + k + r":\s*(\S+)", part)      # noqa: E731
            if field("vgpr_count"):
                sym = re.search(r"\.symbol:\s*'?([^'\s]+?)\.kd", part).group(1)
                found.append((sym, {"vgpr": int(field("vgpr_count").group(1)), "sgpr": int(field("sgpr_count").group(1)),
                                    "scratch": int(field("private_segment_fixed_size").group(1))}))
        names = subprocess.run([CXXFILT], input="\n".join(s for s, _ in found), capture_output=True, text=True,
                               check=True).stdout.split("\n")
        out.update({n: v for n, (_, v) in zip(names, found)})
    return out


def waves(vgpr: int) -> int:
    """Waves of a SIMD by vector registers: 512 a lane, given out in eights."""
    return min(8, 512 // max(8, -(-vgpr // 8) * 8))
