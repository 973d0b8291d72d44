"""The GPU code of a source as assembly, compiled as the build compiles it."""
import concurrent.futures as cf
import os
import re
import subprocess
import tempfile

from sparse_mixture_experts_gate_amd import build as B

SOURCES = ["combine.hip", "dispatch.hip", "mx4.hip", "norm.hip", "rmsnorm.hip"]
_texts = {}


def no_hipcc() -> bool:
    return not os.path.exists(B.HIPCC)


def _compile(src: str) -> str:
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, src + ".s")
        subprocess.run([B.HIPCC, *B.flags(src), "--cuda-device-only", "-S",
                        os.path.join(B.CSRC, src), "-o", out], check=True, capture_output=True)
        return open(out).read()


def assembly(src: str) -> str:
    """One of SOURCES; all of them are compiled at the first call."""
    if not _texts:
        with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
            _texts.update(zip(SOURCES, ex.map(_compile, SOURCES)))
    return _texts[src]


def kernels(asm: str) -> dict:
    """{mangled name: its code}."""
    return dict(re.findall(r"^(_Z\w+):.*?\n(.*?)^\.Lfunc_end", asm, re.M | re.S))
