"""Compiled code of the kernels that choose at run time whether their 16-byte stores go
past the caches: both kinds of store are there. The compiler merges two stores that
differ in the hint alone into one without it, unless the source keeps them apart, and
nothing but time shows that."""
import re

import pytest

from asm_util import assembly, kernels, no_hipcc

pytestmark = pytest.mark.skipif(no_hipcc(), reason="no hipcc")

# bf16 (t) row outputs; 4-byte words of codes; fp32 rows are never stored past the caches
KERNELS = [("norm.hip", r"norm_fwd(_long)?_kernelIt", "dwordx4"),
           # layer norm's backward: with dresidual, and rows of 8 waves and 2 chunks
           ("norm.hip", r"norm_bwd_kernelIt(Li\dELi\dELb1|Li8ELi2E)", "dwordx4"),
           ("rmsnorm.hip", r"rms_(fwd|bwd)(_long)?_kernelIt", "dwordx4"),
           ("combine.hip", r"token_combine(_bwd)?_kernelIt", "dwordx4"),
           ("dispatch.hip", r"(move|dispatch_few)_kernel", "dwordx4"),
           ("mx4.hip", r"mx4_quantize_kernelI[tf]", "dword"),
           ("mx4.hip", r"mx4_dequantize_kernelIt", "dwordx4")]


@pytest.mark.parametrize("src,name,width", KERNELS)
def test_both_kinds_of_store(src, name, width):
    found = {k: code for k, code in kernels(assembly(src)).items() if re.search(name, k)}
    assert found
    for k, code in found.items():
        stores = re.findall(rf"^\s*global_store_{width}\s.*$", code, re.M)
        past = [s for s in stores if re.search(r"\bnt\b", s)]
        assert past and len(past) < len(stores), (k, len(past), len(stores))


@pytest.mark.parametrize("src,name", [("norm.hip", r"norm_bwd_kernelIt(?!Li8ELi2E)Li\dELi\dELb0"),
                                      ("norm.hip", r"norm_(fwd|bwd)\w*_kernelIf"),
                                      ("rmsnorm.hip", r"rms_(fwd|bwd)\w*_kernelIf"),
                                      ("combine.hip", r"token_combine\w*_kernelIf")])
def test_none_past_the_caches(src, name):
    """fp32 rows, whose lanes store every other 16 bytes, and the backward's rows that are
    slower that way."""
    found = {k: code for k, code in kernels(assembly(src)).items() if re.search(name, k)}
    assert found
    for k, code in found.items():
        assert not re.search(r"^\s*global_store_\w+\s.*\bnt\b", code, re.M), k
