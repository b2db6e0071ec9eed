"""Every global access of the FP8 quantise and read-back kernels is range-checked
in the checked build (read from the source)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_quantized_rank_b200", "csrc")


def _kernel(s, name):
    at = s.index(name + "(Fp8Shape s")
    return s[at:s.index("\n}\n", at)]


def test_sites():
    s = open(os.path.join(CSRC, "fp8.cu")).read()
    q, d = _kernel(s, "k_fp8_quantize"), _kernel(s, "k_fp8_dequantize")
    assert {int(v) for v in re.findall(r"CQL_IN\(.*, (\d+)\)", q)} == {402, 403, 404}     # source, codes, scales
    assert {int(v) for v in re.findall(r"CQL_IN\(.*, (\d+)\)", d)} == {405, 406, 407}     # scales, codes, output
    assert q.count("CQL_IN(") == 4 and d.count("CQL_IN(") == 4                             # vector and single accesses


def test_no_site_is_shared():
    sites = []
    for f in ("fp8.cu", "fp8_decode.cu", "fp8_gemm.cu"):
        s = open(os.path.join(CSRC, f)).read()
        sites.append(set(re.findall(r"CQL_IN\([^;]*?, (4\d\d)\)", s)))
    assert not sites[0] & sites[1] and not sites[0] & sites[2] and not sites[1] & sites[2]
    assert all(sites)
