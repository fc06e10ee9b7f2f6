"""LDS arrays that are read or written in wider pieces than their elements state the alignment that this takes."""

import glob
import os
import re

from fp8_w8a8_quantized_token_amd.build import CSRC

WIDE = ("uint4", "float4", "v4u", "v4u32", "v4i", "v4f", "v8bf")  # 16 bytes each


def test_arrays_accessed_by_16_bytes_are_aligned():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path).read()
        for line in re.findall(r"__shared__ [^;]*;", text):
            aligned = int((re.search(r"aligned\((\d+)\)", line) or [0, 0])[1])
            if re.search(r"__shared__ (?:%s) " % "|".join(WIDE), line):
                continue
            for name in re.findall(r"(\w+)\[", re.sub(r"__attribute__\(\(.*?\)\)\)?", "", line)):
                wide = r"reinterpret_cast<(?:const )?(?:%s)\*>\(&?%s\b" % ("|".join(WIDE), name)
                if re.search(wide, text):
                    seen += 1
                    assert aligned >= 16, f"{os.path.basename(path)}: {line}"
    assert seen >= 3  # the pattern still finds what it is meant for
