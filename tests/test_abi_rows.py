"""fp8_rows is described three times: in the header, as a ctypes structure, and as the packed bytes that the
binding hands over. They agree."""

import ctypes
import re

from fp8_w8a8_quantized_token_amd import _lib
from tests.test_abi import HEADER

C_TYPES = {"void*": ctypes.c_void_p, "int64_t": ctypes.c_int64}


def test_structure_is_the_headers():
    body = re.search(r"typedef struct fp8_rows \{(.*?)\} fp8_rows;", open(HEADER).read(), re.S).group(1)
    fields = re.findall(r"^\s*([\w*]+) (\w+);", body, re.M)
    assert [(name, C_TYPES[kind]) for kind, name in fields] == list(_lib.Rows._fields_)


def test_packed_bytes_are_the_structures():
    for values in ((0x7F00_0000_1230, 24, 3072, 128), (16, 1, 0, -8), (1 << 63, 65535, (1 << 63) - 1, -(1 << 63))):
        assert _lib.pack_rows(*values) == bytes(_lib.Rows(*values))
