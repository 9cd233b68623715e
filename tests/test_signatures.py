"""The ctypes signatures against the prototypes in include/fa.h (no GPU): as many arguments, each of
its kind.  One too few and a stream goes to the library as a 32-bit int."""

import ctypes
import re

import pytest

from tiled_attention_fa_gb300 import _lib

SCALARS = {"int": ctypes.c_int, "long long": ctypes.c_longlong, "size_t": ctypes.c_size_t, "float": ctypes.c_float,
           "unsigned long long": ctypes.c_ulonglong, "unsigned int": ctypes.c_uint, "fa_status": ctypes.c_int,
           "unsigned": ctypes.c_uint, "const char*": ctypes.c_char_p}


def prototypes():
    """{name: (result, [argument])}: the C types, "*" for a pointer argument."""
    with open(_lib.HEADER) as fh:
        src = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    found = {}
    for res, name, args in re.findall(r"^([a-z_][a-z_ *]*?)\s*\b(fa_\w+)\s*\(([^)]*)\)\s*;", src, flags=re.M):
        args = [" ".join(a.split()) for a in args.split(",") if a.strip() not in ("", "void")]
        found[name] = (res.strip(), ["*" if "*" in a else a.rsplit(" ", 1)[0] for a in args])
    return found


PROTOTYPES = prototypes()


def test_every_function_is_there():
    assert set(PROTOTYPES) == set(_lib._SIGS) >= set(_lib.header_functions())


@pytest.mark.parametrize("name", sorted(PROTOTYPES))
def test_signature(name):
    res, args = PROTOTYPES[name]
    want = [ctypes.c_void_p if a == "*" else SCALARS[a] for a in args]
    assert _lib._SIGS[name] == (want, SCALARS[res])
