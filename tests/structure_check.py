"""Compares a ctypes structure with its declaration in include/dwpt_seq.h."""
import ctypes
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"int32_t": ctypes.c_int32, "uint32_t": ctypes.c_uint32, "uint64_t": ctypes.c_uint64, "int64_t": ctypes.c_int64, "double": ctypes.c_double}


def check_structure(name, cls, nested=()):
    text = open(os.path.join(ROOT, "include", "dwpt_seq.h"), encoding="utf-8").read()
    end = text.index("} %s;" % name)
    body = text[text.rindex("typedef struct {", 0, end) + len("typedef struct {"):end]
    fields = []
    for decl in body.split(";"):
        decl = decl.strip()
        if not decl:
            continue
        base, names = re.match(r"((?:const )?\w+)\s*(.*)", decl, re.S).groups()
        for n in names.split(","):
            n = n.strip()
            fields.append((n.lstrip("* "), ctypes.c_void_p if n.startswith("*") or "*" in base else {**TYPES, **dict(nested)}[base]))
    assert [(f[0], f[1]) for f in cls._fields_] == fields
