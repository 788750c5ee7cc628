"""The argument structs of include/w4a4.h for calls of the C ABI itself, as struct formats with the
fields' names read off the header."""
import os
import re
import struct

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a4.h")
FORMATS = {  # Q: a size or pointer, q: a stride, i: an int, f: a float
    "w4a4_kv_cache": struct.Struct("=Q5Q7q8i"),
    "w4a4_kv_append_args": struct.Struct("=Q9Q8q6ifi"),
    "w4a4_paged_attention_args": struct.Struct("=Q5QQ4qf3i"),
    "w4a4_block_norm_args": struct.Struct("=Q9Q5q7iffi"),
}


def fields(name):
    """Field names of a struct of the header, in order."""
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, src).group(1)
    return [re.sub(r".*[ *]", "", part.strip()) for line in body.split(";") for part in line.split(",") if part.strip()]


def pack(name, **values):
    """The struct's bytes; what is not given is 0, `bytes` the struct's size."""
    names = fields(name)
    assert set(values) <= set(names), set(values) - set(names)
    values = {"bytes": FORMATS[name].size, **values}
    return FORMATS[name].pack(*[values.get(n, 0) for n in names])
