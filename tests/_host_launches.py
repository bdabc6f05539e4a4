"""The block-selected attention's host side without a GPU: the library's objects linked with a runtime that
only takes notes (_fake_runtime.cpp)."""
import ctypes
import os
import re
import subprocess
from collections import namedtuple

import free_sparse_attention_head_b200 as svoo
from free_sparse_attention_head_b200 import build as svoo_build

HERE = os.path.dirname(os.path.abspath(__file__))
OBJECTS = ["block_select.o", "block_attn.o", "block_grad.o", "cache.o"]
MOST_SMEM = 232448   # dynamic shared memory of one block

Launch = namedtuple("Launch", "kernel grid threads smem bad")


class Host:
    """Calls of the C API; `launches`, `allowed` and `maps` are those of the last one."""

    def __init__(self, folder):
        svoo_build.build()
        objects = [os.path.join(svoo_build.BUILD, o) for o in OBJECTS]
        if not all(os.path.exists(o) for o in objects):
            svoo_build.build(force=True)
        path = os.path.join(folder, "libhost.so")
        cuda = os.path.join(os.path.dirname(os.path.dirname(svoo_build._nvcc())), "include")
        if not os.path.isdir(cuda):
            cuda = "/usr/local/cuda/include"
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", cuda,
                               os.path.join(HERE, "_fake_runtime.cpp"), *objects, "-o", path])
        self.lib = ctypes.CDLL(path)
        self.lib.fake_log.restype = ctypes.c_char_p
        for name, (res, args) in svoo._SIGS.items():
            if re.match("svoo_(block|cache)_", name):
                fn = getattr(self.lib, name)
                fn.restype, fn.argtypes = res, args

    def __call__(self, name, *args):
        self.lib.fake_clear()
        status = getattr(self.lib, name)(*args)
        lines = [x.split() for x in self.lib.fake_log().decode().splitlines()]
        self.launches = [Launch(x[1], tuple(map(int, x[2:5])), int(x[5]), int(x[6]), x[7] == "1")
                         for x in lines if x[0] == "launch"]
        self.allowed = [(x[1], int(x[2])) for x in lines if x[0] == "allow"]
        self.maps = [tuple(map(int, x[1:])) for x in lines if x[0] == "map"]   # address, rows, columns, box
        return status

    # every pointer is a number that nothing reads
    def select(self, s, x=0x10000):
        return self("svoo_block_select", s, x, x, None, x, x, 1 << 60, None, None)

    def attn(self, s, x=0x10000, k=0x20000, v=0x30000):
        return self("svoo_block_attn", s, x, k, v, x, None, 0.1, x, x, x, 1 << 60, None, None)

    def backward(self, s, x=0x10000, k=0x20000, v=0x30000):
        return self("svoo_block_attn_backward", s, x, k, v, x, x, x, x, None, 0.1, x, x, x, x, 1 << 60, None, None)

    def cache(self, s, x=0x10000, k=0x20000, v=0x30000, idx=None, weight=None):
        return self("svoo_cache_attn", s, x, k, v, None, idx, 0.1, weight, x, x, x, 1 << 60, None, None)


def shape(**fields):
    return ctypes.pointer(svoo.BlockShape(**fields))
