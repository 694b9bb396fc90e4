"""The cache operators' host code over a stand-in for the CUDA runtime (fake_cudart.cpp):
pointers are numbers that nothing reads."""
import ctypes as C
import os
import subprocess

from decode_megakernel_sm_gb300 import _lib as L
from decode_megakernel_sm_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def _compiled():
    """Its library, built where a source is newer."""
    out = os.path.join(B.BUILD, "fake")
    so, obj = os.path.join(out, "libkv_fake.so"), os.path.join(out, f"kv_ops.{os.getpid()}.o")
    fake = os.path.join(HERE, "fake_cudart.cpp")
    if os.path.exists(so) and all(os.path.getmtime(f) <= os.path.getmtime(so) for f in B._deps() + [fake, __file__]):
        return so
    os.makedirs(out, exist_ok=True)
    nvcc = B._nvcc()
    # (device code as PTX only: it is not used)
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-std=c++17", "-O1",
                    "-Xcompiler", "-fPIC", "-I", B.INCLUDE, "-c", os.path.join(B.CSRC, "kv_ops.cu"),
                    "-o", obj], check=True)
    tmp = f"{so}.tmp{os.getpid()}"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I",
                    os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
                    fake, obj, "-o", tmp], check=True)
    os.replace(tmp, so)
    os.remove(obj)
    return so


class Fake:
    def __init__(self):
        self.lib = C.CDLL(_compiled())
        for name, (res, args) in L.SIGNATURES.items():
            if name.startswith(("mk_kv_", "mk_attn_")):
                f = getattr(self.lib, name)
                f.restype, f.argtypes = res, args
        self.lib.fake_launch.restype = C.c_char_p
        self.lib.fake_reset()

    def launches(self):
        return [self.lib.fake_launch(i).decode() for i in range(self.lib.fake_launches())]

    def fail(self, call, after=0, error=2):
        self.lib.fake_fail(call.encode(), after, error)
