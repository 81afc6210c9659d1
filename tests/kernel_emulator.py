"""The linear attention and rotary kernels on the CPU: their own sources, built against a stand-in
for the HIP runtime (tests/emulation), called through their C entry points.

Every array ends at a page that cannot be touched, LDS starts out as NaN, and the waves of a
workgroup run one after the other between barriers, in ascending or descending order.  A call is a
process of its own, so that a fault is a failed test.
"""
import ctypes
import mmap
import os
import shutil
import signal
import subprocess

import torch

from state_space_sequence_cumsum_amd import build, linattn

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "emulation")
OUT = os.path.join(HERE, "_build")
LIBRARY = os.path.join(OUT, "libemulated.so")
PARTS = [os.path.join(build.CSRC, n) for n in
         ("ssd_linattn.hip", "ssd_linattn_step.hip", "ssd_rotary.hip", "ssd_linattn_api.cpp")]
PARTS.append(os.path.join(HERE, "emulator.cpp"))


def _compiler():
    for c in (shutil.which("amdclang++"), os.path.join(os.path.dirname(build.hipcc()), "amdclang++")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("amdclang++ not found; the ROCm toolchain is required")


def _made():
    """Builds the library where a source is newer than it; its path."""
    sources = PARTS + [os.path.join(HERE, "hip", "hip_runtime.h")]
    sources += [os.path.join(build.CSRC, n) for n in os.listdir(build.CSRC) if n.endswith(".h")]
    sources.append(os.path.join(build.ROOT, "include", "ssd.h"))
    if os.path.exists(LIBRARY) and all(os.path.getmtime(s) <= os.path.getmtime(LIBRARY) for s in sources):
        return LIBRARY
    os.makedirs(OUT, exist_ok=True)
    tag = f"{os.getpid()}.tmp"
    flags = ["-x", "c++", "-std=c++17", "-O2", "-fPIC", "-w", "-I", HERE, "-include", "hip/hip_runtime.h"]
    objects, runs = [], []
    for s in PARTS:
        objects.append(os.path.join(OUT, f"{os.path.basename(s)}.{tag}.o"))
        runs.append(subprocess.Popen([_compiler(), *flags, "-c", s, "-o", objects[-1]],
                                     stderr=subprocess.PIPE, text=True))
    for r in runs:
        err = r.communicate()[1]
        if r.returncode != 0:
            raise RuntimeError(f"the emulated kernels do not build:\n{err}")
    subprocess.run([_compiler(), "-shared", *objects, "-o", f"{LIBRARY}.{tag}"], check=True)
    for o in objects:
        os.remove(o)
    os.replace(f"{LIBRARY}.{tag}", LIBRARY)
    return LIBRARY


_lib = None


def lib():
    global _lib
    if _lib is None:
        L = ctypes.CDLL(_made())
        real = linattn.lib()
        for n in ("ssd_linattn", "ssd_linattn_step", "ssd_linattn_backward", "ssd_rotary",
                  "ssd_linattn_workspace_bytes", "ssd_linattn_backward_workspace_bytes"):
            getattr(L, n).argtypes, getattr(L, n).restype = getattr(real, n).argtypes, getattr(real, n).restype
        _lib = L
    return _lib


_libc = ctypes.CDLL(None, use_errno=True)
_libc.mmap.restype = ctypes.c_void_p
_libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t] + [ctypes.c_int] * 3 + [ctypes.c_long]
_libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
_libc.munmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t]


class Memory:
    """Arrays that end (on 16 bytes) at a page that cannot be touched, shared with the calls'
    processes."""

    def __init__(self):
        self._maps = []

    def room(self, nbytes):
        n, page = (nbytes + 15) // 16 * 16, mmap.PAGESIZE
        size = (n + page - 1) // page * page + 2 * page
        p = _libc.mmap(None, size, mmap.PROT_READ | mmap.PROT_WRITE,
                       mmap.MAP_SHARED | mmap.MAP_ANONYMOUS, -1, 0)
        assert p not in (None, ctypes.c_void_p(-1).value)
        self._maps.append((p, size))
        for guard in (p, p + size - page):
            assert _libc.mprotect(guard, page, 0) == 0
        return p + size - page - n

    def put(self, t):
        """The address of a copy of t (None for None)."""
        if t is None:
            return None
        t = t.contiguous()
        n = t.numel() * t.element_size()
        p = self.room(n)
        ctypes.memmove(p, t.data_ptr(), n)
        return p

    @staticmethod
    def get(p, shape, dtype):
        t = torch.empty(shape, dtype=dtype)
        ctypes.memmove(t.data_ptr(), p, t.numel() * t.element_size())
        return t

    def close(self):
        for p, size in self._maps:
            _libc.munmap(p, size)


def start(fn, args, descending):
    """Starts a call of a C entry point in a process of its own."""
    L = lib()
    pid = os.fork()
    if pid == 0:
        try:
            signal.alarm(300)
            L.emulator_descending(int(descending))
            os._exit(getattr(L, fn)(*args))
        finally:
            os._exit(255)
    return pid


def finish(pid, what):
    _, status = os.waitpid(pid, 0)
    assert os.WIFEXITED(status), f"{what} ended by signal {os.WTERMSIG(status)}"
    assert os.WEXITSTATUS(status) == 0, f"{what} returned {os.WEXITSTATUS(status)}"
