"""The state-space layer's host code linked with tests/launch_recorder.cpp: what
its calls would launch, without a GPU."""
import collections
import ctypes
import os
import subprocess

import momentum_delta_rule_gb300 as mdn
from momentum_delta_rule_gb300 import build

Launch = collections.namedtuple("Launch", "kernel limit grid block shared")   # limit: None for a launch
WRAPPED = ("cudaGetDevice", "cudaGetLastError", "cudaMemsetAsync", "cudaFuncSetAttribute", "__cudaGetKernel",
           "__cudaLaunchKernel")
UNITS = ("mdn_ssm_api", "mdn_conv", "mdn_norm", "mdn_scan", "mdn_scan_bwd")


class Recorder:
    def __init__(self, folder):
        build.build()
        here = os.path.dirname(os.path.abspath(__file__))
        path = os.path.join(str(folder), "librecorder.so")
        cmd = [build.NVCC, build.ARCH, "-shared", "-std=c++17", "-Xcompiler", "-fPIC", "-o", path,
               os.path.join(here, "launch_recorder.cpp")]
        cmd += [os.path.join(build.BUILD_DIR, u + ".o") for u in UNITS]
        # the library's own runtime and symbols, not those of another one in the process
        cmd += ["-Xlinker", "-Bsymbolic"] + [a for w in WRAPPED for a in ("-Xlinker", "--wrap=" + w)]
        subprocess.run(cmd, check=True)
        self.lib = ctypes.CDLL(path)
        mdn.ssm.declare(self.lib)

    def calls(self, name, *args):
        """The limits set and the kernels launched by one call that succeeds."""
        self.lib.recorder_clear()
        st = getattr(self.lib, name)(*args)
        assert st == 0, (name, st)
        out = []
        for i in range(self.lib.recorder_count()):
            k, lim, g, b, s = (ctypes.c_uint64(), ctypes.c_long(), ctypes.c_uint(), ctypes.c_uint(), ctypes.c_long())
            self.lib.recorder_event(i, *map(ctypes.byref, (k, lim, g, b, s)))
            out.append(Launch(k.value, None if lim.value < 0 else lim.value, g.value, b.value, s.value))
        return out


def norm_args(rows, D, dtype, gate=False, bwd=False):
    """Arguments of mdn_norm_residual_fwd or _bwd on addresses never dereferenced."""
    p = lambda i: ctypes.c_void_p(0x100000 * (i + 1))
    g = p(2) if gate else None
    if not bwd:
        return (p(0), p(1), g, p(3), p(4), p(5), p(6), p(7), None, rows, D, 0, 1e-6, D, D, D, dtype, None)
    return (p(0), p(1), g, p(3), p(4), p(5), p(6), p(7), p(8), p(9), p(10), p(11) if gate else None, p(12), p(13), p(14),
            rows, D, 0, D, D, D, D, D, dtype, p(15), 1 << 40, None)


def conv_args(n_seq, packed, tokens, D, W, dtype, bwd=False):
    """Arguments of mdn_short_conv_fwd or _bwd."""
    p = lambda i: ctypes.c_void_p(0x100000 * (i + 1))
    cu = p(20) if packed else None
    B, T = (1, tokens) if packed else (n_seq, tokens // n_seq)
    if not bwd:
        return (p(0), p(1), p(2), p(3), p(4), p(5), cu, n_seq, B, T, D, W, 1, D, dtype, None)
    return (p(0), p(1), p(2), p(3), p(4), p(5), p(6), p(7), p(8), p(9), cu, n_seq, B, T, D, W, 1, D, D, dtype, p(10),
            1 << 40, None)


def scan_bwd_args(n_seq, packed, tokens, D, G, N, dtype):
    """Arguments of mdn_ssm_scan_bwd."""
    p = lambda i: ctypes.c_void_p(0x100000 * (i + 1))
    cu = p(30) if packed else None
    B, T = (1, tokens) if packed else (n_seq, tokens // n_seq)
    return tuple(p(i) for i in range(20)) + (cu, n_seq, B, T, D, G, N, 1, D, D, G * N, G * N, D, D, dtype, p(40), 1 << 60,
                                             None)
