"""What the host code of linear attention and of the group norm launches (no GPU:
the CUDA runtime's calls are recorded)."""
import ctypes
import os
import subprocess

import pytest

import momentum_delta_rule_gb300 as mdn
from momentum_delta_rule_gb300 import build
from tests import _launches
from tests.test_abi_attn import BWD, FWD, P
from tests.test_gpu_attn_paths import COMBINED, JOINED

UNITS = ("mdn_attn_api", "mdn_attn", "mdn_attn_tc", "mdn_attn_tc32", "mdn_attn_step", "mdn_group_norm")
WRAPPED = _launches.WRAPPED + ("cudaLaunchKernelExC", "cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags", "cudaMemcpyAsync")


class Recorder(_launches.Recorder):
    def __init__(self, folder):
        build.build()
        here = os.path.dirname(os.path.abspath(__file__))
        path = os.path.join(str(folder), "libattnrecorder.so")
        cmd = [build.NVCC, build.ARCH, "-shared", "-std=c++17", "-Xcompiler", "-fPIC", "-o", path,
               os.path.join(here, "attn_launch_recorder.cpp")]
        cmd += [os.path.join(build.BUILD_DIR, u + ".o") for u in UNITS]
        cmd += ["-Xlinker", "-Bsymbolic"] + [a for w in WRAPPED for a in ("-Xlinker", "--wrap=" + w)]
        subprocess.run(cmd, check=True)
        self.lib = ctypes.CDLL(path)
        mdn.attn.declare(self.lib)

    def copies(self, name, *args):
        """The kernels launched and the copies (to, from or None for zeros, bytes) of
        one call that succeeds."""
        self.lib.recorder_clear_copies()
        launched = self.calls(name, *args)
        out = []
        for i in range(self.lib.recorder_copies()):
            t, f, n = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
            self.lib.recorder_copy(i, *map(ctypes.byref, (t, f, n)))
            out.append((t.value, f.value or None, n.value))
        return launched, out


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return Recorder(tmp_path_factory.mktemp("recorder"))


def _args(d, **over):
    v = dict(d, **over)
    return [v[k] for k in d]


NOTHING = dict(q=None, k=None, v=None, log_decay=None, T=0, ws=None, bytes=0)
BYTES = 2 * 4 * 16 * 8 * 4        # the states of 2 sequences and 4 heads of 16 x 8


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("over", [{}, dict(cu=P(0x9000), B=1)])
def test_without_tokens_no_kernel_reads_the_decays(rec, dtype, over):
    # Everything that has no tokens may be NULL, the decays with it, so the states
    # are copied as they are.
    kw = dict(NOTHING, dtype=dtype, **over)
    S0, S_T = P(0xa000), P(0xb000)
    fwd = lambda **s: rec.copies("mdn_linear_attn_fwd", *_args(FWD, o=None, **kw, **s))
    assert fwd(S0=S0, S_T=S_T) == ([], [(0xb000, 0xa000, BYTES)])
    assert fwd(S0=None, S_T=S_T) == ([], [(0xb000, None, BYTES)])
    assert fwd(S0=S0, S_T=S0) == ([], [])
    assert fwd(S0=S0, S_T=None) == ([], [])
    bwd = lambda **s: rec.copies("mdn_linear_attn_bwd", *_args(BWD, do=None, dq=None, dk_out=None, dv_out=None, **kw, **s))
    assert bwd(dS_T=S0, dS0=S_T) == ([], [(0xb000, 0xa000, BYTES)])
    assert bwd(dS_T=None, dS0=S_T) == ([], [(0xb000, None, BYTES)])
    assert bwd(dS_T=S0, dS0=None) == ([], [])


def test_without_sequences_nothing_happens(rec):
    assert rec.copies("mdn_linear_attn_fwd", *_args(FWD, **dict(NOTHING, o=None, S_T=P(0xb000), B=0, n_seq=0))) == ([], [])


def test_with_tokens_kernels_run(rec):
    launched, copies = rec.copies("mdn_linear_attn_fwd", *_args(FWD, S_T=P(0xb000)))
    assert len([e for e in launched if e.limit is None]) == 1 and copies == []


@pytest.mark.parametrize("n_seq,rows,D,G", [(32768, 32768, 2048, 16), (16384, 32768, 4096, 32), (1 << 20, 1 << 20, 512, 4),
                                            (4096, 4096, 16384, 8), (30000, 90000, 96, 3)])
def test_the_norms_gradient_over_many_sequences_asks_for_less_than_its_rows(n_seq, rows, D, G):
    """Each sequence leaves sums of weight and bias behind: however many there are,
    they take less than the bf16 rows themselves."""
    size = mdn.lib().mdn_group_norm_bwd_workspace_size(n_seq, rows, D, G, 1, 1)
    assert 0 < size <= rows * D * 2, size


def _kernels(rec, bwd, dtype, lens, H, Hkv, dk, dv, packed):
    """Launches of a call by what they do: laying packed sequences out and summing
    shared heads' gradients left out."""
    n = len(lens)
    B, T = (1, sum(lens)) if packed else (n, lens[0])
    kw = dict(cu=P(0x9000) if packed else None, n_seq=n, B=B, T=T, H=H, Hkv=Hkv, dk=dk, dv=dv, ld_q=H * dk, ld_k=Hkv * dk,
              ld_v=Hkv * dv, dtype=dtype)
    call = ("mdn_linear_attn_bwd", *_args(BWD, ld_do=H * dv, **kw)) if bwd else ("mdn_linear_attn_fwd", *_args(FWD, **kw))
    out = [e for e in rec.calls(*call) if e.limit is None]
    if packed and out[0].grid == 1 and out[0].block == 1024:
        out = out[1:]
    return out[:-2] if bwd and H != Hkv else out


@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed,where", JOINED)
def test_where_segments_join_the_states_themselves(rec, lens, H, Hkv, dk, dv, packed, where):
    # the segments' own states, then the outputs: nothing between them
    for w in where:
        out = _kernels(rec, w.startswith("bwd"), w.endswith("bf16"), lens, H, Hkv, dk, dv, packed)
        assert len(out) == 2, w


@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed,offset", COMBINED)
def test_where_a_kernel_joins_the_states(rec, lens, H, Hkv, dk, dv, packed, offset):
    for bwd in (False, True):
        for dtype in (0, 1):
            out = _kernels(rec, bwd, dtype, lens, H, Hkv, dk, dv, packed)
            assert len(out) == 3 and out[1].grid == len(lens) * H
