"""Refusals of the operators around the rule (decode_runs, short_conv, rms_norm): bad
arguments are rejected on the host before anything is launched, by the C entry points
(made-up pointers, never dereferenced) and by the binding (CPU tensors)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_130_b200", "csrc")
CUDA_INC = "/usr/local/cuda/include"
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_130_b200 import binding
    return binding.LIB


def _runs(lib, **kw):
    a = dict(q=1 << 20, k=1 << 21, v=1 << 22, la=1 << 23, be=1 << 24, S=1 << 40, slots=1 << 26,
             cu=1 << 27, o=1 << 30, N=2, total=8, Hk=1, Hv=2, Dk=16, Dv=8, n_slots=4, qs=16, ks=16,
             vs=16, las=2, bes=2, dtype=1, flags=0)
    a.update(kw)
    return lib.gdn_decode_runs(a["q"], a["k"], a["v"], a["la"], a["be"], a["S"], a["slots"], a["cu"],
                               a["o"], a["N"], a["total"], a["Hk"], a["Hv"], a["Dk"], a["Dv"],
                               a["n_slots"], a["qs"], a["ks"], a["vs"], a["las"], a["bes"],
                               a["dtype"], a["flags"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(la=None), INVALID),
    (dict(be=None), INVALID), (dict(S=None), INVALID), (dict(q=None), INVALID),
    (dict(N=-1), INVALID), (dict(total=-1), INVALID), (dict(Hk=-1), INVALID), (dict(Dk=0), INVALID),
    (dict(Dv=-2), INVALID), (dict(n_slots=-1), INVALID), (dict(dtype=5), INVALID),
    (dict(flags=8), INVALID), (dict(Hk=2, Hv=3, ks=32, qs=32, vs=24, las=3, bes=3), INVALID),
    (dict(cu=None), INVALID),                              # without offsets N = total
    (dict(qs=15), INVALID), (dict(ks=-16), INVALID), (dict(vs=0), INVALID), (dict(las=1), INVALID),
    (dict(ks=1 << 31), INVALID),
    (dict(q=(1 << 20) + 8), INVALID), (dict(la=(1 << 23) + 2), INVALID), (dict(cu=4), INVALID),
    (dict(o=(1 << 20) + 16), INVALID), (dict(o=1 << 40), INVALID), (dict(S=1 << 20), INVALID),
    (dict(S=1 << 27), INVALID),
    (dict(Dk=257, qs=257, ks=257), UNSUPPORTED), (dict(Dv=513, vs=2000), UNSUPPORTED),
    (dict(N=65536), UNSUPPORTED), (dict(N=65535, total=65535, Hv=65535), UNSUPPORTED),
    (dict(n_slots=2 ** 31 - 1, Hv=65535, Hk=65535), UNSUPPORTED),
    (dict(total=(1 << 30) + 1), UNSUPPORTED),
    (dict(N=0), OK), (dict(total=0), OK), (dict(Hv=0, Hk=0), OK),   # nothing to do
])
def test_decode_runs_rejects_before_launch(lib, kw, status):
    assert _runs(lib, **kw) == status


def _arrays(ptrs, strides, begin):
    return ((ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_longlong * len(strides))(*strides),
            (ctypes.c_int * len(begin))(*begin))


def _conv(lib, y=(1 << 30,), strides=(16,), begin=(0, 16), **kw):
    a = dict(x=1 << 20, w=1 << 21, b=None, S=1 << 40, slots=1 << 26, cu=1 << 27, N=2, total=8, C=16,
             W=4, n_slots=4, xs=16, silu=1, dtype=1, p=1, parts=len(y))
    a.update(kw)
    p, s, g = _arrays(y, strides, begin)
    return lib.gdn_short_conv_fwd(a["x"], a["w"], a["b"], a["S"], a["slots"], a["cu"], p, s, g,
                                  a["parts"], a["N"], a["total"], a["C"], a["W"], a["n_slots"],
                                  a["xs"], a["silu"], a["dtype"], a["p"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=(None,)), INVALID),
    (dict(N=-1), INVALID), (dict(C=0), INVALID), (dict(W=0), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=0, p=1), INVALID),                         # parameters: float32 or x's type
    (dict(xs=15), INVALID), (dict(strides=(8,)), INVALID), (dict(x=(1 << 20) + 2), INVALID),
    (dict(b=(1 << 21) + 4), INVALID), (dict(cu=None), INVALID), (dict(n_slots=-1), INVALID),
    (dict(begin=(0, 8)), INVALID), (dict(begin=(1, 16)), INVALID), (dict(parts=0), INVALID),
    (dict(y=(1 << 30, 1 << 31), strides=(8, 8), begin=(0, 8, 12)), INVALID),
    (dict(y=(1 << 30, 1 << 31), strides=(8, 8), begin=(0, 16, 16)), INVALID),
    (dict(y=(1 << 30,) * 4, strides=(4,) * 4, begin=(0, 4, 8, 12, 16)), INVALID),
    (dict(y=(1 << 30, 1 << 30), strides=(8, 8), begin=(0, 8, 16)), INVALID),   # parts overlap
    (dict(y=(1 << 20,)), INVALID), (dict(y=(1 << 40,)), INVALID), (dict(S=1 << 20), INVALID),
    (dict(y=(1 << 27,)), INVALID),                         # y over the offsets
    (dict(W=5), UNSUPPORTED), (dict(W=1), UNSUPPORTED), (dict(N=70000), UNSUPPORTED),
    (dict(C=1 << 25, xs=1 << 25), UNSUPPORTED),
    (dict(C=1 << 24, xs=1 << 24, total=1 << 20), UNSUPPORTED),
    (dict(N=0), OK), (dict(total=0), OK),
])
def test_short_conv_fwd_rejects_before_launch(lib, kw, status):
    assert _conv(lib, **kw) == status


def _conv_bwd(lib, dy=(1 << 30,), strides=(16,), begin=(0, 16), **kw):
    a = dict(x=1 << 20, w=1 << 21, b=None, cu=1 << 27, dx=1 << 31, dw=1 << 32, db=None, N=2, total=8,
             C=16, W=4, xs=16, dtype=1, p=1, ws=1 << 40, n=1 << 20)
    a.update(kw)
    p, s, g = _arrays(dy, strides, begin)
    return lib.gdn_short_conv_bwd(p, s, g, len(dy), a["x"], a["w"], a["b"], a["cu"], a["dx"], a["dw"],
                                  a["db"], a["N"], a["total"], a["C"], a["W"], a["xs"], 1, a["dtype"],
                                  a["p"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(ws=None), INVALID), (dict(n=100), INVALID), (dict(dx=1 << 20), INVALID),
    (dict(dw=(1 << 31) + 16), INVALID), (dict(ws=1 << 31), INVALID), (dict(dx=1 << 30), INVALID),
    (dict(db=1 << 32), INVALID), (dict(dw=(1 << 32) + 4), INVALID), (dict(W=9), UNSUPPORTED),
    (dict(cu=None), INVALID), (dict(strides=(3,)), INVALID),
])
def test_short_conv_bwd_rejects_before_launch(lib, kw, status):
    assert _conv_bwd(lib, **kw) == status


def _norm(lib, **kw):
    a = dict(x=1 << 20, w=1 << 21, r=None, g=None, y=1 << 30, sc=None, h=None, tokens=4, heads=2, D=64,
             group=0, xs=128, rs=0, gs=0, eps=1e-6, dtype=1, p=1)
    a.update(kw)
    return lib.gdn_rms_norm_fwd(a["x"], a["w"], a["r"], a["g"], a["y"], a["sc"], a["h"], a["tokens"],
                                a["heads"], a["D"], a["group"], a["xs"], a["rs"], a["gs"], a["eps"],
                                a["dtype"], a["p"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(D=0), INVALID),
    (dict(dtype=9), INVALID), (dict(dtype=0, p=1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(xs=127), INVALID),
    (dict(r=1 << 24, rs=100), INVALID), (dict(g=1 << 24, gs=0), INVALID), (dict(group=-1), INVALID),
    (dict(group=64), INVALID),                             # 8 bits without scales
    (dict(group=32, sc=1 << 33), UNSUPPORTED), (dict(group=128, sc=1 << 33), UNSUPPORTED),
    (dict(y=(1 << 20) + 16), INVALID), (dict(x=(1 << 20) + 4), INVALID),
    (dict(y=1 << 20, xs=130), INVALID),                    # in place needs dense rows
    (dict(r=1 << 24, rs=128, h=1 << 30), INVALID),         # h over y
    (dict(r=1 << 24, rs=130, h=1 << 24), INVALID),
    (dict(y=1 << 20, r=1 << 24, rs=128, h=1 << 25), INVALID),
    (dict(y=1 << 21), INVALID), (dict(group=64, sc=1 << 20), INVALID),
    (dict(D=(1 << 20) + 1, xs=1 << 22), UNSUPPORTED), (dict(tokens=1 << 30, heads=2), UNSUPPORTED),
    (dict(tokens=0), OK), (dict(heads=0), OK),
])
def test_rms_norm_fwd_rejects_before_launch(lib, kw, status):
    assert _norm(lib, **kw) == status


def _norm_bwd(lib, **kw):
    a = dict(dy=1 << 19, x=1 << 20, w=1 << 21, g=None, dr=None, dx=1 << 30, dw=1 << 31, dg=None,
             tokens=4, heads=2, D=64, ys=128, xs=128, gs=0, drs=0, eps=1e-6, ws=1 << 40, n=1 << 20)
    a.update(kw)
    return lib.gdn_rms_norm_bwd(a["dy"], a["x"], a["w"], a["g"], a["dr"], a["dx"], a["dw"], a["dg"],
                                a["tokens"], a["heads"], a["D"], a["ys"], a["xs"], a["gs"], a["drs"],
                                a["eps"], 1, 1, a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
    (dict(g=1 << 24, gs=128), INVALID), (dict(dg=1 << 33), INVALID),      # a gate and its gradient
    (dict(ws=None), INVALID), (dict(n=8), INVALID), (dict(dx=1 << 20), INVALID),
    (dict(dx=1 << 19), INVALID), (dict(ws=1 << 30), INVALID), (dict(dw=1 << 30), INVALID),
    (dict(ys=5), INVALID), (dict(dr=1 << 24, drs=5), INVALID), (dict(dw=(1 << 31) + 8), INVALID),
])
def test_rms_norm_bwd_rejects_before_launch(lib, kw, status):
    assert _norm_bwd(lib, **kw) == status


def test_workspace_sizes(lib):
    from gated_delta_rule_130_b200 import binding as b
    assert b.short_conv_bwd_workspace_size(0, 16, 4) == 0
    assert b.short_conv_bwd_workspace_size(8, 16, 7) == 0
    # one tile of 8 tokens: C (W + 1) floats
    assert b.short_conv_bwd_workspace_size(8, 16, 4) == 16 * 5 * 4
    assert b.rms_norm_bwd_workspace_size(3, 2, 100) == 6 * 100 * 4
    assert b.rms_norm_bwd_workspace_size(0, 2, 100) == 0
    assert b.rms_norm_bwd_workspace_size(10 ** 6, 1, 64) == 148 * 6 * 64 * 4


def test_binding_refuses_bad_shapes_and_cpu_tensors():
    from gated_delta_rule_130_b200 import binding as b
    z = torch.zeros
    q, v, g, S = z(4, 2, 16), z(4, 4, 8), z(4, 4), z(3, 4, 8, 16)
    for f in (lambda: b.decode_runs(q, q, v, g, g, S),               # on the CPU
              lambda: b.decode_runs(None, q, v, g, g, S),            # no q for the output
              lambda: b.decode_runs(q, q, v, g, g, S, out=v, want_output=False),
              lambda: b.decode_runs(q, z(4, 2, 8), v, g, g, S),
              lambda: b.decode_runs(q, q, z(5, 4, 8), g, g, S),
              lambda: b.short_conv_fwd(z(4, 8), z(8, 4)),
              lambda: b.short_conv_fwd(z(4, 8, 1), z(8, 4)),
              lambda: b.short_conv_bwd(z(4, 8), z(4, 8), z(8, 4)),
              lambda: b.rms_norm_fwd(z(4, 8), z(8)),
              lambda: b.rms_norm_bwd(z(4, 8), z(4, 8), z(8)),
              lambda: b.rms_norm_fwd(z(4, 0), z(0))):
        with pytest.raises(b.GdnError):
            f()


def test_binding_refuses_sizes_beyond_32_bits():
    # ctypes would cut 2^32 + 5 rows down to 5
    from gated_delta_rule_130_b200 import binding as b
    assert b._norm_sizes((2 ** 20, 4, 64)) == (2 ** 20, 4, 64)
    for shape in ((2 ** 32 + 5, 1), (1, 2 ** 32 + 8), (2 ** 16, 2 ** 16, 2, 8), (2, 2 ** 31, 8)):
        with pytest.raises(b.GdnError):
            b._norm_sizes(shape)
    with pytest.raises(b.GdnError):
        b._ints(4, 2 ** 31)


STUBS = r"""
#include <cuda_runtime.h>
#include "kernels.h"
int g_calls = 0;
extern "C" cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { ++g_calls; return cudaSuccess; }
namespace gdn {
cudaError_t launch_decode_runs(const RunsArgs &, bool, cudaStream_t) { ++g_calls; return cudaSuccess; }
cudaError_t launch_short_conv_fwd(const ConvArgs &, bool, cudaStream_t) { ++g_calls; return cudaSuccess; }
size_t short_conv_bwd_bytes(int total, int C, int W) { return (size_t)total * C * (W + 1) * 4; }
cudaError_t launch_short_conv_bwd(const ConvArgs &, bool, cudaStream_t) { ++g_calls; return cudaSuccess; }
cudaError_t launch_rms_norm_fwd(const NormArgs &, bool, cudaStream_t) { ++g_calls; return cudaSuccess; }
size_t rms_norm_bwd_bytes(int rows, int D) { return (size_t)rows * D * 4; }
cudaError_t launch_rms_norm_bwd(const NormArgs &, bool, cudaStream_t) { ++g_calls; return cudaSuccess; }
}
"""

HARNESS = r"""
#include <climits>
#include <cstdint>
#include <initializer_list>
#include <cstdio>
#include "gdn.h"
extern int g_calls;
#define P(x) reinterpret_cast<void *>(uintptr_t(x))
#define F(x) reinterpret_cast<float *>(uintptr_t(x))
#define I(x) reinterpret_cast<int *>(uintptr_t(x))
int main() {
    const int sizes[] = {INT_MIN, -1, 0, 1, 2, 3, 4, 64, 128, 256, 512, 65535, 65536, 1 << 20, 1 << 24, INT_MAX};
    const long long strides[] = {LLONG_MIN, -1, 0, 1, 1024, 1ll << 30, 1ll << 31, 1ll << 40, LLONG_MAX};
    const uintptr_t A = 1ull << 62;
    for (int n : sizes) for (int t : sizes) for (int d : sizes) for (long long s : strides)
        for (int dt : {0, 1, 3}) {
            const gdn_dtype_t e = (gdn_dtype_t)dt;
            gdn_decode_runs(P(A), P(A), P(A), F(A), F(A), F(1 << 30), I(A), I(A), P(16), n, t, d, d, 128, 128,
                            n, s, s, s, s, s, e, 4u, nullptr);
            gdn_decode_runs(P(A), P(A), P(A), F(A), F(A), F(1 << 30), nullptr, nullptr, P(16), t, t, 1, d, n, d,
                            INT_MAX, s, s, s, s, s, e, 0u, nullptr);
            void *y[3] = {P(16), P(1 << 20), P(1 << 25)};
            const long long ys[3] = {s, s, 1024};
            const int begin[4] = {0, 1, d > 2 ? 2 : d, d};
            for (int parts : {INT_MIN, 0, 1, 3, 4}) {
                const int b1[2] = {0, d};
                gdn_short_conv_fwd(P(A), P(A + 64), nullptr, P(1 << 30), I(A), I(A), y, ys, parts == 1 ? b1 : begin,
                                   parts, n, t, d, 4, n, s, 1, e, e, nullptr);
                gdn_short_conv_bwd(y, ys, parts == 1 ? b1 : begin, parts, P(A), P(A + 64), nullptr, I(A), P(1ull << 40),
                                   F(1ull << 41), F(1ull << 42), n, t, d, 4, s, 1, e, GDN_F32, P(1ull << 50),
                                   ~size_t(0), nullptr);
            }
            gdn_short_conv_bwd_workspace_size(t, d, n);
            gdn_rms_norm_fwd(P(A), P(A + 64), P(A), P(A), P(16), F(1 << 30), P(1ull << 40), n, t, d, 128, s, s, s,
                             1e-6f, e, e, nullptr);
            gdn_rms_norm_bwd(P(A), P(A), P(A + 64), P(A), P(A), P(16), F(1ull << 40), P(1ull << 50), n, t, d, s, s, s, s,
                             0.f, e, e, P(1ull << 56), ~size_t(0), nullptr);
            gdn_rms_norm_bwd_workspace_size(n, t, d);
        }
    if (!g_calls) { std::printf("nothing passed the checks\n"); return 1; }
    std::printf("sanitized layer ABI ok\n");
    return 0;
}
"""


def test_entry_points_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    """The argument checks with extreme sizes, strides and pointers: no overflow in them."""
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(CUDA_INC):
        pytest.skip("no g++ or no CUDA headers")
    (tmp_path / "stubs.cpp").write_text(STUBS)
    (tmp_path / "harness.cpp").write_text(HARNESS)
    exe = tmp_path / "layer_harness"
    build = subprocess.run(
        [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=undefined", "-I", CUDA_INC, "-I", CSRC,
         "-I", os.path.join(ROOT, "include"), "-x", "c++", os.path.join(CSRC, "layer_api.cu"),
         "-x", "c++", str(tmp_path / "stubs.cpp"), str(tmp_path / "harness.cpp"), "-o", str(exe)],
        capture_output=True, text=True)
    if build.returncode != 0 and "sanitize" in build.stderr:
        pytest.skip("compiler without sanitizer runtime")
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and "sanitized layer ABI ok" in run.stdout, \
        (run.stdout + run.stderr)[-3000:]


@pytest.mark.parametrize("given", [None, 16])
def test_what_a_call_allocates_lives_until_the_entry_point_returns(monkeypatch, given):
    # a stand-in for the C entry points looks whether every array that the binding made for
    # the call, the workspace among them, still belongs to someone while it runs
    import weakref

    from gated_delta_rule_130_b200 import binding as b
    made, passed = [], []
    real = torch.Tensor.new_empty

    def new_empty(self, *a, **kw):
        t = real(self, *a, **kw)
        made.append((weakref.ref(t), t.data_ptr()))
        return t

    def entry(*args):
        for alive, ptr in made:
            assert alive() is not None, "an array was given up before the launch"
            passed.append(ptr in args)
        return 0

    class Lib:
        gdn_short_conv_bwd = gdn_rms_norm_bwd = staticmethod(entry)
        gdn_short_conv_bwd_workspace_size = gdn_rms_norm_bwd_workspace_size = staticmethod(lambda *s: 4096)

    monkeypatch.setattr(b, "LIB", Lib)
    monkeypatch.setattr(b, "_cuda", lambda t, name: t.get_device())
    monkeypatch.setattr(b, "_call", lambda dev, f, *args: f(*args, None))
    monkeypatch.setattr(torch.Tensor, "new_empty", new_empty)
    z = torch.zeros
    ws = None if given is None else z(given, dtype=torch.uint8)  # one that is too small
    b.short_conv_bwd(z(4, 8), z(4, 8), z(8, 4), z(8), cu_seqlens=z(2, dtype=torch.int32), workspace=ws)
    assert passed == [True] * 4  # dx, dweight, dbias, workspace
    made.clear()
    passed.clear()
    b.rms_norm_bwd(z(4, 8), z(4, 8), z(8), workspace=ws)
    assert passed == [True] * 3  # dx, dweight, workspace


def test_outputs_of_one_call_are_arrays_of_their_own():
    # q, k and v (or dx and dgate) share neither memory, so that keeping one does not keep the
    # others, nor a version counter, so that each may be changed in place beside the others
    from gated_delta_rule_130_b200 import binding as b
    scale = torch.ones(8, requires_grad=True)
    for shapes in ([(4, 8)] * 3, [(4, 8), (4, 16)], [(4, 8)]):
        made = b._like_parts(torch.zeros(2, dtype=torch.bfloat16), shapes)
        assert [t.shape for t in made] == shapes and all(t.dtype == torch.bfloat16 for t in made)
        assert all(t._base is None for t in made)
        assert len({t.untyped_storage().data_ptr() for t in made}) == len(made)
        made[0].mul_(scale)
        assert all(t._version == 0 and not t.requires_grad for t in made[1:])
