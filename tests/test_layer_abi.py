"""The layer library's ABI and refusals: what its headers declare is what the library exports and the binding binds, and
calls that the documentation rules out return an error before anything is launched.  Needs no GPU."""
import ctypes
import glob
import math
import os
import re
import subprocess

import pytest
import torch

import linear_attention_recurrent_decode_b200 as kda
from linear_attention_recurrent_decode_b200 import build, layer
from tests import layer_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = sorted(glob.glob(os.path.join(ROOT, "include", "layer", "*.h")))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.layer_library()


def declared_functions():
    names = set()
    for path in HEADERS:
        names |= {re.findall(r"\w+", m)[-1] for m in re.findall(r"^KDA_API([^(;]*)\(", open(path).read(), re.M)}
    return names


def test_binding_and_library_match_the_headers(lib):
    names = declared_functions()
    assert names == set(kda.LAYER_SYMBOLS)
    out = os.popen(f"nm -D --defined-only {kda.LAYER_LIBRARY_PATH}").read()
    syms = {line.split()[-1] for line in out.splitlines() if line.split()[1] in ("T", "t")}
    assert {s for s in syms if s.startswith("kda_")} == names
    for name in ("kda_scan", "kda_scan_backward", "kda_qk_norm_rope", "kda_qk_norm_rope_backward"):
        assert callable(getattr(kda, name)) and name in kda.__all__


@pytest.mark.parametrize("struct,mirror", [("kda_scan_args", layer.ScanArgs), ("kda_scan_grads", layer.ScanGrads),
                                           ("kda_qk_tensor", layer.QkTensor), ("kda_qk_args", layer.QkArgs)])
def test_structures_have_the_c_layout(struct, mirror, tmp_path):
    src = tmp_path / "s.c"
    fields = [f[0] for f in mirror._fields_]
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n" + "".join(f'#include "{h}"\n' for h in HEADERS) +
                   "int main(void) {\n" + f'printf("%zu", sizeof({struct}));\n' +
                   "".join(f'printf(" %zu", offsetof({struct}, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def test_workspace_sizes(lib):
    f = lib.kda_scan_workspace_bytes
    assert f(0, 0, 1, 1, 128, 128, 0) == 0
    assert f(1, 0, 1, 1, 128, 128, 0) > 0  # packed: a slot a sequence
    assert f(1, 0, 0, 1, 128, 128, 0) >= 0
    for bad in ((-1, 1, 1, 1, 128, 128, 0), (1, -1, 1, 1, 128, 128, 0), (1, 1, 1, 0, 128, 128, 0), (1, 1, 1, 1, 64, 128, 0),
                (1, 1, 1, 1, 128, 256, 0), (1 << 40, 1 << 40, 0, 1 << 20, 128, 128, 1)):
        assert f(*bad) == -1
    assert f(4, 1000, 1, 8, 128, 128, 1) > f(4, 1000, 1, 8, 128, 128, 0)
    # every packing of 4 sequences into 1000 rows fits what one size gives for it
    assert f(4, 1000, 1, 8, 128, 128, 0) >= f(1, 1000, 0, 8, 128, 128, 0)
    with pytest.raises(ValueError):
        kda.scan_workspace_bytes(10, 1, 2, 64, 128)
    g = lib.kda_qk_workspace_bytes
    assert g(128) > 0 and g(256) == 2 * g(128)
    assert g(0) == g(7) == g(12) == g(264) == -1


def test_workspace_holds_segments_only_where_they_help(lib):
    """One sequence of 8192 tokens: cut into segments up to 40 heads; with 48, two walks of them would take longer."""
    f = lib.kda_scan_workspace_bytes
    for training in (0, 1):
        record = f(1, 64, 0, 1, 128, 128, training) - 256
        for heads, cut in ((8, True), (32, True), (40, True), (48, False), (64, False), (72, False), (80, False)):
            for packed in (0, 1):
                records = 256 + (128 + packed) * heads * record
                assert (f(1, 8192, packed, heads, 128, 128, training) > records) == cut, heads
                assert f(1, 8192, packed, heads, 128, 128, training) >= records


# ------------------------------------------------------------------------------------------------------ C refusals
BASE = 1 << 32  # fake device addresses, far apart; nothing is dereferenced on the host


def scan_args(**kw):
    a = layer.ScanArgs()
    N, T, H = 2, 100, 3
    a.q, a.k, a.v, a.g, a.beta = (BASE + (i << 28) for i in range(5))
    a.q_row_stride = a.k_row_stride = a.v_row_stride = a.g_row_stride = a.out_row_stride = H * 128
    a.beta_row_stride = H
    a.cu_seqlens, a.initial_state, a.final_state, a.out = (BASE + (i << 28) for i in range(5, 9))
    a.workspace, a.workspace_bytes = BASE + (10 << 28), 1 << 28
    a.N, a.T, a.HV, a.K, a.V, a.scale = N, T, H, 128, 128, 0.1
    for name, value in kw.items():
        setattr(a, name, value)
    return a


def scan_grads(**kw):
    d = layer.ScanGrads()
    d.d_out, d.d_final_state, d.dq, d.dk, d.dv, d.dg, d.dbeta, d.d_initial_state = (BASE + (i << 28) for i in range(12, 20))
    for n in ("d_out", "dq", "dk", "dv", "dg"):
        setattr(d, n + "_row_stride", 3 * 128)
    d.dbeta_row_stride = 3
    for name, value in kw.items():
        setattr(d, name, value)
    return d


def valid(status):
    """A call that passes every check: launched, or refused for want of a GPU."""
    return status == (kda.KDA_OK if torch.cuda.is_available() else kda.KDA_ERR_DEVICE)


A, M, U, I = kda.KDA_ERR_ALIAS, kda.KDA_ERR_MISALIGNED, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), I), (dict(T=-1), I), (dict(HV=0), U), (dict(K=64), U), (dict(V=256), U), (dict(num_slots=-1), I),
    (dict(q=None), I), (dict(k=None), I), (dict(v=None), I), (dict(g=None), I), (dict(beta=None), I), (dict(out=None), I),
    (dict(q=BASE + 2), M), (dict(v=BASE + (2 << 28) + 8), M), (dict(g=BASE + (3 << 28) + 2), M), (dict(out=BASE + (8 << 28) + 4), M),
    (dict(initial_state=BASE + (6 << 28) + 4), M), (dict(cu_seqlens=BASE + (5 << 28) + 2), M), (dict(workspace=BASE + (10 << 28) + 8), M),
    (dict(q_row_stride=3 * 128 - 8), I), (dict(beta_row_stride=2), I), (dict(k_row_stride=3 * 128 + 4), M),
    (dict(workspace=None), I), (dict(workspace_bytes=1000), I), (dict(slot_idx=BASE + (11 << 28), num_slots=0), I),
    (dict(out=BASE), A), (dict(out=BASE + (1 << 28) + 4096), A), (dict(final_state=BASE), A), (dict(workspace=BASE), A),
    (dict(out=BASE + (7 << 28)), A), (dict(final_state=BASE + (6 << 28) + 16), A), (dict(out=BASE + (10 << 28)), A),
    (dict(T=1 << 62), U), (dict(slot_idx=BASE + (11 << 28), num_slots=1 << 62), U), (dict(N=1 << 62, cu_seqlens=None), U), (dict(T=1 << 32, N=1), U),
])
def test_scan_refusals(lib, kw, status):
    assert lib.kda_scan(ctypes.byref(scan_args(**kw)), None) == status


def test_scan_checks_pass_and_nothing_to_do(lib):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a GPU")
    for kw in (dict(), dict(cu_seqlens=None), dict(initial_state=None), dict(final_state=None),
               dict(final_state=BASE + (6 << 28)),                      # a state updated in place
               dict(q_row_stride=1152, k_row_stride=1152, v_row_stride=1152, k=BASE + 768, v=BASE + 1536)):
        assert valid(lib.kda_scan(ctypes.byref(scan_args(**kw)), None)), kw
    assert lib.kda_scan(ctypes.byref(scan_args(N=0)), None) == kda.KDA_OK
    assert lib.kda_scan(None, None) == I
    assert valid(lib.kda_scan_backward(ctypes.byref(scan_args()), ctypes.byref(scan_grads()), None))
    packed = dict(dq_row_stride=1152, dk_row_stride=1152, dv_row_stride=1152, dk=BASE + (14 << 28) + 768, dv=BASE + (14 << 28) + 1536)
    assert valid(lib.kda_scan_backward(ctypes.byref(scan_args()), ctypes.byref(scan_grads(**packed)), None))


@pytest.mark.parametrize("kw,status", [
    (dict(d_out=None), I), (dict(dq=None), I), (dict(dk=None), I), (dict(dv=None), I), (dict(dg=None), I), (dict(dbeta=None), I),
    (dict(dq=BASE), A), (dict(dk=BASE + (14 << 28)), A), (dict(dv=BASE + (12 << 28)), A), (dict(dg=BASE + (10 << 28)), A),
    (dict(d_initial_state=BASE + (6 << 28)), A), (dict(d_initial_state=BASE + (13 << 28)), A), (dict(d_out=BASE + (12 << 28) + 2), M),
    (dict(dq_row_stride=380), I), (dict(dbeta=BASE + (18 << 28) + 1), M), (dict(d_final_state=BASE + (13 << 28) + 8), M),
])
def test_scan_backward_refusals(lib, kw, status):
    assert lib.kda_scan_backward(ctypes.byref(scan_args()), ctypes.byref(scan_grads(**kw)), None) == status


def test_scan_backward_refuses_slots_and_small_workspaces(lib):
    d = scan_grads()
    assert lib.kda_scan_backward(ctypes.byref(scan_args(slot_idx=BASE + (11 << 28), num_slots=4)), ctypes.byref(d), None) == I
    assert lib.kda_scan_backward(None, ctypes.byref(d), None) == I
    assert lib.kda_scan_backward(ctypes.byref(scan_args()), None, None) == I
    small = lib.kda_scan_workspace_bytes(2, 100, 1, 3, 128, 128, 0)  # the forward pass's is too small
    assert lib.kda_scan_backward(ctypes.byref(scan_args(workspace_bytes=small)), ctypes.byref(d), None) == I
    assert lib.kda_scan(ctypes.byref(scan_args(workspace_bytes=small, save=1)), None) == I


def qk_args(**kw):
    a = layer.QkArgs()
    a.rows, a.D, a.rot, a.norm, a.eps, a.rope_scale = 10, 64, 32, 1, 1e-6, 1.0
    a.positions, a.inv_freq = BASE + (1 << 20), BASE + (2 << 20)
    a.workspace, a.workspace_bytes = BASE + (3 << 20), 4096 * 64
    for i, t in enumerate((a.q, a.k)):
        at = BASE + ((16 + 16 * i) << 20)
        t.heads = 2
        t.x, t.y, t.dy, t.dx, t.weight, t.dweight = (at + (j << 20) for j in range(6))
        t.x_row_stride = t.y_row_stride = t.dy_row_stride = t.dx_row_stride = 128
    for name, value in kw.items():
        o = a
        *path, last = name.split("__")
        for part in path:
            o = getattr(o, part)
        setattr(o, last, value)
    return a


Q0, K0 = BASE + (16 << 20), BASE + (32 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), I), (dict(norm=3), I), (dict(norm=-1), I), (dict(D=12), U), (dict(D=0), U), (dict(D=264), U), (dict(rot=8), U),
    (dict(rot=80), U), (dict(rot=-16), U), (dict(q__heads=-1), I), (dict(k__heads=5000), U), (dict(q__x=None), I), (dict(k__y=None), I),
    (dict(q__x=Q0 + 2), M), (dict(k__y_row_stride=132), M), (dict(q__x_row_stride=120), I), (dict(q__weight=Q0 + (4 << 20) + 4), M),
    (dict(norm=0), I),                                             # a weight without a norm
    (dict(positions=None), I), (dict(inv_freq=None), I), (dict(inv_freq=BASE + 4), M), (dict(positions=BASE + 4, positions_64=1), M),
    (dict(q__y=K0), A), (dict(q__y=Q0 + 256), A), (dict(k__y=Q0 + (1 << 20)), A), (dict(q__y=Q0 + (4 << 20)), A),
    (dict(q__y=BASE + (1 << 20)), A), (dict(q__y=Q0, q__y_row_stride=256), A), (dict(rows=1 << 60), U),
])
def test_qk_refusals(lib, kw, status):
    assert lib.kda_qk_norm_rope(ctypes.byref(qk_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q__dy=None), I), (dict(k__dx=None), I), (dict(q__x=None), I), (dict(q__dx=Q0), A), (dict(q__dx=Q0 + (2 << 20) + 256), A),
    (dict(q__dweight=Q0 + (3 << 20)), A), (dict(q__dweight=K0 + (5 << 20)), A), (dict(q__weight=None), I), (dict(workspace=None), I),
    (dict(workspace_bytes=100), I), (dict(workspace=BASE + (3 << 20) + 4), M), (dict(workspace=Q0), A),
    (dict(q__dweight=Q0 + (5 << 20) + 2), M),
])
def test_qk_backward_refusals(lib, kw, status):
    assert lib.kda_qk_norm_rope_backward(ctypes.byref(qk_args(**kw)), None) == status


def test_qk_checks_pass_and_nothing_to_do(lib):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a GPU")
    for kw in (dict(), dict(k__heads=0, k__x=None, k__y=None), dict(q__y=Q0), dict(rot=0, positions=None, inv_freq=None),
               dict(norm=0, q__weight=None, k__weight=None)):
        assert valid(lib.kda_qk_norm_rope(ctypes.byref(qk_args(**kw)), None)), kw
    for kw in (dict(), dict(q__dx=Q0 + (2 << 20)), dict(q__dweight=None, k__dweight=None, workspace=None, workspace_bytes=0),
               dict(norm=0, q__weight=None, k__weight=None, q__dweight=None, k__dweight=None, q__x=None, k__x=None)):
        assert valid(lib.kda_qk_norm_rope_backward(ctypes.byref(qk_args(**kw)), None)), kw
    assert lib.kda_qk_norm_rope(ctypes.byref(qk_args(rows=0)), None) == kda.KDA_OK
    assert lib.kda_qk_norm_rope(ctypes.byref(qk_args(q__heads=0, k__heads=0)), None) == kda.KDA_OK
    assert lib.kda_qk_norm_rope(None, None) == I and lib.kda_qk_norm_rope_backward(None, None) == I


# -------------------------------------------------------------------------------------------------- binding refusals
def test_binding_refuses_cpu_tensors():
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    g, beta, cu = torch.zeros(4, 2, 128), torch.zeros(4, 2), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_scan(q, q, q, g, beta, cu_seqlens=cu)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_scan(q[None], q[None], q[None], g[None], beta[None])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_scan_backward(q, q, q, q, g, beta, cu_seqlens=cu)
    with pytest.raises(ValueError, match="workspace"):
        kda.kda_scan_backward(q, q, q, q, g, beta, cu_seqlens=cu, saved=True)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_qk_norm_rope(q)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_qk_norm_rope_backward(q, None, q)
    with pytest.raises(ValueError, match="norm"):
        kda.kda_qk_norm_rope(q, norm="layer")
    with pytest.raises(TypeError):
        kda.kda_qk_norm_rope(q[0, 0])


# -------------------------------------------------------------------------------------------------- frequencies
def test_rope_frequencies():
    f, s = kda.rope_frequencies(64)
    assert f.dtype == torch.float64 and f.shape == (32,) and s == 1.0
    for i in (0, 1, 31):
        assert math.isclose(float(f[i]), 10000.0 ** (-2 * i / 64), rel_tol=1e-14)
    g, s = kda.rope_frequencies(64, 500000.0, factor=8.0)
    assert s == 1.0 and torch.allclose(g, kda.rope_frequencies(64, 500000.0)[0] / 8, rtol=1e-15, atol=0)
    y, s = kda.rope_frequencies(128, factor=16.0, trained_context=4096)
    base = kda.rope_frequencies(128)[0]
    turns = 4096 * base / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(16.0) + 1)
    assert torch.equal(y[turns > 33], base[turns > 33])                              # fast pairs stay
    assert torch.allclose(y[turns < 0.9], base[turns < 0.9] / 16, rtol=1e-15, atol=0)  # slow ones are divided
    assert bool((y <= base).all()) and bool((y >= base / 16 * (1 - 1e-15)).all()) and bool((y[1:] < y[:-1]).all())
    assert kda.rope_frequencies(0)[0].numel() == 0
    for bad in (dict(rot=3), dict(rot=-2), dict(rot=4, factor=0.5), dict(rot=4, base=1.0)):
        with pytest.raises(ValueError):
            kda.rope_frequencies(**bad)


# -------------------------------------------------------------------------------------------------- the reference itself
def test_reference_gradients_against_differences():
    torch.manual_seed(3)
    cu, H, D = [0, 3, 3, 8], 2, 4
    x = [torch.randn(8, H, D, dtype=torch.float64) * 0.5 for _ in range(4)] + [torch.rand(8, H, dtype=torch.float64),
                                                                              torch.randn(3, H, D, D, dtype=torch.float64)]
    x[3] = -x[3].abs()
    for t in x:
        t.requires_grad_()
    assert torch.autograd.gradcheck(lambda *a: ref.scan(*a, cu, 0.7), x)
    y, w = torch.randn(3, 2, 8, dtype=torch.float64, requires_grad=True), torch.randn(8, dtype=torch.float64, requires_grad=True)
    pos, f = torch.tensor([0, 5, -9]), kda.rope_frequencies(4)[0]
    for norm in ("l2", "rms"):
        for inter in (False, True):
            assert torch.autograd.gradcheck(lambda a, b: ref.qk(a, norm, 1e-6, b, pos, f, inter, 1.3), (y, w))
