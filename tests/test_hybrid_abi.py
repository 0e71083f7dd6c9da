"""Refusals of the hybrid token mixers: every bad argument returns its status before
anything is enqueued, and the binding refuses tensors that the kernels cannot read
(no GPU needed)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda.h")
FAKE = 0x7f0000000000  # never dereferenced: validation fails before any launch
NULL, SHAPE, DTYPE, ALIGN, SEQLENS, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 6, 8


def _kda():
    import serving_kda_chunked_gated_gb300.kda as kda
    return kda


def test_struct_layout_matches_c(tmp_path):
    kda = _kda()
    structs = [("kda_gdn_prefill_args", kda.GdnPrefillArgs), ("kda_gdn_decode_args", kda.GdnDecodeArgs),
               ("kda_qk_norm_rope_args", kda.QkNormRopeArgs), ("kda_window_prefill_args", kda.WindowPrefillArgs),
               ("kda_window_decode_args", kda.WindowDecodeArgs)]
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void){"]
    want = []
    for cname, py in structs:
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(py))
        for f in py._fields_:
            lines.append(f'printf("%zu\\n", offsetof({cname}, {f[0]}));')
            want.append(getattr(py, f[0]).offset)
    (tmp_path / "layout.c").write_text("\n".join(lines + ["return 0;}"]))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", str(tmp_path / "layout.c"), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def _fill(a, **kw):
    for f, typ in a._fields_:
        if typ is ctypes.c_void_p:
            setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _gdn(cu, **kw):
    a = _fill(_kda().GdnPrefillArgs(), num_seqs=len(cu) - 1, T_total=int(cu[-1]), Hk=2, Hv=4, dk=128, dv=128,
              cu_seqlens_host=cu.ctypes.data, workspace_bytes=1 << 40, gate_mode=1, scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), NULL), (dict(beta=None), NULL), (dict(A=None), NULL), (dict(cu_seqlens=None), NULL),
    (dict(cu_seqlens_host=None), NULL), (dict(o=None, S_T=None), NULL), (dict(Hk=3), SHAPE), (dict(Hk=0), SHAPE),
    (dict(Hv=0), SHAPE), (dict(dk=64), SHAPE), (dict(dv=256), SHAPE), (dict(num_seqs=-1), SHAPE),
    (dict(T_total=-1), SHAPE), (dict(qkv_dtype=2), DTYPE), (dict(v=FAKE + 8), ALIGN), (dict(S0=FAKE + 4), ALIGN),
    (dict(T_total=65), SEQLENS), (dict(gate_mode=2), UNSUPPORTED), (dict(Hk=1 << 28, Hv=1 << 28, num_seqs=1), SHAPE),
])
def test_gdn_prefill_refusals(kda_lib, kw, expect):
    cu = np.array([0, 64], dtype=np.int32)
    a = _gdn(cu, **kw)
    assert kda_lib.kda_gdn_prefill(ctypes.byref(a), None) == expect
    assert kda_lib.kda_gdn_prefill_recurrent(ctypes.byref(a), None) == expect
    assert kda_lib.kda_gdn_prefill_workspace_size(ctypes.byref(a)) == 0


def test_gdn_prefill_workspace(kda_lib):
    cu = np.array([0, 64, 64, 300], dtype=np.int32)
    a = _gdn(cu)
    need = kda_lib.kda_gdn_prefill_workspace_size(ctypes.byref(a))
    assert need >= 4
    for kw, expect in ((dict(workspace=None), WORKSPACE), (dict(workspace_bytes=need - 1), WORKSPACE),
                       (dict(workspace=FAKE + 8), ALIGN)):
        assert kda_lib.kda_gdn_prefill(ctypes.byref(_gdn(cu, **kw)), None) == expect
    assert kda_lib.kda_gdn_prefill_workspace_size(ctypes.byref(_gdn(cu, qkv_dtype=1))) == 0     # float32 needs none
    for bad in ([0, 40, 30, 64], [1, 20, 30, 64]):
        b = np.array(bad, dtype=np.int32)
        assert kda_lib.kda_gdn_prefill(ctypes.byref(_gdn(b)), None) == SEQLENS
    assert kda_lib.kda_gdn_prefill(None, None) == NULL
    empty = np.array([0], dtype=np.int32)
    assert kda_lib.kda_gdn_prefill(ctypes.byref(_gdn(empty)), None) == 0       # no sequences: nothing to do


@pytest.mark.parametrize("kw,expect", [
    (dict(state=None), NULL), (dict(o=None), NULL), (dict(z=None), NULL), (dict(Hk=3), SHAPE), (dict(N=-1), SHAPE),
    (dict(dk=64), SHAPE), (dict(slots=None, num_slots=3), SHAPE), (dict(state=FAKE + 4), ALIGN),
    (dict(slots=FAKE + 4), ALIGN), (dict(gate_mode=-1), UNSUPPORTED), (dict(N=1 << 30, num_slots=1 << 30), SHAPE),
])
def test_gdn_decode_refusals(kda_lib, kw, expect):
    a = _fill(_kda().GdnDecodeArgs(), N=4, Hk=2, Hv=4, dk=128, dv=128, num_slots=4, gate_mode=1, **{})
    for k, v in kw.items():
        setattr(a, k, v)
    assert kda_lib.kda_gdn_decode_step(ctypes.byref(a), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), NULL), (dict(k_out=None), NULL), (dict(cos=None), NULL), (dict(positions=None), NULL),
    (dict(d=12), SHAPE), (dict(d=264), SHAPE), (dict(d=68), SHAPE), (dict(rot=8), SHAPE), (dict(rot=24), SHAPE),
    (dict(rot=144), SHAPE), (dict(Hq=0, Hkv=0), SHAPE), (dict(Hq=-1), SHAPE), (dict(T=-1), SHAPE), (dict(num_pos=-1), SHAPE),
    (dict(q_stride=511), SHAPE), (dict(k_stride=100), SHAPE), (dict(q_stride=516), ALIGN), (dict(k=FAKE + 2), ALIGN),
    (dict(sin=FAKE + 4), ALIGN), (dict(dtype=7), DTYPE), (dict(q_out=FAKE, q_stride=1024), SHAPE),
    (dict(T=1 << 30, Hq=1 << 10, q_stride=1 << 18), SHAPE), (dict(T=1, Hq=1 << 20, q_stride=1 << 27), SHAPE),
])
def test_qk_norm_rope_refusals(kda_lib, kw, expect):
    a = _fill(_kda().QkNormRopeArgs(), T=5, Hq=4, Hkv=2, d=128, rot=128, num_pos=9, q_stride=512, k_stride=256, eps=1e-6,
              q_out=FAKE + (1 << 20), k_out=FAKE + (1 << 21))
    for k, v in kw.items():
        setattr(a, k, v)
    assert kda_lib.kda_qk_norm_rope(ctypes.byref(a), None) == expect


def _window(cu, cuk, **kw):
    a = _fill(_kda().WindowPrefillArgs(), num_seqs=len(cu) - 1, T_total=int(cu[-1]), Tk_total=int(cuk[-1]), Hq=4, Hkv=2,
              d=64, window=8, sinks=2, q_stride=256, k_stride=128, v_stride=128, scale=0.125,
              cu_seqlens_host=cu.ctypes.data, cu_seqlens_k_host=cuk.ctypes.data, num_slots=4, cache_rows=10)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


WINDOW_BAD = [
    (dict(q=None), NULL), (dict(v=None), NULL), (dict(o=None), NULL), (dict(v_cache=None), NULL), (dict(Hkv=3), SHAPE),
    (dict(d=96), SHAPE), (dict(window=0), SHAPE), (dict(sinks=-1), SHAPE), (dict(window=2 ** 31 - 1, sinks=1), SHAPE),
    (dict(dtype=1), DTYPE), (dict(k_stride=127), SHAPE), (dict(q_stride=260), ALIGN), (dict(k=FAKE + 4), ALIGN),
    (dict(k_cache=FAKE + 8), ALIGN), (dict(scale=float("nan")), SHAPE), (dict(cache_rows=9), SHAPE),
    (dict(slots=None, num_slots=1), SHAPE), (dict(num_slots=-1), SHAPE),
]


@pytest.mark.parametrize("kw,expect", WINDOW_BAD + [
    (dict(cu_seqlens=None), NULL), (dict(cu_seqlens_k_host=None), NULL), (dict(lse=FAKE + 4), ALIGN),
    (dict(T_total=9), SEQLENS), (dict(Tk_total=9), SEQLENS), (dict(num_seqs=-1), SHAPE),
])
def test_window_prefill_refusals(kda_lib, kw, expect):
    cu = np.array([0, 3, 8], dtype=np.int32)
    a = _window(cu, cu, **kw)
    assert kda_lib.kda_window_prefill(ctypes.byref(a), None) == expect


def test_window_prefill_needs_a_key_for_each_query(kda_lib):
    cu, cuk = np.array([0, 3, 8], dtype=np.int32), np.array([0, 2, 9], dtype=np.int32)
    assert kda_lib.kda_window_prefill(ctypes.byref(_window(cu, cuk)), None) == SEQLENS


@pytest.mark.parametrize("kw,expect", WINDOW_BAD + [(dict(k_cache=None), NULL), (dict(positions=None), NULL),
                                                    (dict(N=-1), SHAPE), (dict(positions=FAKE + 4), ALIGN)])
def test_window_decode_refusals(kda_lib, kw, expect):
    a = _fill(_kda().WindowDecodeArgs(), N=2, Hq=4, Hkv=2, d=64, window=8, sinks=2, q_stride=256, k_stride=128,
              v_stride=128, scale=0.125, num_slots=4, cache_rows=10)
    for k, v in kw.items():
        setattr(a, k, v)
    assert kda_lib.kda_window_decode(ctypes.byref(a), None) == expect


def test_binding_refuses_what_the_kernels_cannot_read():
    """CPU tensors, wrong types, shapes and strides stop in the binding."""
    kda = _kda()
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(kda.KDAError, match="CUDA tensor"):
        kda.gdn_prefill(x, x, x, x, x, x)
    with pytest.raises(kda.KDAError, match="CUDA tensor"):
        kda.window_decode(x, x, x, x, x, x, 4)
    dev = x.device
    assert kda._dense("x", x, (4, 2, 128), torch.bfloat16, dev) == x.data_ptr()
    assert kda._dense("x", None, (4,), torch.int32, dev) is None
    for shape, dtype, t in (((4, 2, 64), torch.bfloat16, x), ((4, 2, 128), torch.float32, x), ((4, 256), torch.bfloat16, x),
                            ((4, 2, 64), torch.bfloat16, x[..., ::2]), ((2, 4, 128), torch.bfloat16, x.transpose(0, 1))):
        with pytest.raises(kda.KDAError, match="expected a contiguous"):
            kda._dense("x", t, shape, dtype, dev)
    packed = torch.zeros(4, 6 * 128, dtype=torch.bfloat16)
    assert kda._heads("q", packed[:, :256].unflatten(1, (2, 128)), (4, 2, 128), torch.bfloat16, dev)[1] == 768
    with pytest.raises(kda.KDAError, match="must be dense"):
        kda._heads("q", packed.unflatten(1, (6, 128))[:, ::2], (4, 3, 128), torch.bfloat16, dev)
    with pytest.raises(kda.KDAError, match="gate must be"):
        kda._gate_code("relu")
    with pytest.raises(kda.KDAError, match="host copy"):
        kda._cu_pair(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0, dev)
    with pytest.raises(kda.KDAError, match="given together"):
        kda._caches(x, None, 2, 128, dev)


def test_window_prefill_error_word(kda_lib):
    """A caller's own error word: checked like every pointer."""
    kda = _kda()
    cu = np.array([0, 3, 8], dtype=np.int32)
    assert kda_lib.kda_window_prefill(ctypes.byref(_window(cu, cu, error=FAKE + 4)), None) == ALIGN
    assert ("error", ctypes.c_void_p) in kda.WindowPrefillArgs._fields_


def test_sizes_past_32_bits_are_refused():
    """A window of 2^32 + 8 is not a window of 8, nor a table of 2^32 + 5 positions one of 5 (meta tensors
    stand for the GPU's: the binding stops before it looks at their memory)."""
    kda = _kda()

    class Cuda(torch.Tensor):
        is_cuda = True

    x = lambda *s, d=torch.bfloat16: torch.empty(*s, dtype=d, device="meta").as_subclass(Cuda)       # noqa: E731
    cu = torch.tensor([0, 4], dtype=torch.int32)
    cud = x(2, d=torch.int32)
    for big in (2 ** 32 + 8, 2 ** 31, -2 ** 32 + 8):
        for kw in (dict(window=big), dict(window=8, sinks=big)):
            with pytest.raises(kda.KDAError, match="32 bits"):
                kda.window_prefill(x(4, 2, 64), x(4, 1, 64), x(4, 1, 64), cu_seqlens=cud, cu_seqlens_host=cu, **kw)
            with pytest.raises(kda.KDAError, match="32 bits"):
                kda.window_decode(x(4, 2, 64), x(4, 1, 64), x(4, 1, 64), x(4, 9, 1, 64), x(4, 9, 1, 64), x(4, d=torch.int32), **kw)
    table = torch.empty(1, 8, device="meta").expand(2 ** 32 + 5, 8).as_subclass(Cuda)
    with pytest.raises(kda.KDAError, match="32 bits"):
        kda.qk_norm_rope(x(4, 2, 64), x(4, 1, 64), table, table, x(4, d=torch.int32))
