"""Host-side checks of the C ABI (no GPU work): the library loads, exports
every function include/mbok.h declares, sizes are right, and argument errors
are reported before anything is launched."""
import ctypes
import os
import re

import pytest

from helpers import ensure_built

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mbok.h")

FAKE = 1 << 20          # a 16-byte aligned non-null address; never dereferenced
FAKE_ODD = FAKE + 1     # misaligned


@pytest.fixture(scope="module")
def L():
    ensure_built()
    import boolean_weight_matmul_b200 as mb
    return mb.lib()


def header_functions():
    text = open(HEADER).read()
    return re.findall(r"^\s*(?:const\s+char\s*\*|int|size_t)\s+(mbok_\w+)\s*\(", text, re.M)


def test_header_declares_the_calls():
    names = set(header_functions())
    for n in ("mbok_pack_bits", "mbok_residual_binarize", "mbok_gemv", "mbok_gemm",
              "mbok_pack_alpha", "mbok_packed_bytes", "mbok_alpha_elems",
              "mbok_gemv_workspace_bytes", "mbok_status_string", "mbok_layout_version"):
        assert n in names


def test_library_exports_every_declared_function(L):
    names = header_functions()
    assert names
    for n in names:
        assert hasattr(L, n), f"{n} declared in include/mbok.h but not exported"


def test_sizes(L):
    assert L.mbok_layout_version() == 1
    assert L.mbok_packed_bytes(3, 4096, 4096) == 512 * 3 * 4096
    assert L.mbok_packed_bytes(1, 13, 384) == 2 * 1 * 384
    assert L.mbok_alpha_elems(3, 4096, 4096) == 4096 * 32 * 3
    assert L.mbok_alpha_elems(2, 13, 256) == 16 * 2 * 2
    assert L.mbok_packed_bytes(0, 8, 128) == 0
    assert L.mbok_packed_bytes(1, 8, 100) == 0
    assert L.mbok_gemv_workspace_bytes(3, 4096, 512, 1) == 0       # one slab: no workspace
    assert L.mbok_gemv_workspace_bytes(3, 4096, 4096, 1) >= 8 * 4096 * 4
    assert L.mbok_gemv_workspace_bytes(3, 4096, 4096, 17) == 0


def test_status_strings(L):
    for s in range(8):
        assert L.mbok_status_string(s).decode() not in ("", "unknown status")
    assert L.mbok_status_string(99).decode() == "unknown status"


def test_gemv_argument_errors(L):
    g = lambda **kw: L.mbok_gemv(*[kw.get(k, v) for k, v in dict(
        packed=FAKE, alpha=FAKE, K=3, M=64, N=1024, group=128, x=FAKE, dt=1, batch=1, y=FAKE,
        ws=FAKE, wsb=1 << 20, stream=None).items()])
    assert g(K=0) == 1 and g(K=5) == 1
    assert g(M=0) == 2 and g(N=100) == 2 and g(N=0) == 2
    assert g(group=64) == 4
    assert g(packed=None) == 1 and g(x=None) == 1 and g(y=None) == 1
    assert g(dt=7) == 1
    assert g(batch=0) == 1 and g(batch=17) == 1
    assert g(x=FAKE_ODD) == 3 and g(packed=FAKE + 4) == 3
    assert g(ws=None) == 6 and g(wsb=16) == 6


def test_gemm_and_pack_argument_errors(L):
    assert L.mbok_read_device_errors(None) == 1
    assert L.mbok_gemm(FAKE, FAKE, 3, 64, 256, 128, FAKE, 0, FAKE, None) == 2
    assert L.mbok_gemm(FAKE, FAKE, 3, 64, 256, 256, FAKE, 8, FAKE, None) == 4
    assert L.mbok_gemm(FAKE, FAKE, 3, 64, 256, 128, FAKE_ODD, 8, FAKE, None) == 3
    assert L.mbok_gemm(None, FAKE, 3, 64, 256, 128, FAKE, 8, FAKE, None) == 1
    assert L.mbok_pack_bits(None, 1, 8, 128, FAKE, None) == 1
    assert L.mbok_pack_bits(FAKE, 1, 8, 130, FAKE, None) == 2
    assert L.mbok_pack_bits(FAKE_ODD, 1, 8, 128, FAKE, None) == 3
    assert L.mbok_pack_alpha(FAKE, 5, 8, 128, FAKE, None) == 1
    assert L.mbok_residual_binarize(FAKE, 8, 128, 2, 64, FAKE, FAKE, None, None) == 4
    assert L.mbok_residual_binarize(FAKE, 8, 128, 2, 128, FAKE, FAKE, FAKE_ODD, None) == 3
    assert L.mbok_residual_binarize(FAKE, 0, 128, 2, 128, FAKE, FAKE, None, None) == 2


def test_binding_refuses_cpu_tensors(L):
    import torch
    import boolean_weight_matmul_b200 as mb
    s = torch.ones(1, 8, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        mb.pack_bits(s, 1, 8, 128, torch.empty(64, dtype=torch.int32))


def test_gemv_kernel_choice(L):
    import boolean_weight_matmul_b200 as mb
    assert L.mbok_gemv_set_kernel(-1) == 1 and L.mbok_gemv_set_kernel(5) == 1
    for k in (mb.GEMV_LOOKUP, mb.GEMV_TENSOR, mb.GEMV_LOOKUP_SLABS, mb.GEMV_LOOKUP_ROWS, mb.GEMV_AUTO):
        assert L.mbok_gemv_set_kernel(k) == 0
    with mb.gemv_kernel(mb.GEMV_TENSOR):
        pass
    with pytest.raises(mb.MbokError):
        mb.gemv_set_kernel(7)


def test_gemv_static_weights_switch(L):
    assert L.mbok_gemv_set_static_weights(2) == 1 and L.mbok_gemv_set_static_weights(-1) == 1
    assert L.mbok_gemv_set_static_weights(0) == 0
    assert L.mbok_gemv_set_static_weights(1) == 0      # the default


def test_gemv_svid_argument_errors(L):
    g = lambda **kw: L.mbok_gemv_svid(*[kw.get(k, v) for k, v in dict(
        packed=FAKE, s_in=FAKE, s_out=FAKE, K=3, M=64, N=1024, x=FAKE, dt=1, batch=1, y=FAKE,
        ws=FAKE, wsb=1 << 20, stream=None).items()])
    assert g(K=0) == 1 and g(K=5) == 1
    assert g(M=0) == 2 and g(N=100) == 2
    assert g(s_in=None) == 1 and g(s_out=None) == 1 and g(x=None) == 1
    assert g(batch=0) == 1 and g(batch=17) == 1 and g(dt=5) == 1
    assert g(s_in=FAKE + 8) == 3 and g(s_out=FAKE_ODD) == 3
    assert g(ws=None) == 6 and g(wsb=16) == 6
    assert L.mbok_gemv_svid_workspace_bytes(3, 4096, 4096, 1) > L.mbok_gemv_workspace_bytes(3, 4096, 4096, 1)
    assert L.mbok_gemv_svid_workspace_bytes(1, 4096, 512, 1) == 0


def test_refit_argument_errors(L):
    assert L.mbok_refit_alpha(FAKE, FAKE, 3, 64, 256, 64, FAKE, None) == 4
    assert L.mbok_refit_alpha(None, FAKE, 3, 64, 256, 128, FAKE, None) == 1
    assert L.mbok_refit_alpha(FAKE_ODD, FAKE, 3, 64, 256, 128, FAKE, None) == 3
    assert L.mbok_refit_alpha(FAKE, FAKE, 0, 64, 256, 128, FAKE, None) == 1
    assert L.mbok_refit_alpha(FAKE, FAKE, 3, 64, 200, 128, FAKE, None) == 2


def test_svid_binarize_argument_errors(L):
    g = lambda **kw: L.mbok_svid_binarize(*[kw.get(k, v) for k, v in dict(
        W=FAKE, M=64, N=256, K=3, iters=6, packed=FAKE, s_in=FAKE, s_out=FAKE, R=FAKE, ws=FAKE,
        wsb=1 << 24, stream=None).items()])
    assert g(K=0) == 1 and g(iters=0) == 1 and g(W=None) == 1 and g(R=None) == 1
    assert g(N=100) == 2 and g(M=0) == 2
    assert g(W=FAKE_ODD) == 3 and g(R=FAKE + 4) == 3
    assert g(ws=None) == 6 and g(wsb=16) == 6
    assert L.mbok_svid_workspace_bytes(64, 256) >= (64 + 2 * 256 + 256) * 4


def test_wait_timeout_check_argument_errors(L):
    assert L.mbok_check_wait_timeout(0, None) == 1
    assert L.mbok_check_wait_timeout(2000000, None) == 1


def test_pointer_marshalling_checks_device(monkeypatch):
    # The binding passes raw device pointers to kernels launched on the
    # current device, so it refuses CPU, non-contiguous and other-device
    # tensors before anything reaches the library.  Stand-in tensors keep this
    # a host-only test.
    import types
    import torch
    import boolean_weight_matmul_b200 as mb

    class Fake:
        def __init__(self, dev, contiguous=True, cuda=True, ptr=0x1000):
            self.is_cuda = cuda
            self.device = types.SimpleNamespace(index=dev, type="cuda" if cuda else "cpu")
            self._c = contiguous
            self._p = ptr

        def is_contiguous(self):
            return self._c

        def data_ptr(self):
            return self._p

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert mb._ptrs(Fake(1, ptr=16), None, 7) == [16, None, 7]
    with pytest.raises(ValueError, match="current device"):
        mb._ptrs(Fake(1), Fake(0))
    with pytest.raises(ValueError, match="CUDA tensors only"):
        mb._ptrs(Fake(None, cuda=False))
    with pytest.raises(ValueError, match="contiguous"):
        mb._ptrs(Fake(1, contiguous=False))
    with pytest.raises(ValueError, match="CUDA tensors only"):
        mb.gemv(torch.zeros(4, dtype=torch.int32), None, 1, 8, 128, 128, None, mb.BF16, 1, None, None)


def test_gemv_multi_sizes_and_argument_errors(L):
    # mbok_gemv_multi: several matrices sharing x, each with its own K and M.
    # Sizes and argument errors are host-side (nothing launches on an error).
    import ctypes
    import boolean_weight_matmul_b200 as mb
    O = lambda M: (M + 7) // 8
    # one region of [N/512 slabs][O_s * 8] fp32 partials per matrix
    assert mb.gemv_multi_workspace_bytes([4, 2, 3], [5120, 136, 77], 5120) == \
        10 * 4 * 8 * (O(5120) + O(136) + O(77))
    assert mb.gemv_multi_workspace_bytes([4, 2], [64, 64], 512) == 0          # one slab: no workspace
    assert mb.gemv_multi_workspace_bytes([5], [8], 1024) == 0                 # K out of range
    assert mb.gemv_multi_workspace_bytes([1] * 9, [8] * 9, 1024) == 0         # more than 8 matrices
    assert mb.gemv_multi_workspace_bytes([1, 1], [8, 1 << 22], 1024) == 0    # more than 2^22 rows in all

    ia = lambda v: (ctypes.c_int * len(v))(*v)
    dummy = (ctypes.c_void_p * 2)(0x1000, 0x2000)
    call = lambda nseg, K, M, N=1024, group=128, dtype=1, batch=1, x=0x3000, y=0x4000: L.mbok_gemv_multi(
        nseg, ctypes.cast(dummy, ctypes.c_void_p), ctypes.cast(dummy, ctypes.c_void_p),
        ctypes.cast(ia(K), ctypes.c_void_p), ctypes.cast(ia(M), ctypes.c_void_p), N, group, x, dtype, batch, y,
        None, 0, None)
    assert call(0, [1], [8]) == 1                       # no matrix
    assert call(9, [1] * 9, [8] * 9) == 1               # too many
    assert call(2, [1, 5], [8, 8]) == 1                 # K out of range
    assert call(2, [1, 2], [8, 0]) == 2                 # M < 1
    assert call(2, [1, 2], [8, 8], N=1000) == 2         # N not a multiple of 128
    assert call(2, [1, 2], [8, 8], group=64) == 4       # group != 128
    assert call(2, [1, 2], [8, 8], dtype=7) == 1        # bad dtype
    assert call(2, [1, 2], [8, 8], batch=17) == 1       # batch out of range
    assert call(2, [1, 2], [8, 8], x=0x3008) == 3       # x not 16-byte aligned
    assert call(2, [1, 2], [8, 8]) == 6                 # N > 512 needs a workspace


def test_gemv_ex_argument_checks(L):
    # Per-call kernel choice and static-weights flag: invalid values are
    # refused on the host before anything is launched (the pointers are never
    # dereferenced).
    P = 1 << 20
    assert L.mbok_gemv_ex(P, P, 3, 64, 512, 128, P, 1, 1, P, P, 1 << 20, 5, 1, None) == 1
    assert L.mbok_gemv_ex(P, P, 3, 64, 512, 128, P, 1, 1, P, P, 1 << 20, -1, 1, None) == 1
    assert L.mbok_gemv_ex(P, P, 3, 64, 512, 128, P, 1, 1, P, P, 1 << 20, 1, 2, None) == 1
    assert L.mbok_gemv_ex(P, P, 3, 64, 500, 128, P, 1, 1, P, P, 1 << 20, 1, 1, None) == 2


def test_gemv_gated_sizes_and_argument_errors(L):
    O = lambda M: (M + 7) // 8
    # both projections' partials [N/512 slabs][O * 8], with one slab too; none for more than one vector
    assert L.mbok_gemv_gated_workspace_bytes(3, 2, 100, 4096, 1) == 2 * 8 * O(100) * 8 * 4
    assert L.mbok_gemv_gated_workspace_bytes(3, 2, 100, 128, 1) == 2 * O(100) * 8 * 4
    assert L.mbok_gemv_gated_workspace_bytes(3, 2, 100, 4096, 2) == 0      # one CTA covers 4096 columns
    assert L.mbok_gemv_gated_workspace_bytes(3, 2, 100, 11008, 2) >= 3 * 2 * 2 * 100 * 4
    assert L.mbok_gemv_gated_workspace_bytes(3, 2, 100, 4096, 17) == 0
    assert L.mbok_gemv_gated_workspace_bytes(0, 2, 100, 4096, 1) == 0
    g = lambda **kw: L.mbok_gemv_gated(*[kw.get(k, v) for k, v in dict(
        pg=FAKE, ag=FAKE, Kg=3, pu=FAKE, au=FAKE, Ku=2, M=64, N=1024, group=128, x=FAKE, dt=1, batch=1, h=FAKE, hd=1,
        ws=FAKE, wsb=1 << 20, stream=None).items()])
    assert g(Kg=0) == 1 and g(Ku=5) == 1 and g(M=0) == 2 and g(N=100) == 2 and g(group=64) == 4
    for name in ("pg", "ag", "pu", "au", "x", "h"):
        assert g(**{name: None}) == 1
    for name in ("pg", "ag", "pu", "au", "x"):
        assert g(**{name: FAKE + 8}) == 3
    assert g(h=FAKE_ODD) == 3 and g(h=FAKE + 2, hd=0) == 3
    assert g(dt=7) == 1 and g(hd=2) == 1 and g(batch=0) == 1 and g(batch=17) == 1
    assert g(ws=None) == 6 and g(wsb=16) == 6 and g(ws=FAKE + 4) == 6


def test_gated_backward_argument_errors(L):
    g = lambda **kw: L.mbok_gated_backward(*[kw.get(k, v) for k, v in dict(
        dH=FAKE, gate=FAKE, up=FAKE, T=4, M=64, dg=FAKE, du=FAKE, H=None, stream=None).items()])
    assert g(T=0) == 2 and g(M=0) == 2 and g(T=1 << 24) == 2 and g(M=1 << 23) == 2 and g(T=1 << 23, M=1 << 22) == 2
    for name in ("dH", "gate", "up", "dg", "du"):
        assert g(**{name: None}) == 1 and g(**{name: FAKE + 2}) == 3
    assert g(H=FAKE + 8) == 3


def test_distill_argument_errors(L):
    base = dict(z=FAKE, dt=0, T=4, V=100, ld=100, teacher=FAKE, index=FAKE, top=8, tau=1.0, weight=FAKE, loss=FAKE,
                lse=FAKE, dz=FAKE, ldz=100, stream=None)
    g = lambda **kw: L.mbok_distill_loss(*[kw.get(k, v) for k, v in base.items()])
    back = dict(z=FAKE, dt=0, T=4, V=100, ld=100, teacher=FAKE, index=FAKE, top=8, tau=1.0, weight=None, lse=FAKE,
                grad=None, dz=FAKE + 4096, ldz=100, stream=None)
    b = lambda **kw: L.mbok_distill_backward(*[kw.get(k, v) for k, v in back.items()])
    for f in (g, b):
        assert f(dt=2) == 1 and f(T=0) == 2 and f(V=0) == 2 and f(V=(1 << 21) + 1, ld=1 << 22) == 2 and f(ld=99) == 2
        assert f(top=0) == 1 and f(top=513) == 1
        assert f(tau=0.0) == 1 and f(tau=-1.0) == 1 and f(tau=float("nan")) == 1 and f(tau=float("inf")) == 1
        for name in ("z", "teacher", "index", "lse"):
            assert f(**{name: None}) == 1
        assert f(z=FAKE + 8) == 3 and f(teacher=FAKE_ODD) == 3 and f(index=FAKE + 2) == 3 and f(dz=FAKE + 8) == 3
        assert f(ldz=99) == 2
        assert f(dz=FAKE, ld=104, ldz=100) == 2      # in place with another row distance
    assert g(loss=None) == 1 and b(dz=None) == 1 and b(grad=FAKE_ODD) == 3 and g(weight=FAKE_ODD) == 3


def test_finetune_binding_refuses_cpu_tensors(L):
    import torch
    import boolean_weight_matmul_b200 as mb
    t = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mb.gated_backward(t, t, t, 1, 64, t, t)
    with pytest.raises(ValueError):
        mb.distill_loss(t, mb.BF16, 1, 64, 64, t, t, 1, 1.0, None, t, t)


def test_gemm_gated_sizes_and_argument_errors(L):
    up = lambda n, m: (n + m - 1) // m * m
    assert L.mbok_gemm_gated_workspace_bytes(100, 256, 33) == up(33 * 256 * 2, 256) + up(up(33, 16) * 4, 256)
    assert L.mbok_gemm_gated_workspace_bytes(100, 250, 33) == 0 and L.mbok_gemm_gated_workspace_bytes(100, 256, 0) == 0
    g = lambda **kw: L.mbok_gemm_gated(*[kw.get(k, v) for k, v in dict(
        pg=FAKE, ag=FAKE, Kg=3, pu=FAKE, au=FAKE, Ku=2, M=64, N=1024, group=128, X=FAKE, T=40, H=FAKE, gate=None,
        up=None, ws=FAKE, wsb=1 << 24, stream=None).items()])
    assert g(Kg=0) == 1 and g(Ku=5) == 1 and g(M=0) == 2 and g(N=100) == 2 and g(group=64) == 4
    assert g(T=0) == 2 and g(T=(1 << 23) + 1) == 2
    for name in ("pg", "ag", "pu", "au", "X", "H"):
        assert g(**{name: None}) == 1 and g(**{name: FAKE + 8}) == 3
    assert g(gate=FAKE) == 1 and g(up=FAKE) == 1                    # both projections or neither
    assert g(gate=FAKE + 2, up=FAKE) == 3 and g(gate=FAKE, up=FAKE + 8) == 3
    assert g(ws=None) == 6 and g(wsb=16) == 6 and g(ws=FAKE + 16) == 6


def test_gemm_backward_sizes_and_argument_errors(L):
    import boolean_weight_matmul_b200 as mb
    one = mb.gemm_backward_workspace_bytes([3], [64], 1024, 40)
    ragged = mb.gemm_backward_workspace_bytes([3], [63], 1024, 40)
    assert one >= 40 * 64 * 2 + 48 * 4 and ragged >= one + 40 * 64 * 2     # the copy with aligned rows
    # few tiles and many tokens: partial sums of several token splits
    assert mb.gemm_backward_workspace_bytes([1], [64], 256, 4096) > 4096 * 64 * 2 + 2 * 64 * 2 * 4
    assert mb.gemm_backward_workspace_bytes([5], [64], 1024, 40) == 0
    assert mb.gemm_backward_workspace_bytes([1] * 9, [8] * 9, 1024, 40) == 0
    assert mb.gemm_backward_workspace_bytes([1], [8], 1000, 40) == 0
    assert mb.gemm_backward_workspace_bytes([1], [8], 1024, 0) == 0

    arr = lambda *v: ctypes.cast((ctypes.c_void_p * len(v))(*v), ctypes.c_void_p)
    ia = lambda *v: ctypes.cast((ctypes.c_int * len(v))(*v), ctypes.c_void_p)
    g = lambda **kw: L.mbok_gemm_backward(*[kw.get(k, v) for k, v in dict(
        n=2, packed=arr(FAKE, FAKE), alpha=arr(FAKE, FAKE), K=ia(3, 2), M=ia(64, 40), N=1024, group=128, X=FAKE, T=40,
        dY=arr(FAKE, FAKE), dX=FAKE, da=arr(FAKE, FAKE), ws=FAKE, wsb=1 << 26, stream=None).items()])
    assert g(n=0) == 1 and g(n=9) == 1 and g(K=None) == 1 and g(M=None) == 1
    assert g(K=ia(3, 5)) == 1 and g(M=ia(64, 0)) == 2 and g(N=1000) == 2 and g(group=64) == 4
    assert g(T=0) == 2 and g(T=(1 << 23) + 1) == 2
    for name in ("packed", "alpha", "dY"):
        assert g(**{name: None}) == 1 and g(**{name: arr(FAKE, None)}) == 1 and g(**{name: arr(FAKE, FAKE + 8)}) == 3
    assert g(da=arr(None, FAKE + 8)) == 3 and g(dX=FAKE + 8) == 3 and g(X=FAKE + 8) == 3
    assert g(dX=None, da=None) == 1 and g(dX=None, da=arr(None, None)) == 1       # nothing asked for
    assert g(X=None) == 1                                                          # scales need X
    assert g(ws=None) == 6 and g(wsb=16) == 6 and g(ws=FAKE + 16) == 6
    with pytest.raises(ValueError):
        mb.gemm_backward([FAKE], [FAKE, FAKE], [1], [8], 128, 128, FAKE, 1, [FAKE], FAKE, None, None)


def test_finetune_calls_refuse_overlapping_buffers(L):
    # refused on the host before anything is launched; buffers that only touch are
    # not (without a GPU such a call then fails to launch: MBOK_ERR_CUDA)
    import torch
    P, MB = 1 << 30, 1 << 20
    g = lambda h, x, hd=1: L.mbok_gemv_gated(P, P, 3, P, P, 2, 64, 1024, 128, x, 1, 2, h, hd, P, MB, None)
    assert g(P, P) == 1 and g(P + 4080, P) == 1 and g(P - 16, P) == 1 and g(P - 496, P, 0) == 1
    b = lambda dh, gate, up, dg, du, H: L.mbok_gated_backward(dh, gate, up, 4, 64, dg, du, H, None)   # 512 bytes each
    a = [P + i * MB for i in range(6)]
    assert b(*a[:3], a[3], a[3], a[5]) == 1 and b(*a[:4], a[5] - 496, a[5]) == 1 and b(*a[:3], a[3], a[4], a[3] + 16) == 1
    assert b(*a[:3], a[0] + 16, a[4], a[5]) == 1 and b(*a[:3], a[3], a[2] - 16, None) == 1
    m = lambda H, gate, up: L.mbok_gemm_gated(P, P, 3, P, P, 2, 64, 1024, 128, P, 40, H, gate, up, P, 1 << 24, None)
    assert m(a[0], a[0], a[1]) == 1 and m(a[0], a[1], a[1] + 16) == 1 and m(a[0], a[2], a[0] + 5104) == 1
    arr = lambda *v: ctypes.cast((ctypes.c_void_p * len(v))(*v), ctypes.c_void_p)
    ia = lambda *v: ctypes.cast((ctypes.c_int * len(v))(*v), ctypes.c_void_p)
    back = lambda X, dY, dX, da: L.mbok_gemm_backward(2, arr(P, P), arr(P, P), ia(3, 2), ia(64, 40), 1024, 128, X, 40,
                                                      arr(*dY), dX, da, P, 1 << 26, None)
    assert back(a[0], a[1:3], a[0] + 81904, arr(a[3], None)) == 1          # X: 81920 bytes
    assert back(a[0], a[1:3], a[2] - 16, arr(None, a[3])) == 1
    assert back(a[0], a[1:3], a[3], arr(a[4], a[4])) == 1                  # one dalpha for two matrices
    loss = lambda lo, ls: L.mbok_distill_loss(P, 0, 4, 100, 100, P, P, 8, 1.0, None, lo, ls, None, 0, None)
    assert loss(a[0], a[0]) == 1 and loss(a[0], a[0] + 12) == 1
    if not torch.cuda.is_available():
        assert loss(a[0], a[0] + 16) == 5
        assert g(P + 4096, P) == 5 and b(*a[:3], a[0], a[1], a[2]) == 5 and m(a[0], a[0] + 5120, a[0] + 10240) == 5
        assert back(a[0], a[1:3], a[0], None) == 5                          # dX alone reads dY before it is written


def test_marshalled_calls_convert_and_refuse(L):
    import torch
    import boolean_weight_matmul_b200 as mb
    # raw pointers, ints and a raw stream reach the library, whose status comes back
    for status, kw in ((2, dict(T=0)), (1, dict(dH=None)), (3, dict(up=FAKE + 2))):
        a = dict(dH=FAKE, gate=FAKE, up=FAKE, T=4, M=64, dgate=FAKE, dup=FAKE, H=None, stream=0)
        with pytest.raises(mb.MbokError) as e:
            mb.gated_backward(**{**a, **kw})
        assert e.value.status == status and "mbok_gated_backward" in str(e.value)
    t = torch.zeros(64, dtype=torch.bfloat16)
    two = [FAKE, FAKE]
    back = lambda **kw: mb.gemm_backward(*[kw.get(k, v) for k, v in dict(
        packed=two, alpha=two, K=[3, 2], M=(64, 40), N=1024, group=128, X=FAKE, T=40, dY=two, dX=FAKE, da=None, ws=None,
        stream=0).items()])
    with pytest.raises(mb.MbokError) as e:
        back()
    assert e.value.status == 6                                   # no workspace: every other argument passed
    for kw, status in ((dict(K=[3, 5]), 1), (dict(M=[64, 0]), 2), (dict(packed=[FAKE, None]), 1), (dict(N=1000), 2),
                       (dict(packed=[FAKE] * 9, alpha=[FAKE] * 9, K=[1] * 9, M=[8] * 9, dY=[FAKE] * 9), 1)):
        with pytest.raises(mb.MbokError) as e:
            back(**kw)
        assert e.value.status == status
    with pytest.raises(ValueError):
        back(dY=[FAKE, t])                                       # a CPU tensor in a list
    with pytest.raises(ValueError):
        back(ws=t)
    with pytest.raises(TypeError):
        back(ws=FAKE)                                            # a workspace has a size
    with pytest.raises(TypeError):
        back(X="x")
    with pytest.raises(TypeError):
        back(K=[3, "x"])
    with pytest.raises(OverflowError):
        back(T=1 << 40)
    with pytest.raises(OverflowError):
        mb.distill_loss(FAKE, mb.F32, 1, 8, -1, FAKE, FAKE, 1, 1.0, None, FAKE, FAKE, stream=0)
    with pytest.raises(TypeError):
        mb.distill_backward(FAKE, mb.F32, 1, 8, 8, FAKE, FAKE, 1, "x", None, FAKE, None, FAKE, 8, 0)
    with pytest.raises(mb.MbokError) as e:
        mb.distill_backward(FAKE, mb.F32, 1, 8, 8, FAKE, FAKE, 1, float("nan"), None, FAKE, None, FAKE, 8, 0)
    assert e.value.status == 1
    with pytest.raises(TypeError):
        mb._marshal().gated_backward(FAKE)                       # too few arguments
    import numpy as np
    with pytest.raises(mb.MbokError) as e:                       # numpy's integers as Python's
        mb.distill_loss(FAKE, mb.F32, np.int64(1), np.int32(8), np.int64(7), FAKE, FAKE, 1, 1.0, None, FAKE, FAKE,
                        stream=0)
    assert e.value.status == 2
