"""Calls of the gated, gradient and distillation operators that the documentation
allows and that are easily got wrong: gradients in place, values near the ends of
their type, masks, uneven batches.  Tolerances as in test_finetune_ops.py."""
import numpy as np
import pytest

from oracle import finetune_oracle as F
from helpers import ensure_built, guarded, to_dev
import test_finetune_ops as ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


# ---- distillation in place -----------------------------------------------------

@pytest.mark.parametrize("dtype,V,T,top,rounds", [("bf16", 2053, 1300, 512, 3), ("f32", 2053, 1300, 512, 3),
                                                  ("bf16", 9, 2400, 9, 20), ("bf16", 17, 2400, 17, 20),
                                                  ("bf16", 33, 1800, 33, 20), ("f32", 5, 2400, 5, 20),
                                                  ("f32", 33, 1800, 33, 20)])
def test_distill_in_place_with_listed_row_ends(dtype, V, T, top, rounds):
    # many rows of every alignment, every element of their partial 16-byte vectors listed: the gradient written over
    # the logits has the bits of the gradient written elsewhere, as have loss and lse
    import torch
    import boolean_weight_matmul_b200 as mb
    tau = 2.0
    z, teacher, index, weight, _ = ops._distill_case(T, V, top, 31, dtype)
    ends = np.concatenate([np.arange(8), np.arange(V - 8, V)]) if V > 33 else np.arange(V)[:top]
    for t in range(4, T):   # at the end of the list, whose entries are gathered last
        index[t, top - len(ends):] = np.roll(ends, t)
    weight[5::11] = 0.0
    index[6::11] = -1
    td, xd, wd = to_dev(teacher), to_dev(index), to_dev(weight)
    loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
    dz = guarded((T, V), ops._dt(dtype))
    mb.distill_loss(z.cuda(), ops._code(dtype), T, V, V, td, xd, top, tau, wd, loss, lse, dz, V)
    torch.cuda.synchronize()
    ops._check_distill(z, teacher, index, weight, np.ones(T, dtype=np.float32), tau, V, dtype, ops._f64(loss),
                       ops._f64(lse), ops._f64(dz))
    for _ in range(rounds):
        zd = z.cuda()
        loss2, lse2 = torch.zeros_like(loss), torch.zeros_like(lse)
        mb.distill_loss(zd, ops._code(dtype), T, V, V, td, xd, top, tau, wd, loss2, lse2, zd, V)
        torch.cuda.synchronize()
        assert mb.read_device_errors() == 0
        assert torch.equal(zd, dz) and torch.equal(loss2, loss) and torch.equal(lse2, lse)


# ---- gated decode ----------------------------------------------------------------

@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tiny", [1e-36, 2.0 ** -126, 2.0 ** -133])
def test_gemv_gated_tiny_activations(x_dtype, tiny):
    # activations far below one, subnormals among them, with zeros between: in all columns, and in one warp's 256
    # columns alone; nothing becomes an infinity or NaN
    import torch
    K, M, N, batch = 2, 37, 512, 3
    gate, up = ops.Layer(K, M, N, 201), ops.Layer(K, M, N, 202)
    rng = np.random.default_rng(203)
    for first in (0, 256):   # columns below `first` are ordinary
        x = rng.standard_normal((batch, N))
        x[:, first:] = np.sign(x[:, first:]) * tiny
        x[:, first::3] = 0.0
        xd = torch.from_numpy(x).to(ops._dt(x_dtype)).cuda()
        x64 = ops._f64(xd)
        assert (x64[:, first:] != 0).any()
        h = ops._gemv_gated(gate, up, xd, x_dtype, batch, "f32")
        g, Eg = F.project(gate.words, gate.alpha, K, M, N, x64)
        u, Eu = F.project(up.words, up.alpha, K, M, N, x64)
        want = F.silu(g) * u
        ops._assert_within(ops._f64(h), want, ops._gated_tol(g, Eg, u, Eu, N * K, want, "f32"), f"{first}")


@pytest.mark.parametrize("batch", [6, 7, 11, 13, 16])
@pytest.mark.parametrize("M,N", [(70, 1664), (1300, 256), (129, 5248)])
def test_gemv_gated_fp32_vectors_in_uneven_chunks(batch, M, N):
    # fp32 vectors go in equal chunks of at most five, of which the last may be shorter: each vector has the bits of
    # a call that brings it in a chunk of the same size
    import torch
    import boolean_weight_matmul_b200 as mb
    gate, up = ops.Layer(3, M, N, 211, pad_nan=True), ops.Layer(2, M, N, 212, pad_nan=True)
    x, x64 = ops._x(batch, N, 213 + batch, "f32")
    h = ops._gemv_gated(gate, up, to_dev(x), "f32", batch, "f32")
    g, Eg = F.project(gate.words, gate.alpha, 3, M, N, x64)
    u, Eu = F.project(up.words, up.alpha, 2, M, N, x64)
    want = F.silu(g) * u
    ops._assert_within(ops._f64(h), want, ops._gated_tol(g, Eg, u, Eu, N * 3, want, "f32"))
    per = -(-batch // -(-batch // 5))
    for v in range(0, batch, per):
        n = min(per, batch - v)
        if n < 2:
            continue   # one vector takes the lookup kernel
        if (3 * n <= 8) != (3 * per <= 8):
            continue   # another tile width, whose warps take other columns
        alone = ops._gemv_gated(gate, up, to_dev(x[v:v + n].copy()), "f32", n, "f32")
        assert torch.equal(alone, h[v:v + n])


# ---- distillation ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_weight_zero_masks_any_incoming_gradient(dtype):
    import torch
    import boolean_weight_matmul_b200 as mb
    T, V, top, tau = 8, 1003, 6, 2.0
    z, teacher, index, weight, grad = ops._distill_case(T, V, top, 41, dtype, masked=False)
    weight[:4] = 0.0
    index[4] = -1
    z[1, 5], z[2, :] = float("nan"), float("-inf")
    grad[0], grad[1], grad[2], grad[4] = np.nan, np.inf, -np.inf, np.nan
    td, xd, wd, gd = to_dev(teacher), to_dev(index), to_dev(weight), to_dev(grad)
    loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
    mb.distill_loss(z.cuda(), ops._code(dtype), T, V, V, td, xd, top, tau, wd, loss, lse)
    dz = guarded((T, V), ops._dt(dtype))
    mb.distill_backward(z.cuda(), ops._code(dtype), T, V, V, td, xd, top, tau, wd, lse, gd, dz, V)
    torch.cuda.synchronize()
    assert (dz[:5] == 0).all() and (loss[:5] == 0).all()
    ops._check_distill(z[5:], teacher[5:], index[5:], weight[5:], grad[5:], tau, V, dtype, ops._f64(loss[5:]),
                       ops._f64(lse[5:]), ops._f64(dz[5:]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,top,tau", [(6, 2053, 9, 1.0), (6, 2053, 9, 2.0), (3, 40000, 9, 8.0), (640, 2053, 9, 2.0),
                                         (640, 515, 9, 1.0)])
def test_distill_masked_by_large_negative_logits(dtype, T, V, top, tau):
    # blocks of logits masked by the lowest value and by other large negative numbers, more than one thread's share:
    # probability 0 at every temperature; a row where nothing else is left has no distribution
    import torch
    import boolean_weight_matmul_b200 as mb
    z, teacher, index, weight, _ = ops._distill_case(T, V, top, 51, dtype, masked=False)
    index = np.stack([np.random.default_rng(52 + t).permutation(V // 4)[:top] for t in range(T)]).astype(np.int32)
    clean = z.clone()
    masks = [torch.finfo(z.dtype).min, -1e30, -1e10, -3e9]
    for t in range(T - 1):
        first = V // 4 + (37 * t) % (V // 2)
        z[t, first:first + V // 4] = masks[t % 4]
        clean[t, first:first + V // 4] = float("-inf")
    z[T - 1] = torch.finfo(z.dtype).min
    td, xd, wd = to_dev(teacher), to_dev(index), to_dev(weight)
    loss, lse, dz = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), ops._dt(dtype))
    ones = np.ones(T, dtype=np.float32)
    args = (z.cuda(), ops._code(dtype), T, V, V, td, xd, top, tau, wd)
    mb.distill_loss(*args, loss, lse, dz, V)
    dz2 = guarded((T, V), ops._dt(dtype))
    mb.distill_backward(*args, lse, None, dz2, V)
    torch.cuda.synchronize()
    for d in (dz, dz2):
        ops._check_distill(clean[:-1], teacher[:-1], index[:-1], weight[:-1], ones[:-1], tau, V, dtype,
                           ops._f64(loss[:-1]), ops._f64(lse[:-1]), ops._f64(d[:-1]))
        assert torch.isnan(loss[-1]) and torch.isnan(d[-1]).all()


@pytest.mark.parametrize("T", [4, 640])
def test_distill_huge_logits(T):
    # logits whose step is many units: all probability on the largest, shared where there are several; the gradient
    # has the ordinary relative error, since the differences of such logits are exact
    import torch
    import boolean_weight_matmul_b200 as mb
    V, top, tau = 1031, 5, 1.5
    _, teacher, index, _, _ = ops._distill_case(T, V, top, 61, "f32", masked=False)
    rng = np.random.default_rng(62)
    for sign in (1.0, -1.0):
        z = torch.from_numpy(sign * 2.0 ** 34 + 4096.0 * rng.integers(0, 3, (T, V))).float()
        loss, lse, dz = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), torch.float32)
        mb.distill_loss(z.cuda(), mb.F32, T, V, V, to_dev(teacher), to_dev(index), top, tau, None, loss, lse, dz, V)
        torch.cuda.synchronize()
        ones = np.ones(T)
        want_loss, want_lse, want, q, p = F.distill(z.double().numpy(), teacher.astype(np.float64), index, tau, ones, ones)
        # exponents of the largest are 0; the teacher's are off by 2^-24 of at most 16, and its sum by top 2^-24
        ops._assert_within(ops._f64(dz), want, (q + p) / tau * 2.0 ** -18 + 1e-38, "dz")
        # the loss is sum p (m - z) / tau and ordinary terms: a few roundings of each
        ops._assert_within(ops._f64(loss), want_loss, np.abs(want_loss) * 2.0 ** -20 + 1e-4, "loss")
        ops._assert_within(ops._f64(lse), want_lse, np.abs(want_lse) * 2.0 ** -22, "lse")


@pytest.mark.parametrize("T,V", [(5, 64), (640, 64), (640, 2048)])
@pytest.mark.parametrize("dtype,shift", [("f32", 0.0), ("bf16", 0.0), ("f32", 56.0), ("bf16", 56.0), ("f32", -56.0),
                                         ("bf16", -56.0), ("f32", 3.0e4)])   # 3e4 + 1/4 is no bf16 value
def test_distill_small_loss_does_not_depend_on_a_shift(dtype, T, V, shift):
    # a student that equals its teacher: loss 0, and a gradient of 0, whatever is added to all of its logits
    import torch
    import boolean_weight_matmul_b200 as mb
    top = min(V, 512)
    rng = np.random.default_rng(71)
    teacher = (rng.integers(-32, 32, (T, top)) / 4.0).astype(np.float32)   # steps of 1/4: exact in bf16 below 64
    index = np.stack([rng.permutation(V)[:top] for _ in range(T)]).astype(np.int32)
    z = np.full((T, V), -np.inf)
    np.put_along_axis(z, index.astype(np.int64), teacher + shift, 1)
    zd = torch.from_numpy(z).to(ops._dt(dtype)).cuda()
    assert (ops._f64(zd) == z).all()
    loss, lse, dz = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), ops._dt(dtype))
    mb.distill_loss(zd, ops._code(dtype), T, V, V, to_dev(teacher), to_dev(index), top, 1.0, None, loss, lse, dz, V)
    torch.cuda.synchronize()
    t64 = teacher.astype(np.float64)
    gap = t64 - t64.max(1, keepdims=True)
    p = np.exp(gap) / np.exp(gap).sum(1, keepdims=True)
    # per entry: the teacher's and the student's exponents are off by 2^-24 of |gap| + 1 each and their factors by as
    # much; the logarithms of the two sums, of their exponentials' 2^-22 and of their own 2^-23 each
    tol = (8 + 4 * (p * np.abs(gap)).sum(1)) * 2.0 ** -23
    ops._assert_within(ops._f64(loss), np.zeros(T), tol, "loss")
    q = np.zeros((T, V))
    np.put_along_axis(q, index.astype(np.int64), p, 1)
    ops._assert_within(ops._f64(dz), np.zeros((T, V)), q * 2.0 ** -18 + 1e-38, "dz")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [515, 2053, 9001])
def test_distill_many_rows_with_peaks_and_holes(dtype, V):
    # single logits far above all others (a row's first reference is far below its sum, or as far as it may be), rows
    # with few logits left, and rows with one
    import torch
    import boolean_weight_matmul_b200 as mb
    T, top, tau = 640, 7, 1.0
    z, teacher, index, weight, _ = ops._distill_case(T, V, top, 81, dtype, masked=False)
    rng = np.random.default_rng(82)
    for t in range(T):
        kind = t % 4
        if kind < 2:
            z[t, rng.integers(0, V)] = (18.0, 24.0, 45.0, 90.0)[t // 4 % 4]
            z[t, index[t, 2]] += (15.0, 40.0)[kind]
        else:
            keep = index[t].astype(np.int64) if kind == 2 else index[t, :1].astype(np.int64)
            row = torch.full((V,), float("-inf") if t % 8 < 4 else -1e9, dtype=z.dtype)
            row[keep] = z[t, keep] + (0.0, -700.0, 900.0)[t // 4 % 3]
            z[t] = row
            if kind == 3:
                index[t, 1:] = -1
    loss, lse, dz = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), ops._dt(dtype))
    mb.distill_loss(z.cuda(), ops._code(dtype), T, V, V, to_dev(teacher), to_dev(index), top, tau, to_dev(weight), loss,
                    lse, dz, V)
    torch.cuda.synchronize()
    assert mb.read_device_errors() == 0
    clean = torch.where(z == torch.tensor(-1e9).to(z.dtype), torch.full_like(z, float("-inf")), z)
    # Here q passes through 2^-126, below which the kernels' exponential is 0: q is then off by up to that and dz by
    # weight / tau of it, 1.5 x 2^-126 = 1.8e-38, which _check_distill (1e-38) does not hold.  Such values are looked
    # at here and handed on as the formula's.
    got = ops._f64(dz)
    z64 = clean.double().numpy()
    ones = np.ones(T)
    _, _, want, q, p = F.distill(z64, teacher.astype(np.float64), index, tau, weight.astype(np.float64), ones)
    flushed = (q < 2.0 ** -125) & (p == 0)
    ops._assert_within(got[flushed], want[flushed], weight.max() / tau * 2.0 ** -126 * (1 + 2.0 ** -8), "flushed")
    ops._check_distill(clean, teacher, index, weight, np.ones(T, dtype=np.float32), tau, V, dtype, ops._f64(loss),
                       ops._f64(lse), np.where(flushed, want, got))


# ---- outputs over inputs, where that is allowed ----------------------------------------

def test_token_products_over_their_inputs():
    # the gated product over X, dX over X's place or a dY (without scale gradients): the bits of separate buffers, whole
    # tiles and cut ones
    import torch
    import boolean_weight_matmul_b200 as mb
    for N, T in ((256, 77), (2304, 40), (1280, 600)):
        gate, up = ops.Layer(2, N, N, 301), ops.Layer(3, N, N, 302)
        X = ops.x_dev(ops.wl.x_normal(T, N, 303), "bf16")
        for keep in (False, True):
            want = ops._gemm_gated(gate, up, X, keep)
            ws = mb.empty_gemm_gated_workspace(N, N, T)
            outs = [X.clone(), torch.zeros_like(X), torch.zeros_like(X)]
            mb.gemm_gated(gate.packed, gate.blocked, 2, up.packed, up.blocked, 3, N, N, 128, outs[0], T, outs[0],
                          outs[1] if keep else None, outs[2] if keep else None, ws)
            torch.cuda.synchronize()
            assert torch.equal(outs[0], want[0])
            assert not keep or (torch.equal(outs[1], want[1]) and torch.equal(outs[2], want[2]))
        dYs = [ops._grads(T, N, 304), ops._grads(T, N, 305)]
        want, _ = ops._gemm_backward([gate, up], X, dYs, want_a=[False, False])
        ws = mb.empty_gemm_backward_workspace([2, 3], [N, N], N, T)
        for over in (0, 1):
            d = [t.clone() for t in dYs]
            mb.gemm_backward([gate.packed, up.packed], [gate.blocked, up.blocked], [2, 3], [N, N], N, 128, None, T, d,
                             d[over], None, ws)
            torch.cuda.synchronize()
            assert torch.equal(d[over], want) and torch.equal(d[1 - over], dYs[1 - over])
        assert mb.read_device_errors() == 0


# ---- scaled activations ------------------------------------------------------------------

def test_gemm_gated_smallest_activations_beside_a_large_one():
    # Each token's values are scaled so that its largest lies in [2^14, 2^15), and rounded to fp16, whose subnormals are
    # 2^-24 apart: off by at most 2^-25, that is 2^-39 of a largest value of 1.  The first group's scales are 0, so
    # that only the small values reach the result.
    import torch
    M, N, T = 16, 256, 8
    gate, up = ops.Layer(1, M, N, 401), ops.Layer(1, M, N, 402)
    x = np.zeros((T, N))
    x[:, 0] = 1.0
    for t in range(T):
        x[t, 128:] = np.where(np.arange(128) % (t + 1) == 0, (1.5, 1.25, 3.5, 0.75)[t % 4], 0.0) * 2.0 ** -38
    X = torch.from_numpy(x).to(torch.bfloat16).cuda()
    assert (ops._f64(X) == x).all()
    for layer in (gate, up):
        blocked = layer.blocked.view(-1, N // 128, 1, 8)
        blocked[:, 0] = 0.0
        blocked[:, 1] = 1.0
        layer.alpha = layer.alpha.copy()
        layer.alpha[:, 0], layer.alpha[:, 1] = 0.0, 1.0
    got = ops._gemm_gated(gate, up, X, True)
    for layer, out in ((gate, got[1]), (up, got[2])):
        want = x @ ops._dense_abs(layer).T
        tol = 2.0 ** -39 * (x[:, 128:] != 0).sum(1, keepdims=True) + np.abs(want) * ops.HALF["bf16"]
        ops._assert_within(ops._f64(out), want, tol)


@pytest.mark.parametrize("dtype,V", [("bf16", 1003), ("f32", 1000)])
def test_distill_many_rows_without_a_distribution(dtype, V):
    # rows with a NaN, with +infinity, with nothing but masks, unused ones among them: NaN and 0 stay in their rows
    import torch
    import boolean_weight_matmul_b200 as mb
    T, top, tau = 640, 6, 2.0
    z, teacher, index, weight, _ = ops._distill_case(T, V, top, 91, dtype, masked=False)
    clean = z.clone()
    for t in range(0, T, 5):
        kind = t // 5 % 6
        if kind < 3:
            z[t, (0, V // 2, V - 1)[kind]] = float("nan")
        elif kind == 3:
            z[t, V - 2] = float("inf")
        else:
            z[t] = float("-inf") if kind == 4 else torch.finfo(z.dtype).min
    index[7::25] = -1
    weight[10::25] = 0.0
    bad = np.zeros(T, dtype=bool)
    bad[::5] = True
    unused = (weight == 0) | (index < 0).all(1)
    args = (ops._code(dtype), T, V, V, to_dev(teacher), to_dev(index), top, tau, to_dev(weight))
    ones = np.ones(T, dtype=np.float32)
    for place in ("own", "over the logits"):
        zd = z.cuda()
        loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
        dz = guarded((T, V), ops._dt(dtype)) if place == "own" else zd
        mb.distill_loss(zd, *args, loss, lse, dz, V)
        torch.cuda.synchronize()
        assert mb.read_device_errors() == 0
        got = ops._f64(dz)
        assert np.isnan(ops._f64(loss)[bad & ~unused]).all() and np.isnan(got[bad & ~unused]).all()
        assert (ops._f64(loss)[unused] == 0).all() and (got[unused] == 0).all()
        good = ~bad
        ops._check_distill(clean[good], teacher[good], index[good], weight[good], ones[good], tau, V, dtype,
                           ops._f64(loss)[good], ops._f64(lse)[good], got[good])
