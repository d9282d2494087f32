"""Gated feed-forward and fine-tuning calls on the GPU against an fp64 oracle
(oracle/finetune_oracle.py), at the sizes and masks where they can go wrong.

Tolerances, derived before the first run:
 * a sum of n fp32 terms taken in any order is off by at most n 2^-24 times the
   sum of their absolute values (GAMMA below);
 * an output rounded once to type t adds half a step, finfo(t).eps / 2 of its
   value (HALF below);
 * what else a formula adds is said where its tolerance is formed."""
import numpy as np
import pytest

from boolean_weight_matmul_b200 import workloads as wl
from oracle import finetune_oracle as F
from oracle import mbok_oracle as O
from helpers import alpha_blocked_gpu, ensure_built, guarded, packed_from_signs_gpu, to_dev, x_dev

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def gamma(n):
    return n * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def _dt(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


def _code(name):
    import boolean_weight_matmul_b200 as mb
    return mb.F32 if name == "f32" else mb.BF16


def _f64(t):
    return t.double().cpu().numpy()


def _assert_within(got, want, tol, what=""):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
    ok = np.abs(got - want) <= tol
    if not ok.all():
        bad = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.size} out of tolerance, e.g. {bad} got {got[bad]} "
                             f"want {want[bad]} tolerance {np.broadcast_to(tol, got.shape)[bad]}")


class Layer:
    """One matrix: host signs and scales, and their device forms."""

    def __init__(self, K, M, N, seed, pad_nan=False):
        import torch
        self.K, self.M, self.N = K, M, N
        signs = wl.random_signs(K, M, N, seed)
        self.alpha = wl.alpha_decaying(K, M, N, seed + 1)
        self.words = O.pack_signs(signs)
        self.packed = packed_from_signs_gpu(signs)
        self.blocked = alpha_blocked_gpu(self.alpha, K, M, N)
        if pad_nan and M % 8:
            # the rows that pad the last octet hold anything: every reader ignores them
            self.blocked.view(-1, N // 128, K, 8)[-1, :, :, M % 8:] = float("nan")
            torch.cuda.synchronize()

    def host(self):
        return self.words, self.alpha, self.K, self.M


# ---- gated decode ------------------------------------------------------------

def _x(batch, N, seed, dtype):
    x = wl.x_normal(batch, N, seed, dtype)
    return x, (x.astype(np.float64) if dtype == "f32" else wl.bf16_bits_to_f32(x).astype(np.float64))


def _gated_tol(g, Eg, u, Eu, n, h, out):
    # g and u are sums of n terms; |silu'| < 1.1; expf, the division and the
    # product add at most 2^-20 of the value, expf's argument |g| 2^-24 more
    e = 1.1 * np.abs(u) * gamma(n) * Eg + np.abs(F.silu(g)) * gamma(n) * Eu
    return e * 1.01 + np.abs(h) * (2.0 ** -20 + np.abs(g) * 2.0 ** -23 + HALF[out]) + 1e-30


def _gemv_gated(gate, up, xd, x_dtype, batch, out):
    import torch
    import boolean_weight_matmul_b200 as mb
    h = guarded((batch, gate.M), _dt(out))
    ws = mb.empty_gated_workspace(gate.K, up.K, gate.M, gate.N, batch)
    ws.fill_(0xFF)   # NaN: nothing may be read before it is written
    mb.gemv_gated(gate.packed, gate.blocked, gate.K, up.packed, up.blocked, up.K, gate.M, gate.N, 128, xd,
                  _code(x_dtype), batch, h, _code(out), ws)
    torch.cuda.synchronize()
    assert mb.read_device_errors() == 0
    return h


@pytest.mark.parametrize("kg,ku", [(1, 1), (3, 3), (4, 1), (2, 4)])
@pytest.mark.parametrize("M,N", [(1, 128), (7, 512), (13, 640), (129, 1024), (200, 4224), (40, 5248)])
@pytest.mark.parametrize("batch", [1, 2, 5, 8, 16])
def test_gemv_gated(kg, ku, M, N, batch):
    gate, up = Layer(kg, M, N, 9000 + kg + M, pad_nan=True), Layer(ku, M, N, 9100 + ku + N, pad_nan=True)
    for x_dtype, out in (("bf16", "bf16"), ("f32", "f32")):
        x, x64 = _x(batch, N, 77 + batch, x_dtype)
        h = _gemv_gated(gate, up, x_dev(x, x_dtype), x_dtype, batch, out)
        g, Eg = F.project(gate.words, gate.alpha, kg, M, N, x64)
        u, Eu = F.project(up.words, up.alpha, ku, M, N, x64)
        want = F.silu(g) * u
        _assert_within(_f64(h), want, _gated_tol(g, Eg, u, Eu, N * max(kg, ku), want, out), f"{x_dtype} -> {out}")


def test_gemv_gated_many_rows():
    # several octets per warp: the ring wraps, the sums' two buffers alternate
    for M, N, batch in ((5000, 256, 3), (2600, 4096, 9), (1300, 5376, 2)):
        gate, up = Layer(3, M, N, 31), Layer(2, M, N, 32)
        x, x64 = _x(batch, N, 33, "bf16")
        h = _gemv_gated(gate, up, x_dev(x, "bf16"), "bf16", batch, "f32")
        g, Eg = F.project(gate.words, gate.alpha, 3, M, N, x64)
        u, Eu = F.project(up.words, up.alpha, 2, M, N, x64)
        want = F.silu(g) * u
        _assert_within(_f64(h), want, _gated_tol(g, Eg, u, Eu, N * 3, want, "f32"))


def test_gemv_gated_mixed_types_and_alignment():
    # fp32 in, bf16 out and the other way round; an output at an odd element
    import torch
    import boolean_weight_matmul_b200 as mb
    K, M, N, batch = 3, 77, 1152, 3
    gate, up = Layer(K, M, N, 1), Layer(K, M, N, 2)
    for x_dtype, out in (("f32", "bf16"), ("bf16", "f32")):
        x, x64 = _x(batch, N, 3, x_dtype)
        g, Eg = F.project(gate.words, gate.alpha, K, M, N, x64)
        u, Eu = F.project(up.words, up.alpha, K, M, N, x64)
        want = F.silu(g) * u
        buf = guarded((batch * M + 1,), _dt(out))
        first = buf[:1].clone()
        h = buf[1:].view(batch, M)
        mb.gemv_gated(gate.packed, gate.blocked, K, up.packed, up.blocked, K, M, N, 128, x_dev(x, x_dtype),
                      _code(x_dtype), batch, h, _code(out), None)
        torch.cuda.synchronize()
        _assert_within(_f64(h), want, _gated_tol(g, Eg, u, Eu, N * K, want, out))
        assert torch.equal(first.view(torch.uint8), buf[:1].view(torch.uint8))


def test_gemv_gated_extremes():
    # a gate far below zero closes (0), far above passes u; a NaN reaches only its vector
    import torch
    K, M, N, batch = 1, 16, 256, 2
    gate, up = Layer(K, M, N, 11), Layer(K, M, N, 12)
    x, _ = _x(batch, N, 13, "f32")
    x *= 1e4
    x[1, 5] = np.nan
    for rows in (1, 2):
        h = _gemv_gated(gate, up, to_dev(x[:rows]), "f32", rows, "f32")
        g, _ = F.project(gate.words, gate.alpha, K, M, N, x[:1].astype(np.float64))
        u, _ = F.project(up.words, up.alpha, K, M, N, x[:1].astype(np.float64))
        got = _f64(h)[0]
        assert np.isfinite(got).all()
        closed = g[0] < -200
        assert closed.any() and (got[closed] == 0).all()
        opened = g[0] > 200
        assert opened.any()
        _assert_within(got[opened], (g * u)[0][opened], np.abs(g * u)[0][opened] * 1e-3)
        if rows == 2:
            assert torch.isnan(h[1]).all()


def test_gemv_gated_fp32_accuracy():
    # In norm, where errors do not line up as in the bound above: a group's sum is
    # eight MMAs, each cutting off at most 2^-23 of a running sum whose root mean
    # square is at most the group's own, so g and u are off by at most 2^-20 of
    # their norm (the groups' errors add as their sums do), and h, with |silu'| <
    # 1.1 and g u ~ h, by twice that; observed errors are a tenth of it.
    for kg, ku, M, N, batch, x_dtype in ((3, 2, 599, 768, 8, "bf16"), (1, 1, 300, 4096, 4, "f32"),
                                         (2, 4, 400, 128, 16, "f32"), (3, 3, 200, 5248, 16, "bf16")):
        gate, up = Layer(kg, M, N, 41), Layer(ku, M, N, 42)
        x, x64 = _x(batch, N, 43, x_dtype)
        h = _gemv_gated(gate, up, x_dev(x, x_dtype), x_dtype, batch, "f32")
        g, _ = F.project(gate.words, gate.alpha, kg, M, N, x64)
        u, _ = F.project(up.words, up.alpha, ku, M, N, x64)
        want = F.silu(g) * u
        assert np.linalg.norm(_f64(h) - want) <= 2.0 ** -19 * np.linalg.norm(want)


def test_gemv_gated_huge_activations():
    # activations near the type's highest: a closed gate gives 0, not infinity x 0
    import torch
    M, N, batch = 24, 256, 3
    gate, up = Layer(1, M, N, 51), Layer(1, M, N, 52)
    gate.blocked.zero_()
    up.blocked.fill_(2.0 ** -14)   # |u| <= 256 x 2^126 x 2^-14
    for x_dtype in ("bf16", "f32"):
        x = torch.full((batch, N), 2.0 ** 126, dtype=_dt(x_dtype), device="cuda")
        x[:, ::3] *= -1
        h = _gemv_gated(gate, up, x, x_dtype, batch, "f32")
        assert torch.equal(h, torch.zeros_like(h))


def test_gemv_gated_deterministic_and_graph():
    import torch
    import boolean_weight_matmul_b200 as mb
    gate, up = Layer(3, 520, 2048, 21), Layer(2, 520, 2048, 22)
    for batch in (1, 7):
        x, _ = _x(batch, 2048, 23, "bf16")
        xd = x_dev(x, "bf16")
        first = _gemv_gated(gate, up, xd, "bf16", batch, "bf16").clone()
        h = torch.zeros(batch, 520, dtype=torch.bfloat16, device="cuda")
        ws = mb.empty_gated_workspace(3, 2, 520, 2048, batch)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mb.gemv_gated(gate.packed, gate.blocked, 3, up.packed, up.blocked, 2, 520, 2048, 128, xd, mb.BF16, batch, h,
                          mb.BF16, ws)
        for _ in range(3):
            h.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, first)


# ---- the gate's gradient -------------------------------------------------------

@pytest.mark.parametrize("T,M", [(1, 1), (1, 7), (3, 5), (33, 1001), (64, 4096)])
@pytest.mark.parametrize("remake", [False, True])
def test_gated_backward(T, M, remake):
    import torch
    import boolean_weight_matmul_b200 as mb
    rng = np.random.default_rng(T * M)
    host = [rng.standard_normal((T, M)) * s for s in (0.3, 4.0, 2.0)]
    host[1].flat[0] = -100.0
    host[1].flat[-1] = 90.0
    dev = [torch.from_numpy(a).to(torch.bfloat16).cuda() for a in host]
    dh, g, u = (_f64(t) for t in dev)
    out = [guarded((T, M), torch.bfloat16) for _ in range(3)]
    mb.gated_backward(*dev, T, M, out[0], out[1], out[2] if remake else None)
    torch.cuda.synchronize()
    dg, du, h, E = F.gated_grad(dh, g, u)
    # the exponential and the reciprocal: a few fp32 steps and |g| 2^-23 of each term
    rel = 2.0 ** -20 + np.abs(g) * 2.0 ** -22
    tiny = 1e-36   # a sigmoid below 2^-126 may come out as 0
    _assert_within(_f64(out[0]), dg, E * rel + np.abs(dg) * HALF["bf16"] + tiny, "dgate")
    _assert_within(_f64(out[1]), du, np.abs(du) * (rel + HALF["bf16"]) + tiny, "dup")
    if remake:
        _assert_within(_f64(out[2]), h, np.abs(h) * (rel + HALF["bf16"]) + tiny, "h")


def test_gated_backward_in_place_and_differences():
    import torch
    import boolean_weight_matmul_b200 as mb
    rng = np.random.default_rng(5)
    T, M = 9, 123
    dh, g, u = (torch.from_numpy(rng.standard_normal((T, M))).to(torch.bfloat16).cuda() for _ in range(3))
    a, b, c = (torch.empty_like(g) for _ in range(3))
    mb.gated_backward(dh, g, u, T, M, a, b, c)
    x, y, z = dh.clone(), g.clone(), u.clone()
    mb.gated_backward(x, y, z, T, M, y, z, x)
    torch.cuda.synchronize()
    assert torch.equal(a, y) and torch.equal(b, z) and torch.equal(c, x)
    # against central differences of the formula
    G, U, D = _f64(g), _f64(u), _f64(dh)
    eps = 1e-5
    dg = D * (F.silu(G + eps) - F.silu(G - eps)) * U / (2 * eps)
    _assert_within(_f64(a), dg, np.abs(dg) * (HALF["bf16"] + 1e-4) + 1e-6)


# ---- distillation --------------------------------------------------------------

def _distill_case(T, V, top, seed, dtype, masked=True, ld=None):
    import torch
    rng = np.random.default_rng(seed)
    ld = V if ld is None else ld
    z = torch.from_numpy(rng.standard_normal((T, ld)) * 3).to(_dt(dtype))
    teacher = (rng.standard_normal((T, top)) * 2 + 4).astype(np.float32)
    index = np.stack([rng.permutation(V)[:top] if top <= V else rng.integers(0, V, top) for _ in range(T)]).astype(np.int32)
    weight = rng.uniform(0.5, 1.5, T).astype(np.float32)
    grad = rng.uniform(0.5, 1.5, T).astype(np.float32)
    if masked and T > 3:
        weight[1] = 0.0
        index[2] = -1
        index[3, top // 2:] = V + 5
        teacher[0, 0] = -np.inf
    return z, teacher, index, weight, grad


def _check_distill(z, teacher, index, weight, grad, tau, V, dtype, got_loss, got_lse, got_dz):
    z64 = z[:, :V].double().numpy()
    loss, lse, dz, q, p = F.distill(z64, teacher.astype(np.float64), index, tau, weight.astype(np.float64),
                                    grad.astype(np.float64))
    live = lse != 0
    y = np.where(np.isfinite(z64), z64, 0) / tau
    span = (np.abs(y).max(1) + np.abs(lse) + np.abs(teacher[np.isfinite(teacher)]).max() / tau + 8)
    # every exponent and logarithm is off by a few fp32 steps of its size: 2^-22 of the row's span
    _assert_within(got_lse, lse, np.where(live, span * 2.0 ** -22, 0), "lse")
    _assert_within(got_loss, loss, np.where(live, np.abs(weight) * span * 2.0 ** -21, 0), "loss")
    scale = np.abs(grad * weight / tau)[:, None]
    tol = scale * (q + p) * (span * 2.0 ** -21)[:, None] + np.abs(dz) * HALF[dtype] + 1e-38
    _assert_within(got_dz, dz, np.where(live[:, None], tol, 0), "dz")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,top,tau", [(1, 1, 1, 1.0), (5, 7, 3, 2.0), (9, 1000, 16, 1.0), (4, 32001, 64, 2.0),
                                         (6, 4099, 512, 3.5), (2, 128000, 20, 1.0), (5, 40, 64, 0.5)])
def test_distill(dtype, T, V, top, tau):
    import torch
    import boolean_weight_matmul_b200 as mb
    z, teacher, index, weight, grad = _distill_case(T, V, top, T + V + top, dtype)
    zd = z.cuda()
    td, xd, wd, gd = to_dev(teacher), to_dev(index), to_dev(weight), to_dev(grad)
    loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
    dz = guarded((T, V), _dt(dtype))
    mb.distill_loss(zd, _code(dtype), T, V, V, td, xd, top, tau, wd, loss, lse, dz, V)
    torch.cuda.synchronize()
    ones = np.ones_like(grad)
    _check_distill(z, teacher, index, weight, ones, tau, V, dtype, _f64(loss), _f64(lse), _f64(dz))
    # the loss alone, then the gradient from its lse
    loss2, lse2, dz2 = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), _dt(dtype))
    mb.distill_loss(zd, _code(dtype), T, V, V, td, xd, top, tau, wd, loss2, lse2)
    mb.distill_backward(zd, _code(dtype), T, V, V, td, xd, top, tau, wd, lse2, gd, dz2, V)
    torch.cuda.synchronize()
    _check_distill(z, teacher, index, weight, grad, tau, V, dtype, _f64(loss2), _f64(lse2), _f64(dz2))
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_strides_and_in_place(dtype):
    # rows that start anywhere in a 16-byte line, gradient rows with another
    # offset, what lies between the rows left as it was, and the gradient in place
    import torch
    import boolean_weight_matmul_b200 as mb
    T, V, top, tau = 7, 2053, 9, 2.0
    z, teacher, index, weight, grad = _distill_case(T, V, top, 3, dtype, ld=V + 4)
    td, xd, wd = to_dev(teacher), to_dev(index), to_dev(weight)
    loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
    ones = np.ones_like(grad)
    for ld_dz in (V, V + 3, V + 4):
        buf = torch.full((T, ld_dz), 7.0, dtype=_dt(dtype), device="cuda")
        mb.distill_loss(z.cuda(), _code(dtype), T, V, V + 4, td, xd, top, tau, wd, loss, lse, buf, ld_dz)
        torch.cuda.synchronize()
        _check_distill(z, teacher, index, weight, ones, tau, V, dtype, _f64(loss), _f64(lse), _f64(buf[:, :V]))
        assert (buf[:, V:] == 7.0).all()
    zd = z.cuda()
    mb.distill_loss(zd, _code(dtype), T, V, V + 4, td, xd, top, tau, wd, loss, lse, zd, V + 4)
    torch.cuda.synchronize()
    assert torch.equal(zd[:, :V], buf[:, :V]) and torch.equal(zd[:, V:].cpu(), z[:, V:])
    zd = z.cuda()
    mb.distill_backward(zd, _code(dtype), T, V, V + 4, td, xd, top, tau, wd, lse, None, zd, V + 4)
    torch.cuda.synchronize()
    _check_distill(z, teacher, index, weight, ones, tau, V, dtype, _f64(loss), _f64(lse), _f64(zd[:, :V]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_same_index_twice_and_masked_logits(dtype):
    import torch
    import boolean_weight_matmul_b200 as mb
    T, V, top, tau = 4, 600, 12, 1.0
    z, teacher, index, weight, grad = _distill_case(T, V, top, 4, dtype, masked=False)
    index[:, 5] = index[:, 2]
    index[:, 7] = index[:, 2]
    free = np.setdiff1d(np.arange(V), index.ravel())
    z[0, free] = float("-inf")                       # masked by -infinity
    z[1, free] = torch.finfo(z.dtype).min            # masked by the lowest value
    z[2, free[:300]] = float("-inf")
    td, xd = to_dev(teacher), to_dev(index)
    loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
    ones = np.ones(T, dtype=np.float32)
    dz = guarded((T, V), _dt(dtype))
    mb.distill_loss(z.cuda(), _code(dtype), T, V, V, td, xd, top, tau, None, loss, lse, dz, V)
    torch.cuda.synchronize()
    clean = z.clone()
    clean[1, free] = float("-inf")
    _check_distill(clean, teacher, index, ones, ones, tau, V, dtype, _f64(loss), _f64(lse), _f64(dz))
    mb.distill_backward(z.cuda(), _code(dtype), T, V, V, td, xd, top, tau, None, lse, None, dz, V)
    torch.cuda.synchronize()
    _check_distill(clean, teacher, index, ones, ones, tau, V, dtype, _f64(loss), _f64(lse), _f64(dz))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_wide_rows(dtype):
    # wider than a cluster's registers: the loss in several passes, the gradient from memory
    import torch
    import boolean_weight_matmul_b200 as mb
    T, V, top, tau = 2, 300001, 5, 1.0
    z, teacher, index, weight, grad = _distill_case(T, V, top, 6, dtype, masked=False)
    loss, lse, dz = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), _dt(dtype))
    mb.distill_loss(z.cuda(), _code(dtype), T, V, V, to_dev(teacher), to_dev(index), top, tau, to_dev(weight), loss,
                    lse, dz, V)
    torch.cuda.synchronize()
    _check_distill(z, teacher, index, weight, np.ones_like(grad), tau, V, dtype, _f64(loss), _f64(lse), _f64(dz))


def test_distill_rows_without_use():
    # no weight or nothing listed: zeros, whatever the logits hold; NaN logits elsewhere stay in their row
    import torch
    import boolean_weight_matmul_b200 as mb
    T, V, top = 5, 333, 4
    z, teacher, index, weight, grad = _distill_case(T, V, top, 8, "f32", masked=False)
    z[0, 3] = float("nan")
    z[1, :] = float("nan")
    z[2, :] = float("-inf")
    weight[0] = 0.0
    index[1] = -1
    loss, lse, dz = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), torch.float32)
    mb.distill_loss(z.cuda(), mb.F32, T, V, V, to_dev(teacher), to_dev(index), top, 1.0, to_dev(weight), loss, lse, dz, V)
    torch.cuda.synchronize()
    for t in (0, 1):
        assert loss[t] == 0 and lse[t] == 0 and (dz[t] == 0).all()
    assert torch.isnan(loss[2]) and torch.isnan(dz[2]).all()
    assert torch.isfinite(dz[3:]).all() and torch.isfinite(loss[3:]).all()


def test_distill_gradient_against_differences():
    import torch
    import boolean_weight_matmul_b200 as mb
    T, V, top, tau = 2, 50, 6, 2.0
    z, teacher, index, weight, grad = _distill_case(T, V, top, 12, "f32", masked=False)
    loss, lse, dz = (torch.empty(s, device="cuda") for s in ((T,), (T,), (T, V)))
    mb.distill_loss(z.cuda(), mb.F32, T, V, V, to_dev(teacher), to_dev(index), top, tau, to_dev(weight), loss, lse, dz, V)
    torch.cuda.synchronize()
    z64, eps = z.double().numpy(), 1e-5
    one = np.ones(T)
    for j in range(V):
        hi, lo = z64.copy(), z64.copy()
        hi[:, j] += eps
        lo[:, j] -= eps
        args = (teacher.astype(np.float64), index, tau, weight.astype(np.float64), one)
        d = (F.distill(hi, *args)[0] - F.distill(lo, *args)[0]) / (2 * eps)
        _assert_within(_f64(dz[:, j]), d, 1e-6)


# ---- gated feed-forward over tokens ---------------------------------------------

def _dense_abs(layer):
    a = np.repeat(layer.alpha.astype(np.float64), 128, axis=1)
    return np.einsum("mnk,kmn->mn", a, F.planes(layer.words, layer.K, layer.M, layer.N))


def _fp16_weights_tol(absx, W, n):
    # Each level is rounded once to fp16: half a step 2^-11 of it, or 2^-23 where
    # it is below 2^-12.  The tensor cores add 16 products at a time into an fp32
    # sum that they may truncate: a full step 2^-23 per addition, n / 16 + 16 deep.
    # Scaled activations are off by at most 2^-40 of their token's largest.
    E = absx @ np.abs(W).T
    return E * (2.0 ** -11 + (n / 16 + 16) * 2.0 ** -23) + absx.sum(1, keepdims=True) * 2.0 ** -23 + \
        absx.max(1, keepdims=True) * 2.0 ** -40 * np.abs(W).sum(1)[None, :]


def _gemm_gated(gate, up, X, keep, ws=None):
    import torch
    import boolean_weight_matmul_b200 as mb
    T = X.shape[0]
    out = [guarded((T, gate.M), torch.bfloat16) for _ in range(3)]
    if ws is None:
        ws = mb.empty_gemm_gated_workspace(gate.M, gate.N, T)
        ws.fill_(0xFF)
    mb.gemm_gated(gate.packed, gate.blocked, gate.K, up.packed, up.blocked, up.K, gate.M, gate.N, 128, X, T, out[0],
                  out[1] if keep else None, out[2] if keep else None, ws)
    torch.cuda.synchronize()
    assert mb.read_device_errors() == 0
    return out


def _check_gated(gate, up, x64, got, keep):
    Wg, Wu, ax = _dense_abs(gate), _dense_abs(up), np.abs(x64)
    g, u = x64 @ Wg.T, x64 @ Wu.T
    tg, tu = _fp16_weights_tol(ax, Wg, gate.N), _fp16_weights_tol(ax, Wu, gate.N)
    h = F.silu(g) * u
    # bf16's smallest value is 2^-133: a result near or below it is off by up to half of that, 2^-134, whatever
    # its relative bound (the products of two 1e-30 tokens are 1e-64 and come out as 0)
    tg, tu = tg + 2.0 ** -134, tu + 2.0 ** -134
    th = 1.01 * (1.1 * np.abs(u) * tg + np.abs(F.silu(g)) * tu + 1.1 * tg * tu) + \
        np.abs(h) * (2.0 ** -20 + np.abs(g) * 2.0 ** -23 + HALF["bf16"]) + 2.0 ** -134
    _assert_within(_f64(got[0]), h, th, "H")
    if keep:
        _assert_within(_f64(got[1]), g, tg + np.abs(g) * HALF["bf16"], "gate")
        _assert_within(_f64(got[2]), u, tu + np.abs(u) * HALF["bf16"], "up")


@pytest.mark.parametrize("kg,ku", [(1, 1), (2, 4), (3, 3), (4, 1)])
@pytest.mark.parametrize("M,N,T", [(128, 128, 32), (1, 128, 1), (7, 256, 17), (200, 640, 77), (1001, 384, 130),
                                   (64, 2048, 300), (136, 128, 700)])
def test_gemm_gated(kg, ku, M, N, T):
    gate, up = Layer(kg, M, N, 500 + kg + M, pad_nan=True), Layer(ku, M, N, 600 + ku + N, pad_nan=True)
    x, x64 = _x(T, N, 700 + T, "bf16")
    for keep in (True, False):
        _check_gated(gate, up, x64, _gemm_gated(gate, up, x_dev(x, "bf16"), keep), keep)


def test_gemm_gated_many_tiles():
    # more tiles than pairs of CTAs: every pair reuses its accumulators
    gate, up = Layer(3, 1500, 256, 31), Layer(2, 1500, 256, 32)
    x, x64 = _x(4100, 256, 33, "bf16")
    _check_gated(gate, up, x64, _gemm_gated(gate, up, x_dev(x, "bf16"), True), True)


@pytest.mark.parametrize("M,N,T", [(101, 2304, 633), (136, 2304, 21), (100, 4096, 300), (9600, 2048, 5)])
def test_gemm_gated_cut_tiles(M, N, T):
    # few or unevenly many tiles: runs of stages begin and end inside tiles, whose parts are added
    import torch
    import boolean_weight_matmul_b200 as mb
    up = lambda n, m: (n + m - 1) // m * m
    assert mb.gemm_gated_workspace_bytes(M, N, T) > up(T * N * 2, 256) + up(up(T, 16) * 4, 256)
    gate, upm = Layer(3, M, N, 131, pad_nan=True), Layer(2, M, N, 132, pad_nan=True)
    x, x64 = _x(T, N, 133, "bf16")
    X = x_dev(x, "bf16")
    got = _gemm_gated(gate, upm, X, True)
    _check_gated(gate, upm, x64, got, True)
    again = _gemm_gated(gate, upm, X, False)
    assert torch.equal(again[0], got[0])


def test_gemm_gated_activation_range():
    # tokens of very different size, zeros, subnormals, infinities and NaN: a token's scale is its own
    import torch
    gate, up = Layer(2, 40, 256, 41), Layer(1, 40, 256, 42)
    rng = np.random.default_rng(43)
    x = rng.standard_normal((12, 256))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3] *= 2.0 ** -130
    x[4, 3], x[5, 7], x[6, 9] = np.inf, -np.inf, np.nan
    x[7, ::2] *= 1e-6
    X = torch.from_numpy(x).to(torch.bfloat16).cuda()
    x64 = _f64(X)
    got = _gemm_gated(gate, up, X, True)
    finite = [t for t in range(12) if t not in (0, 4, 5, 6)]
    _check_gated(gate, up, x64[finite], [o[finite] for o in got], True)
    # the large token's projections (their product overflows)
    Wg, Wu = _dense_abs(gate), _dense_abs(up)
    for o, W in ((got[1], Wg), (got[2], Wu)):
        _assert_within(_f64(o[:1]), x64[:1] @ W.T, _fp16_weights_tol(np.abs(x64[:1]), W, 256) +
                       np.abs(x64[:1] @ W.T) * HALF["bf16"])
    assert not torch.isfinite(got[1][4]).any() and not torch.isfinite(got[1][5]).any() and torch.isnan(got[1][6]).all()


# ---- backward pass of layers that share X ---------------------------------------

def _unblock(a, K, M, N):
    """fp32 [M][G][K] from the scales' layout [octet][group][kernel][8]."""
    return a.reshape(-1, N // 128, K, 8).transpose(0, 3, 1, 2).reshape(-1, N // 128, K)[:M]


def _grads(T, M, seed, scale=1e-2):
    import torch
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((T, M)) * scale).to(torch.bfloat16).cuda()


def _gemm_backward(layers, X, dYs, want_x=True, want_a=None, ws=None):
    import torch
    import boolean_weight_matmul_b200 as mb
    T, N = X.shape
    Ks, Ms = [m.K for m in layers], [m.M for m in layers]
    want_a = [True] * len(layers) if want_a is None else want_a
    dX = guarded((T, N), torch.bfloat16) if want_x else None
    das = [guarded((mb.alpha_elems(m.K, m.M, N),), torch.float32) if w else None for m, w in zip(layers, want_a)]
    if ws is None:
        ws = mb.empty_gemm_backward_workspace(Ks, Ms, N, T)
        ws.fill_(0xFF)
    mb.gemm_backward([m.packed for m in layers], [m.blocked for m in layers], Ks, Ms, N, 128, X, T, dYs, dX, das, ws)
    torch.cuda.synchronize()
    assert mb.read_device_errors() == 0
    return dX, das


def _check_backward(layers, X, dYs, dX, das):
    N, T = X.shape[1], X.shape[0]
    x64, dy64 = _f64(X), [_f64(d) for d in dYs]
    want, _, wa = F.layer_grad([m.host() for m in layers], N, x64, dy64)
    if dX is not None:
        tol = np.abs(want) * HALF["bf16"]
        rows = sum(m.M for m in layers)
        top = np.max([np.abs(d).max(1) for d in dy64], axis=0)[:, None]   # one scale per token
        for m, d in zip(layers, dy64):
            W = _dense_abs(m)
            E = np.abs(d) @ np.abs(W)
            tol = tol + E * (2.0 ** -11 + (rows / 16 + 16 * len(layers) + 16) * 2.0 ** -23) + \
                np.abs(d).sum(1, keepdims=True) * 2.0 ** -23 + top * 2.0 ** -40 * np.abs(W).sum(0)[None, :]
        _assert_within(_f64(dX), want, tol, "dX")
    for m, da, (w, E) in zip(layers, das, wa):
        if da is None:
            continue
        blocked = da.cpu().numpy()
        got = _unblock(blocked, m.K, m.M, N)
        # exact products; at most 64 tensor-core steps a run, then 32 + 8 fp32 additions and one per run or split
        tol = E * (min(T, 1024) / 16 + 16) * 2.0 ** -23 + E * (48 + T / 256) * 2.0 ** -24
        _assert_within(got, w, tol, "dalpha")
        pad = blocked.reshape(-1, N // 128, m.K, 8)[-1, :, :, m.M % 8:] if m.M % 8 else np.zeros(1)
        assert (pad == 0).all()


@pytest.mark.parametrize("spec", [[(1, 1)], [(3, 7)], [(2, 64)], [(4, 200)], [(3, 136), (2, 77)],
                                  [(2, 200), (1, 77), (3, 77)], [(1, 8), (2, 9), (3, 65), (4, 130), (1, 300), (2, 1),
                                                                 (3, 64), (4, 15)]])
@pytest.mark.parametrize("N,T", [(128, 1), (256, 33), (640, 130)])
def test_gemm_backward(spec, N, T):
    layers = [Layer(K, M, N, 50 + 7 * i + M, pad_nan=True) for i, (K, M) in enumerate(spec)]
    X = x_dev(wl.x_normal(T, N, 60 + T), "bf16")
    dYs = [_grads(T, m.M, 70 + i) for i, m in enumerate(layers)]
    dX, das = _gemm_backward(layers, X, dYs)
    _check_backward(layers, X, dYs, dX, das)


@pytest.mark.parametrize("M,N,T", [(300, 384, 2500), (1500, 1280, 300), (513, 2304, 1100)])
def test_gemm_backward_runs_splits_and_tiles(M, N, T):
    # several token runs, token splits, more tiles than pairs
    layers = [Layer(3, M, N, 81), Layer(2, 40, N, 82)]
    X = x_dev(wl.x_normal(T, N, 83), "bf16")
    dYs = [_grads(T, m.M, 84 + i) for i, m in enumerate(layers)]
    first = _gemm_backward(layers, X, dYs)
    _check_backward(layers, X, dYs, *first)
    import torch
    again = _gemm_backward(layers, X, dYs)
    assert torch.equal(first[0], again[0]) and all(torch.equal(a, b) for a, b in zip(first[1], again[1]))


@pytest.mark.parametrize("spec,N,T", [([(2, 2764)], 128, 235), ([(2, 1499), (3, 213), (3, 64)], 1408, 21),
                                      ([(1, 700), (4, 1300)], 256, 400)])
def test_gemm_backward_cut_tiles(spec, N, T):
    # as above, runs that begin and end in different matrices
    import torch
    import boolean_weight_matmul_b200 as mb
    Ks, Ms = [k for k, _ in spec], [m for _, m in spec]
    up = lambda n, m: (n + m - 1) // m * m
    base = sum(up(T * up(m, 8) * 2, 256) * (2 if m % 8 else 1) for m in Ms) + up(up(T, 16) * 4, 256)
    assert mb.gemm_backward_workspace_bytes(Ks, Ms, N, T) > base
    layers = [Layer(k, m, N, 141 + i, pad_nan=True) for i, (k, m) in enumerate(spec)]
    X = x_dev(wl.x_normal(T, N, 143), "bf16")
    dYs = [_grads(T, m.M, 144 + i) for i, m in enumerate(layers)]
    first = _gemm_backward(layers, X, dYs)
    _check_backward(layers, X, dYs, *first)
    again = _gemm_backward(layers, X, dYs, want_a=[False] * len(spec))
    assert torch.equal(first[0], again[0])


def test_gemm_backward_parts():
    # dX alone (no X needed), scales alone, one matrix's scales frozen: the same bits as all together
    import torch
    import boolean_weight_matmul_b200 as mb
    N, T = 512, 90
    layers = [Layer(2, 100, N, 91), Layer(3, 64, N, 92)]
    X = x_dev(wl.x_normal(T, N, 93), "bf16")
    dYs = [_grads(T, m.M, 94 + i) for i, m in enumerate(layers)]
    dX, das = _gemm_backward(layers, X, dYs)
    only_a = _gemm_backward(layers, X, dYs, want_x=False)
    frozen = _gemm_backward(layers, X, dYs, want_a=[False, True])
    assert all(torch.equal(a, b) for a, b in zip(das, only_a[1]))
    assert torch.equal(frozen[0], dX) and torch.equal(frozen[1][1], das[1])
    alone = guarded((T, N), torch.bfloat16)
    ws = mb.empty_gemm_backward_workspace([2, 3], [100, 64], N, T)
    mb.gemm_backward([m.packed for m in layers], [m.blocked for m in layers], [2, 3], [100, 64], N, 128, None, T, dYs,
                     alone, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(alone, dX)


def test_gemm_backward_range():
    # gradients far below and above one, zero rows, an infinity and a NaN that stay in their token
    import torch
    N, T = 256, 20
    layers = [Layer(3, 72, N, 101)]
    X = x_dev(wl.x_normal(T, N, 102), "bf16")
    d = _grads(T, 72, 103)
    d[0] *= 1e-30
    d[1] *= 1e30
    d[2] = 0
    clean = d.clone()
    d[3, 5], d[4, 6] = float("inf"), float("nan")
    dX, _ = _gemm_backward(layers, X, [d], want_a=[False])
    keep = [t for t in range(T) if t not in (3, 4)]
    _check_backward(layers, X[keep].contiguous(), [clean[keep].contiguous()], dX[keep], [None])
    assert not torch.isfinite(dX[3]).any() and torch.isnan(dX[4]).all()


def test_gemm_backward_against_differences():
    # the scales' gradient by the definition: move one scale, take the difference of sum(dY * Y)
    K, M, N, T = 2, 16, 256, 40
    layer = Layer(K, M, N, 111)
    X = x_dev(wl.x_normal(T, N, 112), "bf16")
    dY = _grads(T, M, 113)
    _, (da,) = _gemm_backward([layer], X, [dY])
    got = _unblock(da.cpu().numpy(), K, M, N)
    x64, d64 = _f64(X), _f64(dY)
    for r, g, k in ((0, 0, 0), (5, 1, 1), (15, 0, 1)):
        vals = []
        for sign in (1, -1):
            a = layer.alpha.astype(np.float64).copy()
            a[r, g, k] += sign * 1e-3
            vals.append((d64 * F.project(layer.words, a, K, M, N, x64)[0]).sum())
        want = (vals[0] - vals[1]) / 2e-3
        assert abs(got[r, g, k] - want) <= 1e-4 * max(1.0, abs(want))


# ---- a run of them together -------------------------------------------------------

def test_block_training_step():
    # gated block -> down projection -> output layer -> distillation, and back to every scale and the input
    import torch
    import boolean_weight_matmul_b200 as mb
    T, D, M, V, top, tau = 48, 256, 384, 640, 8, 2.0
    gate, up, down, head = Layer(2, M, D, 121), Layer(3, M, D, 122), Layer(2, D, M, 123), Layer(3, V, D, 124)
    x, x64 = _x(T, D, 125, "bf16")
    X = x_dev(x, "bf16")
    H, G, U = _gemm_gated(gate, up, X, True)
    Y = guarded((T, D), torch.bfloat16)
    mb.gemm(down.packed, down.blocked, down.K, D, M, 128, H, T, Y, precision=mb.GEMM_SPLIT)
    Z = guarded((T, V), torch.bfloat16)
    mb.gemm(head.packed, head.blocked, head.K, V, D, 128, Y, T, Z, precision=mb.GEMM_SPLIT)
    _, teacher, index, weight, _ = _distill_case(T, V, top, 126, "bf16")
    loss, lse, dZ = guarded((T,), torch.float32), guarded((T,), torch.float32), guarded((T, V), torch.bfloat16)
    mb.distill_loss(Z, mb.BF16, T, V, V, to_dev(teacher), to_dev(index), top, tau, to_dev(weight), loss, lse, dZ, V)
    torch.cuda.synchronize()
    dY, (da_head,) = _gemm_backward([head], Y, [dZ])
    dH, (da_down,) = _gemm_backward([down], H, [dY])
    dG, dU, H2 = (guarded((T, M), torch.bfloat16) for _ in range(3))
    mb.gated_backward(dH, G, U, T, M, dG, dU, H2)
    dX, (da_gate, da_up) = _gemm_backward([gate, up], X, [dG, dU])
    torch.cuda.synchronize()
    # the same step in fp64 from the same inputs: every bf16 rounding on the way adds its half step, about
    # sqrt(8) x 2^-8 of a result's size after eight of them
    f = lambda layer, a: a @ _dense_abs(layer).T
    g, u = f(gate, x64), f(up, x64)
    h = F.silu(g) * u
    y = f(down, h)
    z = f(head, y)
    _, _, dz, _, _ = F.distill(z, teacher.astype(np.float64), index, tau, weight.astype(np.float64), np.ones(T))
    dy, _, ((a_head, _),) = F.layer_grad([head.host()], D, y, [dz])
    dh, _, ((a_down, _),) = F.layer_grad([down.host()], M, h, [dy])
    dg, du, _, _ = F.gated_grad(dh, g, u)
    dx, _, ((a_gate, _), (a_up, _)) = F.layer_grad([gate.host(), up.host()], D, x64, [dg, du])
    rel = lambda got, want: np.linalg.norm(got - want) / np.linalg.norm(want)
    for name, got, want in (("dX", _f64(dX), dx),
                            ("head", _unblock(da_head.cpu().numpy(), 3, V, D), a_head),
                            ("down", _unblock(da_down.cpu().numpy(), 2, D, M), a_down),
                            ("gate", _unblock(da_gate.cpu().numpy(), 2, M, D), a_gate),
                            ("up", _unblock(da_up.cpu().numpy(), 3, M, D), a_up)):
        assert rel(got, want) <= 8 ** 0.5 * 2.0 ** -8, (name, rel(got, want))


def test_gemm_calls_captured_and_on_another_stream():
    import torch
    import boolean_weight_matmul_b200 as mb
    gate, up = Layer(3, 200, 512, 131), Layer(2, 200, 512, 132)
    T = 70
    X = x_dev(wl.x_normal(T, 512, 133), "bf16")
    want = [t.clone() for t in _gemm_gated(gate, up, X, True)]
    dYs = [_grads(T, 200, 134), _grads(T, 200, 135)]
    bwd = _gemm_backward([gate, up], X, dYs)
    ws, wb = mb.empty_gemm_gated_workspace(200, 512, T), mb.empty_gemm_backward_workspace([3, 2], [200, 200], 512, T)
    out = [torch.zeros_like(t) for t in want]
    dX, das = torch.zeros_like(bwd[0]), [torch.zeros_like(a) for a in bwd[1]]

    def calls():
        mb.gemm_gated(gate.packed, gate.blocked, 3, up.packed, up.blocked, 2, 200, 512, 128, X, T, *out, ws)
        mb.gemm_backward([gate.packed, up.packed], [gate.blocked, up.blocked], [3, 2], [200, 200], 512, 128, X, T, dYs,
                         dX, das, wb)

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.equal(dX, bwd[0]) and all(torch.equal(a, b) for a, b in zip(das, bwd[1]))
        for t in (*out, dX, *das):
            t.zero_()
        torch.cuda.synchronize()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        graph.replay()
        check()


@pytest.mark.parametrize("dtype,V,T", [("bf16", 2053, 1300), ("f32", 1000, 700), ("bf16", 8, 610), ("f32", 3, 600)])
def test_distill_many_rows(dtype, V, T):
    # more rows than SMs keep in flight, rows of every alignment, masked rows among them; fused, in place and apart
    import torch
    import boolean_weight_matmul_b200 as mb
    top, tau = min(V, 24), 2.0
    z, teacher, index, weight, grad = _distill_case(T, V, top, 21, dtype)
    weight[::7] = 0.0
    # rows far from zero on either side, and rows where most logits are masked
    z[4::9] += 300.0
    z[5::9] -= 300.0
    listed = torch.zeros(T, V, dtype=torch.bool)
    rows = torch.arange(T)[:, None].expand(T, top)
    ok = torch.from_numpy((index >= 0) & (index < V))
    listed[rows[ok], torch.from_numpy(index)[ok].long()] = True
    z[6::9] = torch.where(listed[6::9], z[6::9], torch.full_like(z[6::9], float("-inf")))
    td, xd, wd = to_dev(teacher), to_dev(index), to_dev(weight)
    loss, lse = guarded((T,), torch.float32), guarded((T,), torch.float32)
    ones = np.ones_like(grad)
    for ld_dz in (V, V + 1):
        buf = torch.full((T, ld_dz), 7.0, dtype=_dt(dtype), device="cuda")
        mb.distill_loss(z.cuda(), _code(dtype), T, V, V, td, xd, top, tau, wd, loss, lse, buf, ld_dz)
        torch.cuda.synchronize()
        assert mb.read_device_errors() == 0
        _check_distill(z, teacher, index, weight, ones, tau, V, dtype, _f64(loss), _f64(lse), _f64(buf[:, :V]))
        assert (buf[:, V:] == 7.0).all()
        if ld_dz == V:
            first = buf.clone()
    zd = z.cuda()
    mb.distill_loss(zd, _code(dtype), T, V, V, td, xd, top, tau, wd, loss, lse, zd, V)
    torch.cuda.synchronize()
    assert torch.equal(zd, first)


def _call_set(seed, T=150, batch=6):
    """One of each call on inputs of a seed: functions that issue them, their outputs and what they read."""
    import torch
    import boolean_weight_matmul_b200 as mb
    M, N, V = 333, 2304, 3000
    gate, up = Layer(3, M, N, 151), Layer(2, M, N, 152)
    X = x_dev(wl.x_normal(T, N, seed), "bf16")
    x = x_dev(wl.x_normal(batch, N, seed + 1), "bf16")
    dYs = [_grads(T, M, seed + 2), _grads(T, M, seed + 3)]
    Z = _grads(T, V, seed + 4, 2.0)
    rng = np.random.default_rng(seed + 5)
    teacher = to_dev(rng.standard_normal((T, 8)).astype(np.float32))
    index = to_dev(rng.integers(0, V, (T, 8)).astype(np.int32))
    e = lambda *shape, dt=torch.bfloat16: torch.zeros(shape, dtype=dt, device="cuda")
    H, G, U, h, dX, dZ = e(T, M), e(T, M), e(T, M), e(batch, M), e(T, N), e(T, V)
    das = [e(mb.alpha_elems(3, M, N), dt=torch.float32), e(mb.alpha_elems(2, M, N), dt=torch.float32)]
    loss, lse = e(T, dt=torch.float32), e(T, dt=torch.float32)
    dG, dU = e(T, M), e(T, M)
    packed, alpha = [gate.packed, up.packed], [gate.blocked, up.blocked]

    def issue(ws):
        mb.gemm_gated(gate.packed, gate.blocked, 3, up.packed, up.blocked, 2, M, N, 128, X, T, H, G, U, ws[0])
        mb.gemv_gated(gate.packed, gate.blocked, 3, up.packed, up.blocked, 2, M, N, 128, x, mb.BF16, batch, h, mb.BF16,
                      ws[1])
        mb.gated_backward(dYs[0], G, U, T, M, dG, dU)
        mb.gemm_backward(packed, alpha, [3, 2], [M, M], N, 128, X, T, [dG, dYs[1]], dX, das, ws[2])
        mb.distill_loss(Z, mb.BF16, T, V, V, teacher, index, 8, 1.5, None, loss, lse, dZ, V)

    space = lambda: (mb.empty_gemm_gated_workspace(M, N, T), mb.empty_gated_workspace(3, 2, M, N, batch),
                     mb.empty_gemm_backward_workspace([3, 2], [M, M], N, T))
    return issue, [H, G, U, h, dG, dU, dX, *das, loss, lse, dZ], [X, x, *dYs, Z], space


def test_calls_back_to_back_and_on_two_streams():
    # launches that start before the preceding grid ends: two sets of calls in turn through one workspace, inputs
    # overwritten right behind the calls, and two streams at once each with its own; always the bits of a call alone
    import torch
    import boolean_weight_matmul_b200 as mb
    sets = [_call_set(161), _call_set(171)]
    want = []
    for issue, outs, _, space in sets:
        issue(space())
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])

    def check():
        torch.cuda.synchronize()
        assert mb.read_device_errors() == 0
        for (_, outs, _, _), w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w))
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()

    shared = sets[0][3]()
    for _ in range(5):
        for issue, *_ in sets:
            issue(shared)
    check()
    kept = [[t.clone() for t in ins] for _, _, ins, _ in sets]
    for issue, _, ins, _ in sets:
        issue(shared)
        for t in ins:
            t.fill_(float("nan"))
    check()
    for (_, _, ins, _), k in zip(sets, kept):
        for t, v in zip(ins, k):
            t.copy_(v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [s[3]() for s in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for (issue, *_), stream, ws in zip(sets, streams, spaces):
            with torch.cuda.stream(stream):
                issue(ws)
    check()
    # captured together, replayed twice
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for issue, *_ in sets:
            issue(shared)
    for _ in range(2):
        graph.replay()
        check()


def test_marshalled_calls_check_tensors_and_take_streams():
    import torch
    import boolean_weight_matmul_b200 as mb
    T, M = 12, 40
    a = [_grads(T, M, 181 + i) for i in range(3)]
    out = [torch.zeros_like(a[0]) for _ in range(2)]
    mb.gated_backward(*a, T, M, *out)
    torch.cuda.synchronize()
    want = [o.clone() for o in out]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, None):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        mb.gated_backward(*a, T, M, *out, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    wide = torch.zeros((T, 2 * M), dtype=torch.bfloat16, device="cuda")[:, :M]
    with pytest.raises(ValueError):
        mb.gated_backward(wide, a[1], a[2], T, M, *out)
    with pytest.raises(ValueError):
        mb.gated_backward(a[0].cpu(), a[1], a[2], T, M, *out)
    with torch.cuda.stream(side):                               # the current stream, while another one is busy
        mb.gated_backward(a[0].data_ptr(), a[1], a[2], T, M, *out)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, want))
