"""The feed-forward operators at their limits: operands above 4 GiB, pitches just
below 2^23, tensors of more than 2^31 elements in a clip list, two calls at
once on two streams, and lists and captures that are refused."""
import math

import pytest
import torch

import ffn_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu


def randn(gen, *shape, std=1.0, dt=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dt).mul_(std)


def pick(n, k):
    """k indices of 0 .. n - 1, the first and last ones among them."""
    return torch.unique(torch.linspace(0, n - 1, k, device="cuda").round().long())


def test_operands_above_4_gib():
    M, N, K = 65541, 40, 36000   # A and dA: 4.7 GB each
    gen = torch.Generator(device="cuda").manual_seed(1)
    A = randn(gen, M, K)
    Bs = [randn(gen, K, N, std=K ** -0.5) for _ in range(2)]
    r = pick(M, 300)
    H, Z = mk.gated_gemm_train(A, *Bs, act="silu")
    v, e, zg, zu = ref.gated(A[r], *Bs, None, None, "silu", A.dtype)
    ref.check(H[r], (v, e), "H")
    ref.check(Z[0][r], zg, "Zg")
    ref.check(Z[1][r], zu, "Zu")
    progress("forward")
    dY = randn(gen, M, N)
    g = mk.gated_gemm_backward(A, *Bs, Z, dY, want_dbias=True)
    assert g.dA.numel() * 2 > 1 << 32
    ref.check(g.dA[r], ref.backward(A[r], Bs, [z[r] for z in Z], dY[r], "silu", torch.float32)["dA"], "dA")
    c = pick(K, 200)             # rows of dB
    w = ref.backward(A[:, c], [b[c] for b in Bs], Z, dY, "silu", torch.float32)
    for got, want, name in ((g.dBg[c], w["dB"][0], "dBg"), (g.dBu[c], w["dB"][1], "dBu"),
                            (g.dbias_g, w["dbias"][0], "dbias_g"), (g.dbias_u, w["dbias"][1], "dbias_u")):
        ref.check(got, want, name)
    progress("backward")


def test_wide_outputs():
    M, N, K = 70, 8388600, 72    # B and Y of pitches just below 2^23; B: 1.2 GB, fp32 Y: 2.3 GB
    gen = torch.Generator(device="cuda").manual_seed(2)
    A, B, R = randn(gen, M, K), randn(gen, K, N, std=K ** -0.5), randn(gen, M, N, dt=torch.float32)
    c = pick(N, 3000)
    for m in (M, 3):             # tiles, and the few-row kernel
        Y = mk.gemm_residual(A[:m], B, R[:m], act="gelu")
        v, e, _ = ref.residual(A[:m], B[:, c], None, R[:m, c], "gelu", torch.float32)
        ref.check(Y[:, c], (v, e), "Y")
    progress("wide")


@pytest.mark.parametrize("M,N,K", [(260, 130, 200), (130, 260, 200), (260, 200, 130)])
def test_pitches_below_2_23(M, N, K):
    P = (1 << 23) - 8
    gen = torch.Generator(device="cuda").manual_seed(3)

    def wide(rows, cols, dt=torch.bfloat16):
        t = torch.empty(rows * P, device="cuda", dtype=dt).view(rows, P)[:, :cols]
        t.copy_(randn(gen, rows, cols, dt=dt))
        return t
    A, B, R = wide(M, K), wide(K, N), wide(M, N)
    out, pre = wide(M, N), wide(M, N)
    Y, Z = mk.gemm_residual_train(A, B, R, act="relu", out=out, preact=pre)
    v, e, z = ref.residual(A, B, None, R, "relu", A.dtype)
    ref.check(Y, (v, e), "Y")
    ref.check(Z, z, "Z")
    progress("forward")
    dY, dA, dB = wide(M, N), wide(M, K), wide(K, N)
    g = mk.gemm_residual_backward(A, B, dY, Z, act="relu", grad_dtype=A.dtype, dA=dA, dB=dB)
    w = ref.backward(A, [B], [Z], dY, "relu", A.dtype)
    ref.check(g.dA, w["dA"], "dA")
    ref.check(g.dB, w["dB"][0], "dB")


def test_clip_above_2_31_elements():
    n = (1 << 31) + 4099
    t = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    t[-1] = 2.0
    small = torch.full((77,), -3.0, device="cuda")
    norm = mk.clip_grad_norm([small, t], 1.0)
    want = math.sqrt((n - 1) * 0.25 + 4.0 + 77 * 9.0)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    # every 0.5 becomes the same bf16 value; the sampled ones, the ends and an fp32 tensor behind
    half = torch.tensor(0.5 / want, dtype=torch.float64)
    got = t[pick(n - 1, 5000)].double()
    assert bool(((got - half.item()).abs() <= ref.half_step(half, torch.bfloat16).item() * 1.001).all())
    assert int((t[:-1] != t[0]).sum()) == 0
    assert abs(float(t[-1]) * want / 2 - 1) <= 2.0 ** -8 and abs(float(small[5]) * want / -3 - 1) <= 2.0 ** -22


@pytest.mark.parametrize("norm_type", [2, math.inf])
def test_clip_of_many_large_tensors(norm_type):
    # several tables of every type, more than the cache holds: each part of the
    # list read and written its own way
    gen = torch.Generator(device="cuda").manual_seed(5)
    ts = [randn(gen, 1500000 + 7 * i, dt=(torch.bfloat16, torch.float32, torch.float16)[i % 3 if i % 10 else 0])
          for i in range(150)]
    assert sum(t.numel() * t.element_size() for t in ts) > 500 << 20
    want = torch.stack([t.double().norm(norm_type) for t in ts]).norm(norm_type)
    outs = [torch.empty_like(t) for t in ts]
    norm = mk.clip_grad_norm(ts, 0.5, norm_type=norm_type, out=outs)
    # one rounding of the norm to fp32
    assert abs(float(norm) - float(want)) <= 2.0 ** -24 * 1.001 * float(want)
    c = 0.5 / (want + 1e-6)
    for t, o in zip(ts, outs):
        v = t.double() * c
        # c and the product rounded to fp32, the product to the type
        assert bool(((o.double() - v).abs() <= 2 * 2.0 ** -24 * v.abs() + ref.half_step(v, t.dtype)).all())
    again = mk.clip_grad_norm(ts, 0.5, norm_type=norm_type)
    assert torch.equal(norm, again) and all(torch.equal(a, b) for a, b in zip(ts, outs))


def test_two_calls_at_once():
    gen = torch.Generator(device="cuda").manual_seed(4)
    jobs = []
    for M, N, K in ((777, 1030, 4100), (500, 1030, 2050)):   # both split their contraction
        rows = lambda *a, **k: mk.aligned_copy(randn(gen, *a, **k), "cuda")  # noqa: E731
        A, Bs, dY = rows(M, K), [rows(K, N, std=K ** -0.5) for _ in range(2)], rows(M, N)
        H, Z = mk.gated_gemm_train(A, *Bs)
        g = mk.gated_gemm_backward(A, *Bs, Z, dY, want_dbias=True)
        jobs.append((A, Bs, dY, [H, *Z, *g], torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (A, Bs, dY, _, s) in enumerate(jobs):
            H, Z = mk.gated_gemm_train(A, *Bs, stream=s)
            g = mk.gated_gemm_backward(A, *Bs, Z, dY, want_dbias=True, stream=s)
            outs[i].append([H, *Z, *g])
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for got in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, job[3]))


def test_lists_that_are_refused():
    t = torch.ones(1000, device="cuda")
    u = torch.ones(1000, device="cuda")
    keep = t.clone()
    for grads, out in (([t, t], None), ([t, t[10:20]], None), ([t, u], [u, t]), ([t], [t.view(-1)[:999]]),
                       ([t[:500]], [t[1:501]]), ([t[::2]], None)):
        with pytest.raises((ValueError, RuntimeError)):
            mk.clip_grad_norm(grads, 1.0, out=out)
    with pytest.raises((ValueError, RuntimeError)):
        mk.clip_grad_norm([t], 1.0, norm=t[3])
    assert torch.equal(t, keep)
    # read twice is fine where nothing is written
    assert abs(float(mk.grad_norm([t, t])) - math.sqrt(2000)) <= 1e-5
    assert abs(float(mk.clip_grad_norm([t, t], 1.0, out=[u, torch.empty_like(t)])) - math.sqrt(2000)) <= 1e-5


def test_second_derivatives_are_refused():
    m = mk.GatedFFN(64, 128)
    x = torch.randn(8, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    g, = torch.autograd.grad(m(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_capture_with_an_eager_graph_alive_is_refused(monkeypatch):
    m, other = mk.GatedFFN(64, 128), mk.GatedFFN(64, 128)
    x = torch.randn(8, 64, device="cuda", dtype=torch.bfloat16)
    y = m(x)
    # nothing is captured here: the module is told so
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="still alive"):
        m(x)
    with torch.no_grad():
        m(x)
    other(x)
    del y
    m(x)


def test_module_step_captured_and_replayed():
    torch.manual_seed(6)
    m = mk.GatedFFN(72, 200, bias=True)
    x = torch.randn(50, 72, device="cuda", dtype=torch.bfloat16)

    def step():
        for p in m.parameters():
            p.grad = None
        y = m(x)
        y.backward(x)
        norm = mk.clip_grad_norm([p.grad for p in m.parameters()], 1.0)
        return y.detach(), norm
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, norm = step()
    grads = [p.grad for p in m.parameters()]
    for i in range(4):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone(), norm.clone()] + [g.clone() for g in grads]
        with torch.cuda.stream(side):
            want_y, want_norm = step()
            want = [want_y, want_norm] + [p.grad for p in m.parameters()]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
