"""Gradients through rkv_rope_apply: the transpose of the rotation, to q and k,
whichever of them asks for one."""
import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from tests import cache_ref as ref
from tests.test_gpu_cache import BF, DEV, FP, gen, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d, rot, inter", [(64, 64, False), (128, 64, True), (64, 20, False)])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_is_the_transpose(dt, d, rot, inter, inverse):
    n, hq, hk, m = 37, 4, 2, 1.25
    plan = pkg.RopePlan(rot, interleaved=inter, attn_factor=m)
    f = ref.freqs(rot)
    pos = torch.randint(0, 131072, (n,), generator=gen(1), dtype=torch.int32)
    q, k = rnd((n, hq, d), dt, 2).requires_grad_(), rnd((n, hk, d), dt, 3).requires_grad_()
    oq, ok = pkg.rkv_rope_apply(plan, pos.to(DEV), q, k, inverse=inverse)
    with torch.no_grad():
        pq, pk = pkg.rkv_rope_apply(plan, pos.to(DEV), q, k, inverse=inverse)
    assert torch.equal(oq, pq) and torch.equal(ok, pk) and not pq.requires_grad
    gq, gk = rnd(oq.shape, dt, 4), rnd(ok.shape, dt, 5)
    torch.autograd.backward([oq, ok], [gq, gk])
    for x, g in ((q, gq), (k, gk)):
        e = ref.rotate(g, pos, f, inter, m, not inverse)
        assert ((x.grad.double().cpu() - e).abs() <= ref.rotate_bound(g, e, rot, inter, dt, m)).all()


def test_gradient_against_differences():
    """The map is linear: the slope along any direction is the map of the
    direction, exactly, whatever the step."""
    n, d = 5, 64
    plan = pkg.RopePlan(d, interleaved=True, attn_factor=0.75)
    pos = torch.tensor([0, 3, 900, 70000, 131071], dtype=torch.int32, device=DEV)
    x, w, u = (rnd((n, 2, d), FP, i) for i in (1, 2, 3))
    a = x.clone().requires_grad_()
    (pkg.rkv_rope_apply(plan, pos, a) * w).sum().backward()
    slope = (a.grad.double() * u.double()).sum()
    with torch.no_grad():
        moved = (pkg.rkv_rope_apply(plan, pos, u).double() * w.double()).sum()
    # each side: n * 2 * d products, a factor off by 8 * 2^-24 (|x| + |x'|)
    lim = 2 * 8 * ref.U32 * 2 * 2 * float(u.abs().amax() * w.abs().sum())
    assert abs(float(slope - moved)) <= lim


def test_one_of_two_and_expanded_gradients():
    n, d = 9, 128
    plan = pkg.RopePlan(d)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    for first in (True, False):
        q, k = rnd((n, 4, d), FP, 2), rnd((n, 2, d), FP, 3)
        one, other = (q, k) if first else (k, q)
        one.requires_grad_()
        oq, ok = pkg.rkv_rope_apply(plan, pos, q, k)
        hot, cold = (oq, ok) if first else (ok, oq)
        assert hot.requires_grad and not cold.requires_grad
        hot.sum().backward()  # its gradient is one element, expanded
        e = ref.rotate(torch.ones(hot.shape), pos, ref.freqs(d), inverse=True)
        assert ((one.grad.double().cpu() - e).abs() <= 16 * ref.U32).all() and other.grad is None
    # only one of two outputs used; a gradient whose rows lie apart by an odd stride
    q, k = rnd((n, 4, d), BF, 2).requires_grad_(), rnd((n, 2, d), BF, 3).requires_grad_()
    oq, ok = pkg.rkv_rope_apply(plan, pos, q, k)
    g = rnd((n, 2, d + 1), BF, 8)[..., 1:]
    ok.backward(g)
    e = ref.rotate(g, pos, ref.freqs(d), inverse=True)
    assert ((k.grad.double().cpu() - e).abs() <= ref.rotate_bound(g, e, d, False, BF)).all()
    assert q.grad is None


def test_second_gradients_streams_and_empty():
    n, d = 6, 64
    plan = pkg.RopePlan(d)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    q = rnd((2, 3, 4, d), FP, 2).requires_grad_()
    y = pkg.rkv_rope_apply(plan, pos.view(2, 3), q)
    g, = torch.autograd.grad((y ** 3).sum(), q, create_graph=True)
    h, = torch.autograd.grad(g.sum(), q)  # R^T diag(6 y) R 1
    with torch.no_grad():
        one = pkg.rkv_rope_apply(plan, pos.view(2, 3), torch.ones_like(q))
        e = pkg.rkv_rope_apply(plan, pos.view(2, 3), 6 * y * one, inverse=True)
    assert torch.allclose(h, e, rtol=1e-5, atol=1e-4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    z = pkg.rkv_rope_apply(plan, pos.view(2, 3), q, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    gz, = torch.autograd.grad(z, q, torch.ones_like(z))
    torch.cuda.synchronize()
    with torch.no_grad():
        assert torch.equal(gz, pkg.rkv_rope_apply(plan, pos.view(2, 3), torch.ones_like(q), inverse=True))
    none = torch.zeros(0, 4, d, device=DEV, requires_grad=True)
    pkg.rkv_rope_apply(plan, pos[:0], none).sum().backward()
    assert none.grad.shape == (0, 4, d)


def test_captured_forward_and_backward():
    n, d = 64, 128
    plan = pkg.RopePlan(d)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    q, w = rnd((n, 4, d), BF, 2).requires_grad_(), rnd((n, 4, d), BF, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(pkg.rkv_rope_apply(plan, pos, q), q, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, = torch.autograd.grad(pkg.rkv_rope_apply(plan, pos, q), q, w)
    for seed in (5, 6):
        w.copy_(rnd(w.shape, BF, seed))
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            assert torch.equal(g, pkg.rkv_rope_apply(plan, pos, w, inverse=True))


def test_refusals_where_a_gradient_is_asked_for():
    plan = pkg.RopePlan(64)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    q, k = rnd((3, 2, 64), BF, 2).requires_grad_(), rnd((3, 1, 64), BF, 3)
    for kw in (dict(out_q=torch.empty_like(q)), dict(k=k, out_k=torch.empty_like(k)), dict(out_q=q)):
        with pytest.raises(ValueError):
            pkg.rkv_rope_apply(plan, pos, q, **kw)
        with torch.no_grad():
            pkg.rkv_rope_apply(plan, pos, q.clone(), **kw) if kw.get("out_q") is not q else None
    saved = pos.clone()
    y = pkg.rkv_rope_apply(plan, saved, q)
    saved += 1  # what the gradient needs has changed
    with pytest.raises(RuntimeError):
        y.sum().backward()
