"""A forward pass may write the stream in the residual's place; the backward pass reads
the residual as it was before. The forward's arrays given to it as they were then name
the new stream as the residual: refused, where it can be seen."""
import pytest
import torch as th

import test_gpu_norm as base
import weight_quantized_swiglu_gb300 as q
from test_gpu_norm import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def test_backward_refuses_the_arrays_of_a_forward_in_place(torch):  # noqa: F811
    M, K, dt = 21, 256, th.bfloat16
    d = base.make(torch, M, K, dt, dt, dt, "none", True, True, 5)
    z, r, wp, wr, dout, dh = (d[n] for n in ("z", "residual", "post_w", "pre_w", "dout", "dresidual_out"))
    norm = q.BlockNorm(K, dtype=dt)
    stats, y, h = torch.empty((M, 2), device="cuda"), torch.empty_like(z), r.clone()
    p = lambda t: t.data_ptr()  # noqa: E731
    io = q.qmlp_norm_io(p(z), p(h), p(wp), p(wr), None, p(h), p(y), p(stats))
    assert q.qmlp_norm_forward(norm.h, io, M) == 0
    dz, dr = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
    g = q.qmlp_norm_grads(p(dout), p(dh), p(dz), p(dr), None, None, None)
    assert q.qmlp_norm_backward(norm.h, io, g, M) == 3  # ALIAS
    torch.cuda.synchronize()
    assert dz.eq(7.0).all() and dr.eq(7.0).all()
    # the residual kept: what a forward beside it gives, with residual_out named or not
    outs = []
    for keep, ro in ((r, h), (r, None)):
        io = q.qmlp_norm_io(p(z), p(keep), p(wp), p(wr), None, ro if ro is None else p(ro), None, p(stats))
        assert q.qmlp_norm_backward(norm.h, io, g, M) == 0
        outs.append((dz.clone(), dr.clone()))
    stats2 = torch.empty_like(stats)
    norm.forward(z=z, residual=r, post_w=wp, pre_w=wr, residual_out=torch.empty_like(r), out=y, stats=stats2)
    norm.backward(stats2, z=z, residual=r, post_w=wp, pre_w=wr, dout=dout, dresidual_out=dh, dz=dz, dresidual=dr)
    for a in outs:
        assert torch.equal(a[0], dz) and torch.equal(a[1], dr)
    norm.close()
