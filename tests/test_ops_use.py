"""Use of the training operators beyond single calls on one stream: the kernels of a few
rows in a graph and on other streams, calls that overlap, outputs left out, and the drift
of long sums."""
import threading

import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from matrix_orthogonalising_optimizer_gb300 import _lib
from test_ops import ffn_inputs, gen, randn


def chain(n, dtype, seed):
    """A norm, a block and a loss with their gradients, of n tokens: work(stream) returns
    everything; buffers of its own, so that chains may overlap."""
    x, wg, wu, wd, _ = ffn_inputs(n, 512, 1024, dtype, seed)
    t = torch.randint(0, 1024, (n,), device="cuda")
    coef = torch.full((n,), 1.0 / n, device="cuda")
    ws = torch.empty(max(pkg.gated_ffn_workspace(n, 512, 1024, dtype, backward=True),
                         pkg.vocab_loss_workspace(n, 512, 1024, dtype, grad=True),
                         pkg.layer_norm_workspace(n, 512, dtype)), dtype=torch.uint8, device="cuda")

    def work(stream=None):
        y, m, r = pkg.layer_norm(x, stream=stream)
        z = pkg.gated_ffn(y, wg, wu, wd, workspace=ws, stream=stream)
        z2, saved, h = pkg.gated_ffn(y, wg, wu, wd, save=True, workspace=ws, stream=stream)
        only, lse = pkg.vocab_loss(z, wg, t, workspace=ws, stream=stream)
        loss, _, dz, dw = pkg.vocab_loss_grad(z2, wg, t, coef=coef, workspace=ws, stream=stream)
        dy, *dws = pkg.gated_ffn_backward(dz, y, wg, wu, wd, saved, h, workspace=ws, stream=stream)
        return (z, only, lse, loss, dw, *dws, *pkg.layer_norm_backward(dy, x, None, m, r, workspace=ws, stream=stream))

    return work


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 14, 29])
def test_few_rows_on_another_stream_and_in_a_graph(n, dtype):
    work = chain(n, dtype, n)
    want = [o.clone() for o in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = work(side)
    side.synchronize()
    assert same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        for o in got:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.gpu
def test_overlapping_streams_and_threads():
    """Calls with workspaces of their own may overlap: two streams of one thread, then two threads."""
    works = [chain(n, dt, 40 + n) for n, dt in ((5, torch.bfloat16), (300, torch.bfloat16), (40, torch.float32))]
    wants = [[o.clone() for o in w()] for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    for _ in range(5):
        gots = [w(s) for w, s in zip(works, streams)]
        torch.cuda.synchronize()
        assert all(same(g, w) for g, w in zip(gots, wants))
    bad = []

    def loop(work, want, stream):
        try:
            for _ in range(10):
                got = work(stream)
                stream.synchronize()
                if not same(got, want):
                    bad.append("outputs differ")
        except Exception as e:  # reported by the test's own thread
            bad.append(repr(e))

    threads = [threading.Thread(target=loop, args=a) for a in zip(works, wants, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(3, 70), (700, 256), (2500, 96), (20, 40000)])
def test_norm_backward_without_one_of_the_sums(lib, rows, cols):
    g = gen(rows)
    x, dy, w = randn(g, rows, cols), randn(g, rows, cols), randn(g, cols)
    _, mean, rstd = pkg.layer_norm(x, w)
    dx, dw, db = pkg.layer_norm_backward(dy, x, w, mean, rstd)
    need = pkg.layer_norm_workspace(rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for with_dw, with_db in ((True, False), (False, True), (False, False)):
        dx2 = torch.empty_like(dx)
        dw2, db2 = torch.full_like(dw, 7.0), torch.full_like(db, 7.0)
        space = ws.data_ptr() if with_dw or with_db else None  # neither: no workspace needed
        assert lib.dmuon_layer_norm_backward(
            dy.data_ptr(), x.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), dx2.data_ptr(),
            dw2.data_ptr() if with_dw else None, db2.data_ptr() if with_db else None, rows, cols, _lib.BF16, space,
            need if space else 0, stream) == _lib.OK
        assert torch.equal(dx2, dx)
        assert torch.equal(dw2, dw) if with_dw else (dw2 == 7).all()
        assert torch.equal(db2, db) if with_db else (db2 == 7).all()


@pytest.mark.gpu
def test_long_sums_have_no_bias():
    """The mean relative error of sums of 140000 positive terms, more than are left in one
    chain of tensor-core additions.  Rounding the results averages out over 10^6 of them
    (2^-9 / 1000); truncated additions do not, and are to stay below 2^-13."""
    n, d = 140000, 1024
    g = gen(4)
    x = torch.rand(n, d, generator=g, device="cuda").mul_(1 / 32).bfloat16()
    dy = torch.rand(n, d, generator=g, device="cuda").bfloat16()
    wg, wu, wd = (torch.rand(d, d, generator=g, device="cuda").mul_(1 / 32).bfloat16() for _ in range(3))
    _, saved, h = pkg.gated_ffn(x, wg, wu, wd, save="compact")
    dwd = pkg.gated_ffn_backward(dy, x, wg, wu, wd, saved, h)[3].double()
    want = torch.zeros(d, d, device="cuda", dtype=torch.double)
    for i in range(0, n, 20000):
        want += dy[i:i + 20000].double().T @ h[i:i + 20000].double()
    assert abs(float(((dwd - want) / want).mean())) <= 2.0 ** -13
