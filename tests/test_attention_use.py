"""Use of the head norms and of attention beyond single calls on one stream: a transformer
block's chain in a graph and on other streams, calls that overlap, repeated calls, offsets
past 2^31 elements, and a training step of the example model against autograd in 64 bits."""
import importlib.util
import os
import threading

import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from test_attention import DT, NEG, inputs
from test_ops import gen, randn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def chain(n, h, kv, d, dtype, seed, offsets=None):
    """Norm and rotation, attention and both backward passes on views of one projection: work(stream)
    returns everything; buffers of its own, so that chains may overlap."""
    g, dt = gen(seed), DT[dtype]
    q, k, v = randn(g, n, (h + 2 * kv) * d, dt=dt).split([h * d, kv * d, kv * d], 1)
    q, k, v = q.view(n, h, d), k.view(n, kv, d), v.view(n, kv, d)
    do = randn(g, n, h, d, std=1e-2, dt=dt)
    off = None if offsets is None else torch.tensor(offsets, device="cuda")
    seqs = 1 if offsets is None else len(offsets) - 1
    table, pos = pkg.rotary_table(n, d // 2 * 2), torch.arange(n, device="cuda")
    w = torch.ones(d, dtype=dt, device="cuda")
    ws = torch.empty(max(pkg.attention_workspace(n, h, kv, d, dtype, sequences=seqs, backward=True),
                         pkg.qk_norm_rotary_workspace(n, h, kv, d, dtype)), dtype=torch.uint8, device="cuda")

    def work(stream=None):
        a, b = pkg.qk_norm_rotary(q, k, pos, table, w, w, stream=stream)
        o, lse = pkg.attention(a, b, v, off, workspace=ws, stream=stream)
        da, db, dv = pkg.attention_backward(do, a, b, v, o, lse, off, workspace=ws, stream=stream)
        return (a, b, o, lse, da, db, dv, *pkg.qk_norm_rotary_backward(da, db, q, k, pos, table, w, w, workspace=ws,
                                                                      stream=stream))

    return work


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


CHAINS = [(1, 12, 12, 64, None), (37, 4, 2, 128, None), (300, 8, 1, 64, [0, 5, 140, 300]), (700, 6, 2, 80, [0, 700]),
          (150, 3, 3, 33, [0, 70, 150]), (520, 16, 2, 128, [3, 130, 510])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,h,kv,d,offsets", CHAINS)
def test_on_another_stream_and_in_a_graph(n, h, kv, d, offsets, dtype):
    work = chain(n, h, kv, d, dtype, n, offsets)
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
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    assert pkg.ops_status() == 0


@pytest.mark.gpu
def test_calls_that_overlap():
    works = [chain(n, h, kv, d, dtype, s, off) for s, (n, h, kv, d, off) in enumerate(CHAINS) for dtype in ("bf16", "fp32")]
    want = [[o.clone() for o in w()] for w in works]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    got = [None] * len(works)

    def run(i):
        for _ in range(5):
            got[i] = works[i](streams[i])

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,kv,d,offsets", [(2048, 32, 8, 128, None), (1500, 32, 1, 64, [0, 900, 1500]),
                                              (3000, 4, 4, 64, [0, 1, 800, 2900]), (1200, 16, 2, 128, None)])
def test_repeated_calls_agree_bit_for_bit(n, h, kv, d, offsets):
    work = chain(n, h, kv, d, "bf16", n, offsets)
    want = [o.clone() for o in work()]
    for _ in range(4):
        assert same(work(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_does_not_change_results(dtype):
    # the same sequences with rows of no sequence before, behind and NaN in them (every query head
    # with its own key head: how many blocks share a group's sums goes by the number of tokens)
    n, h, kv, d = 300, 4, 4, 64
    q, k, v, do, _ = inputs([0, n], n, h, kv, d, dtype, False, 3)
    off = torch.tensor([0, 100, 300], device="cuda")
    o, lse = pkg.attention(q, k, v, off)
    want = (o, *pkg.attention_backward(do, q, k, v, o, lse, off))

    def pad(x):
        y = torch.full((n + 170, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda")
        y[61:61 + n] = x
        return y

    q, k, v, do = (pad(x) for x in (q, k, v, do))
    o, lse2 = pkg.attention(q, k, v, off + 61)
    got = (o, *pkg.attention_backward(do, q, k, v, o, lse2, off + 61))
    for a, b in zip(got, want):
        assert torch.equal(a[61:61 + n], b) and not a[:61].any() and not a[61 + n:].any()
    assert torch.equal(lse2[:, 61:61 + n], lse)
    assert (lse2[:, :61] == NEG).all() and (lse2[:, 61 + n:] == NEG).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [(300, 400), (300, 3000), (100, 28)])
def test_values_of_the_next_sequence_do_not_show(lengths, d, dtype):
    # rows of the next sequence lie in the same tile; here their logits grow much faster
    n = sum(lengths)
    q, k, v, do, _ = inputs([0, n], n, 4, 2, d, dtype, False, n)
    off = torch.tensor([0, lengths[0], n], device="cuda")
    results = []
    for f in (1.0, 40.0):
        a = [x.clone() for x in (q, k, v, do)]
        for x in a:
            x[lengths[0]:] *= f
        o, lse = pkg.attention(*a[:3], off)
        first = (o, lse.T, *pkg.attention_backward(a[3], *a[:3], o, lse, off))
        results.append([x[:lengths[0]].clone() for x in first])
    assert same(*results)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 40, 33])
def test_heads_before_tokens(dim, dtype):
    # heads x tokens x dim tensors read in place, and a single token with any stride
    q, k, v, do, _ = inputs([0, 290], 290, 4, 2, dim, dtype, False, dim)
    table, pos = pkg.rotary_table(290, dim // 2 * 2), torch.arange(290, device="cuda")

    def turn(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def all_of(q, k, v, do):
        a, b = pkg.qk_norm_rotary(q, k, pos[:len(q)], table)
        o, lse = pkg.attention(q, k, v)
        return a, b, o, lse, *pkg.attention_backward(do, q, k, v, o, lse)

    for n in (290, 1):
        x = [y[:n].contiguous() for y in (q, k, v, do)]
        assert same(all_of(*(turn(y) for y in x)), all_of(*x))
    assert same(all_of(*(turn(y)[:1] for y in (q, k, v, do))), all_of(*x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mostly_padding(dtype):
    # one short sequence somewhere in many tokens, odd sizes: everything else is cleared
    for n, h, kv, d, at in ((20001, 3, 1, 72, 7000), (9000, 2, 2, 7, 0), (5000, 8, 2, 128, 4990)):
        q, k, v, do, out = inputs([at, at + 10], n, h, kv, d, dtype, False, n)
        off = torch.tensor([at, at + 10], device="cuda")
        o, lse = pkg.attention(q, k, v, off)
        for x in (o, *pkg.attention_backward(do, q, k, v, o, lse, off)):
            assert not x[out].any() and x[~out].any()
        assert (lse[:, out] == NEG).all() and lse[:, ~out].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_elements_past_two_to_the_31(dtype):
    # 2.3e9 elements: the last tokens alone, as part of the whole and by themselves (two sequences of more
    # than one tile: shorter ones take other kernels where the average length is short)
    n, h, d, last = 70000, 256, 128, 300
    x = torch.zeros(n, h, d, dtype=DT[dtype], device="cuda")
    x[-last:] = randn(gen(5), last, h, d, dt=DT[dtype])
    off = torch.tensor([n - last, n - 140, n], device="cuda")
    small = x[-last:].clone()
    o, lse = pkg.attention(x, x, x, off)
    want, lse2 = pkg.attention(small, small, small, off - (n - last))
    assert torch.equal(o[-last:], want) and torch.equal(lse[:, -last:], lse2) and not o[:-last].any()
    grads = pkg.attention_backward(x, x, x, x, o, lse, off)
    del o
    for a, b in zip(grads, pkg.attention_backward(small, small, small, small, want, lse2, off - (n - last))):
        assert torch.equal(a[-last:], b) and not a[-last - 200:-last].any()
    del grads
    table, pos = pkg.rotary_table(64, d), torch.arange(n, device="cuda") % 64
    a, b = pkg.qk_norm_rotary(x, x[:, :1], pos, table)
    c, e = pkg.qk_norm_rotary(small, small[:, :1], pos[-last:], table)
    assert torch.equal(a[-last:], c) and torch.equal(b[-last:], e)


def example():
    spec = importlib.util.spec_from_file_location("train_transformer_lm",
                                                  os.path.join(ROOT, "examples", "train_transformer_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference_loss(model, blocks, top, tokens, targets, offsets, positions):
    """The example model's mean loss in 64 bits, from its parameters as given."""
    h, kv, d, n = model.heads, model.kv, model.head_dim, tokens.shape[0]
    cos, sin = model.table[positions].double().chunk(2, 1)

    def norm(x, w):
        x = x - x.mean(-1, keepdim=True)
        return x * (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w

    def head_norm(x, w):
        y = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = y.chunk(2, -1)
        c, s = cos[:, None], sin[:, None]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    text = torch.searchsorted(offsets, torch.arange(n, device="cuda"), right=True)
    seen = (text[:, None] == text[None]) & torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    x = top["embed"][tokens]
    for b in blocks:
        q, k, v = (norm(x, b["norm1"]) @ b["w_qkv"].T).split([h * d, kv * d, kv * d], 1)
        q, k = head_norm(q.view(n, h, d), b["q_norm"]), head_norm(k.view(n, kv, d), b["k_norm"])
        k, v = (y.reshape(n, kv, d).repeat_interleave(h // kv, 1) for y in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        p = s.masked_fill(~seen, NEG).softmax(-1)
        x = x + torch.einsum("hij,jhd->ihd", p, v).flatten(1) @ b["w_out"].T
        y = norm(x, b["norm2"])
        x = x + (torch.nn.functional.silu(y @ b["w_gate"].T) * (y @ b["w_up"].T)) @ b["w_down"].T
    return torch.nn.functional.cross_entropy(norm(x, top["norm"]) @ top["head"].T, targets)


@pytest.mark.gpu
def test_example_runs_in_bf16():
    losses = example().train(steps=3, vocab=120, dim=128, hidden=256, tokens=512, sequences=5)
    assert all(x == x and 0 < x < 20 for x in losses)


@pytest.mark.gpu
def test_example_gradients_against_autograd():
    # fp32 all through: every product, norm and softmax is good to about 1e-6 of its terms' sizes, a block
    # chains some ten of them, and cancellation inside the norms and the softmax's gradient costs at most a
    # factor 10 on these unit-scale activations: 2e-4 of each gradient's norm
    mod = example()
    model = mod.Model(100, 64, 160, 4, 2, 2, 384, 4, torch.float32, 1)
    data = mod.batch(gen(2), 100, 384, 4)
    loss, blocks, top = model.gradients(*data)
    ref_blocks = [{k: w.double().requires_grad_() for k, w in b.items()} for b in model.blocks]
    ref_top = {k: w.double().requires_grad_() for k, w in model.top.items()}
    want = reference_loss(model, ref_blocks, ref_top, *data)
    want.backward()
    assert (loss - want.detach()).abs() <= 1e-5 * want.detach()
    for got, ref in [*zip(blocks, ref_blocks), (top, ref_top)]:
        for name, w in ref.items():
            err = (got[name].double() - w.grad).norm() / w.grad.norm()
            assert err <= 2e-4, (name, float(err))
