"""The operators around the blocks together, as a program uses them: a training step of a model with a
tied embedding, and a serving step that verifies drafts; and what they write and read of memory that
is not theirs."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_dropout import dropped, factor, kept
from test_train_guards import Guards
from test_train_streams import _busy, _reuse

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _training_step(ids, targets, W, weight, bias, way, p, seed, stream=None):
    """Embedding, dropout, a stand-in for the blocks (y = way * h), the branch's dropout and layer norm,
    the tied head's loss; the gradients of W, weight and bias."""
    kw = {"stream": stream}
    h = sb.embedding(ids, W, scale=1.5, **kw)
    h0 = sb.dropout(h, p, seed=seed, **kw)
    y = h0 * way
    n = sb.layer_norm(h0, weight, bias, y=y, p=p, seed=seed + 1, **kw)
    ce = sb.cross_entropy(n["x"], W, targets, **kw)
    g = sb.cross_entropy_backward(n["x"], W, targets, ce["lse"], **kw)
    b = sb.layer_norm_backward(g["dH"], None, n["h"], weight, need_dy=True, p=p, seed=seed + 1, **kw)
    dh0 = (b["dh"].float() + b["dy"].float() * way.float()).to(BF)
    dh = sb.dropout(dh0, p, seed=seed, **kw)
    sb.embedding_backward(ids, dh, dW=g["dW"], scale=1.5, **kw)
    return ce["loss"], g["dW"], b["dweight"], b["dbias"]


def _inputs(M, d, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).to(BF)
    ids = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    ids[::7] = ids[0]
    targets = ids.roll(-1).clone()
    targets[-1] = ids[-3] = -100
    weight, bias = 1 + 0.1 * torch.randn(d, generator=g, device="cuda"), 0.1 * torch.randn(d, generator=g, device="cuda")
    return ids, targets, W, weight, bias, torch.full((d,), 0.5, device="cuda", dtype=BF)


def test_a_training_step_with_a_tied_embedding():
    """Against autograd in 64 bits.  The chain rounds to bf16 at ten places in turn (h, h0, y, x, G's
    products, dH, dh, dy, dh0, and again): each is off by 2^-9 of its values in the root mean square at
    most, and no step enlarges a relative error more than fourfold in norm (the layer norm's backward
    subtracts two projections; h0 and y add up): 10 · 4 · 2^-9 = 0.08 bounds the 2-norm."""
    M, d, V, p, seed = 300, 256, 1000, 0.1, 21
    ids, targets, W, weight, bias, way = _inputs(M, d, V)
    loss, dW, dweight, dbias = _training_step(ids, targets, W, weight, bias, way, p, seed)

    leaf = [t.to(F64).requires_grad_() for t in (W, weight, bias)]

    def drop(x, seed):
        return torch.where(kept(x.numel(), p, seed).view(x.shape), x * factor(p), 0.0)

    h = leaf[0][ids.clamp(min=0).long()] * 1.5 * (ids != -100)[:, None]
    h = drop(h, seed)
    h = h + drop(h * way.to(F64), seed + 1)
    var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
    x = (h - mean) / torch.sqrt(var + 1e-5) * leaf[1] + leaf[2]
    want = torch.nn.functional.cross_entropy(x @ leaf[0].T, targets.long(), ignore_index=-100)
    grads = torch.autograd.grad(want, leaf)
    want = float(want.detach())
    assert abs(float(loss) - want) < 0.08 * want
    for got, exact in zip((dW, dweight, dbias), grads):
        assert torch.isfinite(got).all()
        assert (got.to(F64) - exact).norm() <= 0.08 * exact.norm()
    # the rows of W that only the lookup reaches are those of the lookup's gradient plus the head's
    assert dropped(W, p, seed)[1].any()


def test_a_captured_step_and_an_eager_one():
    """One step in a graph, replayed between eager steps on the same tensors, each giving its own bits."""
    M, d, V = 200, 264, 777
    a = _inputs(M, d, V, 1)
    want = _training_step(*a, 0.1, 5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _training_step(*a, 0.1, 5)
    for _ in range(3):
        eager = _training_step(*a, 0.1, 5)
        graph.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(want, got, eager):
            assert torch.equal(x, y) and torch.equal(x, z)


def test_a_serving_step():
    """Drafted tokens in through the embedding, out through norm and head, verified; the answers go in
    again.  The greedy answers and the logits' own softmax say what has to come."""
    d, V, lengths = 256, 3001, [3, 0, 5, 2]
    g = torch.Generator(device="cuda").manual_seed(2)
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).to(BF)
    rows = [n + 1 for n in lengths]
    starts = torch.tensor([0, 4, 5, 11, 14], dtype=torch.int32, device="cuda")
    R = sum(rows)
    ids = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    weight = torch.ones(d, device="cuda")
    x = sb.layer_norm(sb.embedding(ids, W, scale=16.0), weight)["x"]
    res = sb.project(x, W, 1, sb.SB_FULL_LOGITS)
    # greedy: the drafts are the head's own answers but in one place
    drafts = res["token"].clone()
    drafts[6] += 1
    f = sb.verify_greedy(res["token"], drafts, starts)
    assert f["accepted"].tolist() == [3, 0, 1, 2] and f["token"][7:11].tolist() == [-1] * 4
    # sampled, with the head's logsumexp: the drafts that stay have p > u
    u = torch.rand(R, generator=g, device="cuda") * 0.01
    s = sb.verify_drafts(res["logits"], drafts, starts, u, lse=res["lse"], seed=3)
    p = (res["logits"].double() - res["lse"].double()[:, None]).exp()
    at = 0
    for b, k in enumerate(rows):
        n = int(s["accepted"][b])
        for i in range(k):
            r = at + i
            if i < n:
                assert s["token"][r] == drafts[r] and p[r, drafts[r]] > u[r]
            elif i == n:
                assert 0 <= s["token"][r] < V and (i == k - 1 or not p[r, drafts[r].clamp(max=V - 1)] > u[r])
                lp = p[r, s["token"][r]].log()
                assert abs(float(lp) - float(s["token_logprob"][r])) < 1e-5
            else:
                assert s["token"][r] == -1
        at += k
    again = sb.embedding(s["token"], W, ignore_index=-1)
    assert (again[s["token"] == -1] == 0).all() and torch.equal(again[0], W[s["token"][0]])


@pytest.mark.parametrize("raw", [False, True])
def test_inputs_may_go(raw):
    """What the calls on a busy side stream read may be let go of as soon as they return."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    M, d, V = 64, 1024, 9000

    def inputs():
        ids, targets, W, weight, bias, way = _inputs(M, d, V, 3)
        z = W[:M, :].clone()
        starts = torch.arange(0, M + 1, 4, dtype=torch.int32, device="cuda")
        return (ids, W, weight, bias, z, starts, torch.full((M,), 0.5, device="cuda"),
                torch.full((1,), 3, device="cuda"), W[:M - len(starts) + 1].flip(1))

    def calls(stream, ids, W, weight, bias, z, starts, u, off, q):
        kw = {"stream": stream}
        e = sb.embedding(ids, W, **kw)
        b = sb.embedding_backward(ids, z, vocab=V, **kw)
        n = sb.layer_norm(z, weight, bias, y=z.flip(0), p=0.2, seed=1, seed_offset=off, **kw)
        k = sb.layer_norm_backward(z.flip(0), z.flip(1), z, weight, need_dy=True, p=0.2, seed=1,
                                   seed_offset=off, **kw)
        r = sb.dropout(z, 0.3, seed=2, seed_offset=off, residual=z.flip(0), **kw)
        v = sb.verify_drafts(z, ids % d, starts, u, draft_logits=q, lse=u + 6, draft_lse=(u + 6)[:len(q)],
                             seed=4, **kw)
        w = sb.verify_greedy(ids, ids.flip(0), starts, **kw)
        return e, b["dW"], n["h"], n["x"], k["dh"], k["dy"], k["dweight"], r, v["token"], w["token"]

    want = calls(None, *inputs())
    torch.cuda.synchronize()
    a = inputs()
    torch.cuda.synchronize()
    _busy(side)
    got = calls(stream, *a)
    del a
    junk = _reuse([((M, d), BF), ((V, d), BF), ((M,), torch.int32), ((1,), torch.int64), ((M,), F32),
                   ((d,), F32)])
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x, y), i
    del junk


@pytest.mark.parametrize("M,d,V", [(1, 1, 1), (5, 77, 9), (33, 1028, 40), (70, 640, 7), (8200, 24, 100)])
@pytest.mark.parametrize("t", [BF, F32])
def test_embedding_writes_its_own_arrays_only(M, d, V, t):
    g = Guards()
    kind = sb.SB_F32 if t is F32 else sb.SB_BF16
    ids = torch.randint(0, V, (M,), device="cuda", dtype=torch.int32)
    W, dout = torch.randn(V, d, device="cuda").to(t), torch.randn(M, d, device="cuda").to(t)
    out, dW = g.like((M, d), t), g.like((V, d), t)
    n = sb.sb_embedding_backward_workspace_bytes(M, d)
    ws = g.like((n,), torch.uint8)
    assert sb.sb_embedding_forward(ids, W, M, d, V, -100, 1.0, kind, kind, out) == sb.SB_OK
    for add in (0, 1):
        assert sb.sb_embedding_backward(ids, dout, M, d, V, -100, 1.0, kind, kind, add, dW, ws, n) == sb.SB_OK
    g.check()


@pytest.mark.parametrize("M,d", [(1, 1), (5, 77), (37, 1028), (400, 640), (160, 6144), (9, 8200)])
@pytest.mark.parametrize("t", [BF, F32])
def test_layer_norm_and_dropout_write_their_own_arrays_only(M, d, t):
    g = Guards()
    kind = sb.SB_F32 if t is F32 else sb.SB_BF16
    h, dh = (torch.randn(M, d, device="cuda").to(t) for _ in range(2))
    y, dx = (torch.randn(M, d, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(d, device="cuda")
    ho, x, out = g.like((M, d), t), g.like((M, d), BF), g.like((M, d), t)
    assert sb.sb_layer_norm_forward(h, y, w, w, M, d, kind, 1, 0.1, 1, None, 1e-5, ho, x) == sb.SB_OK
    assert sb.sb_dropout(y, h, M * d, 0, kind, 0.1, 1, None, out) == sb.SB_OK
    n = sb.sb_layer_norm_workspace_bytes(M, d)
    ws, dho, dy = g.like((n,), torch.uint8), g.like((M, d), t), g.like((M, d), BF)
    dw, db = g.like((d,), F32), g.like((d,), F32)
    assert sb.sb_layer_norm_backward(dx, dh, ho, w, M, d, kind, 1, 0.1, 1, None, 1e-5, dho, dy, dw, db, ws,
                                     n) == sb.SB_OK
    g.check()
    assert torch.equal(out, ho)


@pytest.mark.parametrize("lengths,V", [([0], 1), ([3, 0, 5], 777), ([2] * 40, 9001), ([1], 151936)])
def test_verification_writes_its_own_arrays_only(lengths, V):
    g = Guards()
    R, D, B = sum(lengths) + len(lengths), sum(lengths), len(lengths)
    starts = torch.tensor([sum(lengths[:b]) + b for b in range(B + 1)], dtype=torch.int32, device="cuda")
    z, q = torch.randn(R, V, device="cuda").bfloat16(), torch.randn(D, V, device="cuda").bfloat16()
    drafts = torch.zeros(R, dtype=torch.int32, device="cuda")
    token, accepted, lp = g.like((R,), torch.int32), g.like((B,), torch.int32), g.like((R,), F32)
    n = sb.sb_verify_workspace_bytes(R, D, V)
    ws = g.like((n,), torch.uint8)
    assert sb.sb_verify_drafts(z, q, drafts, starts, torch.full((R,), 0.7, device="cuda"), None, None, R, D, B, V,
                               0, 1.0, 5, token, accepted, lp, ws, n) == sb.SB_OK
    g.check()
    assert ((token >= -1) & (token < V)).all()
    assert sb.sb_verify_greedy(drafts, drafts, starts, R, B, token, accepted) == sb.SB_OK
    g.check()
