"""Verification of drafted tokens against the definition in 64 bits.

Tolerances: a log-probability y - lse, with y = z·(1/T) rounded to fp32 and lse a sum of V
exponentials, is off by at most D = 2^-22·(max|y| + |lse| + 4): the product's and the difference's
roundings (e each), the reference's own lse against one from fp32 (max, sum) pieces whose exponentials
are within 2^-22 of their arguments' e, and the caller's where it is one in fp32.  A ratio p/q is then
off by 2D relatively, a weight p - q by D(p + q), a score w / -log u by that over w and 2^-19 (the
logarithm's 1e-6 and its division).  Where a decision is nearer than that to its border both answers
are right and the rest of the request is not compared; everywhere else the answers have to be equal.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_dropout import splitmix

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _make(lengths, V, *, kind=BF, draft=True, seed=0, spread=2.0, noise=0.7, T=1.0, behind=0):
    """Requests with the given numbers of drafts (None: a request without rows)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = [0 if n is None else n + 1 for n in lengths]
    R, D = sum(rows) + behind, sum(n or 0 for n in lengths)
    z = (spread * torch.randn(R, V, generator=g, device="cuda")).to(kind)
    starts = np.concatenate([[0], np.cumsum(rows)])
    drafted = [int(starts[b]) + i for b, n in enumerate(lengths) for i in range(n or 0)]
    at = torch.tensor(drafted, dtype=torch.long, device="cuda")
    q = (z[at].float() + noise * torch.randn(D, V, generator=g, device="cuda")).to(kind)
    drafts = torch.full((R,), -5, dtype=torch.int32, device="cuda")
    if D:
        noise = -torch.log(-torch.log(torch.rand(D, V, generator=g, device="cuda").clamp(1e-7, 1 - 1e-6)))
        drafts[at] = ((q if draft else z[at]).float() / T + noise).argmax(1).int()
    return {"logits": z, "draft_logits": q if draft else None, "drafts": drafts,
            "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "uniforms": torch.rand(R, generator=g, device="cuda")}


def _logs(row, inv_t, given=None):
    y = (row.float() * inv_t).double().cpu().numpy()
    top = y.max()
    lse = top + np.log(np.exp(y - top).sum()) if given is None else float(given)
    d = 2.0 ** -22 * (np.abs(y[np.isfinite(y)]).max() + abs(lse) + 4)
    return y - lse, d


def _reference(s, T=1.0, seed=0, lse=None, draft_lse=None):
    """(per request: token list or None where it is ambiguous from there on, log-probs, bounds)."""
    inv_t = float(np.float32(1) / np.float32(T))
    z, q, V = s["logits"], s["draft_logits"], s["logits"].shape[1]
    drafts, u, starts = s["drafts"].tolist(), s["uniforms"].tolist(), s["starts"].tolist()
    answers, at = [], 0
    for b in range(len(starts) - 1):
        first, n = starts[b], starts[b + 1] - starts[b] - 1
        out = []
        for i in range(n + 1):
            r = first + i
            lp, d = _logs(z[r], inv_t, None if lse is None else lse[r])
            w, dw = np.exp(lp), d * np.exp(lp)
            if i < n:
                x = drafts[r]
                if 0 <= x < V:
                    ratio, off = np.exp(lp[x]), d
                    if q is not None:
                        lq, e = _logs(q[at + i], inv_t, None if draft_lse is None else draft_lse[at + i])
                        with np.errstate(invalid="ignore"):  # (two columns without probability)
                            ratio, off = np.exp(np.minimum(lp[x] - lq[x], 700.0)), d + e
                    if abs(ratio - u[r]) <= 2 * off * max(ratio, u[r]):
                        out.append(None)
                        break
                    if ratio > u[r]:
                        out.append((x, lp[x], d))
                        continue
                    if q is None:
                        w[x] = 0
                    else:
                        w, dw = np.maximum(w - np.exp(lq), 0), d * w + e * np.exp(lq)
            if w.max() <= 0:
                w, dw = np.exp(lp), d * np.exp(lp)
            bits = (splitmix(np.arange(r * V, (r + 1) * V, dtype=np.uint64), seed) >> np.uint64(40)).astype(np.float64)
            with np.errstate(divide="ignore", invalid="ignore"):
                t = -np.log(bits * 2.0 ** -24)
                low, high = (w - dw) / t * (1 - 2.0 ** -19), (w + dw) / t * (1 + 2.0 ** -19)
                score = w / t
            j = int(np.argmax(score))
            rivals = (high >= low[j]) & (score != score[j])
            out.append(None if rivals.any() else (j, lp[j], d))
            break
        answers.append((first, n, out))
        at += max(n, 0)
    return answers


def _check(s, T=1.0, seed=0, least=0.98, **kw):
    f = sb.verify_drafts(**s, temperature=T, seed=seed, **kw)
    assert sb.device_status(f["workspace"]) == sb.SB_OK
    token, accepted, lp = f["token"].tolist(), f["accepted"].tolist(), f["token_logprob"].tolist()
    sure = 0
    answers = _reference(s, T, seed, kw.get("lse"), kw.get("draft_lse"))
    for b, (first, n, out) in enumerate(answers):
        if n < 0:
            assert accepted[b] == 0
            sure += 1
            continue
        for i, want in enumerate(out):
            if want is None:
                break
            x, value, d = want
            assert token[first + i] == x, (b, i)
            assert abs(lp[first + i] - value) <= d + 2.0 ** -23 * abs(value), (b, i)
        else:
            sure += 1
            assert accepted[b] == len(out) - 1, b
            assert token[first + len(out):first + n + 1] == [-1] * (n + 1 - len(out))
            assert lp[first + len(out):first + n + 1] == [0.0] * (n + 1 - len(out))
    end = s["starts"].tolist()[-1]
    assert token[end:] == [-1] * (len(token) - end) and lp[end:] == [0.0] * (len(token) - end)
    assert sure >= least * len(answers)
    return f


@gpu
@pytest.mark.parametrize("lengths", [[0], [1], [4], [3, 0, 1, 5], [None, 2, None, None, 7, 0], [None],
                                     [2] * 33, [40], [700, 3]])
@pytest.mark.parametrize("V", [1, 2, 7, 1003, 4096])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("draft", [True, False])
def test_against_the_definition(lengths, V, kind, draft):
    s = _make(lengths, V, kind=kind, draft=draft, seed=V + len(lengths))
    _check(s, seed=V)


@gpu
@pytest.mark.parametrize("B", [9, 10, 38, 39, 76, 77, 152, 153, 400])
@pytest.mark.parametrize("draft", [True, False])
def test_many_requests(B, draft):
    """Each number of blocks to a request, and more requests than fit the GPU at a time."""
    s = _make([(5 * b) % 4 for b in range(B)], 1003, draft=draft, seed=B)
    _check(s, seed=B)


@gpu
@pytest.mark.parametrize("V", [50257, 151936, 200064])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("draft,T", [(True, 0.7), (False, 1.3), (True, 1.0)])
def test_large_vocabularies(V, kind, draft, T):
    s = _make([4, 0, 6], V, kind=kind, draft=draft, seed=3, T=T)
    _check(s, T=T, seed=2 ** 64 - 3, least=0.6)


@gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("T", [0.01, 0.5, 100.0])
def test_temperatures(draft, T):
    _check(_make([5] * 12, 3001, draft=draft, seed=4, T=T), T=T, seed=9, least=0.9)


@gpu
def test_the_smallest_temperature():
    """A row's largest logits share it all, each with 1 / their number (of equal bf16 values there may be
    two): a draft stays if it is one of them and that is above u, and one of them replaces it."""
    s = _make([3, 2, 0], 500, seed=18)
    z, u = s["logits"].float(), s["uniforms"].tolist()
    best = z == z.amax(1, keepdim=True)
    p = (best.double() / best.sum(1, keepdim=True)).cpu()
    top = z.argmax(1).int()
    for drafts in (top, (top + 1) % 500):
        f = sb.verify_drafts(s["logits"], drafts, s["starts"], s["uniforms"], temperature=1e-30)
        for b, (a, end) in enumerate(zip(s["starts"].tolist(), s["starts"].tolist()[1:])):
            x = drafts[a:end].tolist()
            n = next((i for i in range(end - a - 1) if not p[a + i, x[i]] > u[a + i]), end - a - 1)
            assert f["accepted"][b] == n and f["token"][a:a + n].tolist() == x[:n]
            t = int(f["token"][a + n])
            # (without the refused draft, where another one is left)
            left = best[a + n].clone()
            if n < end - a - 1 and int(left.sum()) > int(left[x[n]]):
                left[x[n]] = False
            assert left[t]


@gpu
def test_given_logsumexps_are_taken():
    s = _make([3, 5, 0], 2003, seed=5)
    lse = torch.logsumexp(s["logits"].double(), 1).float()
    qlse = torch.logsumexp(s["draft_logits"].double(), 1).float()
    want = _check(s, seed=1)
    for kw in ({"lse": lse}, {"draft_lse": qlse}, {"lse": lse, "draft_lse": qlse}):
        got = _check(s, seed=1, **kw)
        assert torch.equal(got["token"], want["token"])
    # other ones count: a target said to be a thousand times less likely keeps nothing
    got = sb.verify_drafts(**s, seed=1, lse=lse + 50, draft_lse=qlse)
    assert (got["accepted"] == 0).all()


@gpu
def test_rows_behind_the_last_request_and_no_requests():
    s = _make([2, 0], 333, seed=6, behind=700)
    f = _check(s, seed=2)
    assert (f["token"][4:] == -1).all()
    s["starts"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = sb.verify_drafts(**s)
    assert (f["token"] == -1).all() and (f["token_logprob"] == 0).all() and f["accepted"].shape == (0,)
    s = _make([], 10)
    assert sb.verify_drafts(**s)["token"].shape == (0,)


@gpu
def test_columns_without_probability():
    """Masked columns are never drafted successfully and never sampled; rows of one column."""
    V = 1000
    s = _make([6] * 20, V, seed=7)
    off = torch.rand(V, device="cuda") < 0.9
    off[0] = False
    s["logits"][:, off] = float("-inf")
    f = _check(s, seed=3)
    t = f["token"]
    assert not off[t[t >= 0].long()].any()
    s["draft_logits"][:, off] = float("-inf")
    _check(s, seed=3)
    # all but one column
    s["logits"][:] = float("-inf")
    s["logits"][:, 17] = -3.0
    s["drafts"][:] = 17
    f = _check(s, seed=3)
    assert (f["token"] == 17).all() and (f["token_logprob"] == 0).all() and (f["accepted"] == 6).all()


@gpu
def test_a_row_without_any_column():
    s = _make([3, 3], 500, seed=8)
    s["draft_logits"][:] = s["logits"][[0, 1, 2, 4, 5, 6]]  # every draft stays ...
    s["logits"][2] = float("-inf")                          # ... but where nothing is left
    s["logits"][7] = float("nan")
    f = sb.verify_drafts(**s)
    assert f["accepted"].tolist() == [2, 3]
    assert f["token"][:2].tolist() == s["drafts"][:2].tolist() and f["token"][2:4].tolist() == [-1, -1]
    assert f["token"][4:7].tolist() == s["drafts"][4:7].tolist() and f["token"][7] == -1
    lp = f["token_logprob"]
    assert lp[[2, 7]].isnan().all() and lp[3] == 0 and torch.isfinite(lp[[0, 1, 4, 5, 6]]).all()


@gpu
def test_equal_distributions_keep_every_draft():
    V = 4097
    s = _make([8] * 30, V, noise=0.0, seed=9)
    s["uniforms"].fill_(1 - 2.0 ** -12)  # p/q = 1 but for the bound's 2D, some 2^-17
    f = sb.verify_drafts(**s)
    assert (f["accepted"] == 8).all()
    # a draft that is refused although p = q: the difference is nowhere positive, p is sampled
    s["uniforms"].fill_(2.0)
    f = sb.verify_drafts(**s, seed=4)
    bonus = sb.verify_drafts(logits=s["logits"][::9].contiguous(), drafts=s["drafts"][::9].contiguous(),
                             starts=torch.arange(31, dtype=torch.int32, device="cuda"),
                             uniforms=s["uniforms"][::9].contiguous())
    assert (f["accepted"] == 0).all() and (f["token"][::9] >= 0).all()
    assert bonus["token"].shape == (30,)


@gpu
def test_the_tokens_are_distributed_as_the_targets():
    """The first token of 40000 requests against p, whatever q: a chi-square of six degrees of freedom
    is below 40 but for 5 in 10 million."""
    V, B = 7, 40_000
    g = torch.Generator(device="cuda").manual_seed(10)
    zp = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -2.0, 1.5], device="cuda")
    zq = torch.tensor([1.5, -1.0, 0.0, 0.5, 2.0, 0.0, -3.0], device="cuda")
    starts = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    T = 0.8
    p, q = (torch.softmax(x / T, 0) for x in (zp, zq))
    drafts = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    for with_q in (True, False):
        drafts[::2] = torch.multinomial(q, B, replacement=True, generator=g).int() if with_q else 4
        f = sb.verify_drafts(zp.expand(2 * B, V).contiguous(), drafts, starts,
                             torch.rand(2 * B, generator=g, device="cuda"),
                             draft_logits=zq.expand(B, V).contiguous() if with_q else None,
                             temperature=T, seed=12)
        for first, count in ((f["token"][::2], B), (f["token"][1::2][f["accepted"] == 1], None)):
            n = first.numel() if count is None else count
            seen = torch.bincount(first.long(), minlength=V).double()
            chi = ((seen - n * p.double()) ** 2 / (n * p.double())).sum()
            assert chi < 40, (with_q, count, float(chi))
        # a draft stays with probability sum of min(p, q): five deviations
        a = float(torch.minimum(p, q).sum()) if with_q else float(p[4])
        assert abs(float(f["accepted"].double().mean()) - a) < 5 * (a * (1 - a) / B) ** 0.5


@gpu
def test_samples_are_those_of_the_projection():
    """Where all drafts stay the last row's sample is the Gumbel-max choice of SB_GUMBEL_TOKEN (keys
    nearer than 1e-5 aside): here with logits that bf16 holds exactly, columns of W themselves."""
    M, d, V, T, seed = 16, 64, 4096, 0.9, 99
    g = torch.Generator(device="cuda").manual_seed(11)
    W = (2 * torch.randn(V, d, generator=g, device="cuda")).bfloat16()
    H = torch.zeros(M, d, device="cuda", dtype=BF)
    H[torch.arange(M), torch.arange(M)] = 1
    want = sb.project(H, W, 2, sb.SB_GUMBEL_TOKEN, temperature=T, seed=seed)
    full = sb.project(H, W, 2, sb.SB_FULL_LOGITS)
    assert torch.equal(full["logits"], W[:, :M].t())
    got = sb.verify_drafts(full["logits"], torch.zeros(M, dtype=torch.int32, device="cuda"),
                           torch.arange(M + 1, dtype=torch.int32, device="cuda"),
                           torch.zeros(M, device="cuda"), temperature=T, seed=seed)
    y = full["logits"].double().cpu().numpy() / T
    bits = (splitmix(np.arange(M * V, dtype=np.uint64), seed) >> np.uint64(40)).reshape(M, V)
    with np.errstate(divide="ignore"):
        keys = np.sort(y - np.log(-np.log(bits.astype(np.float64) * 2.0 ** -24)), 1)
    clear = torch.from_numpy(keys[:, -1] - keys[:, -2] > 1e-5).cuda()
    assert clear.sum() >= M - 1
    assert torch.equal(got["token"][clear], want["token"][clear])
    # 5e-3 is the projection's own tolerance
    assert ((got["token_logprob"] - want["token_logprob"]).abs()[clear] <= 5e-3).all()


@gpu
def test_tokens_and_starts_out_of_range():
    V = 777
    s = _make([3, 2, 4], V, seed=12)
    s["draft_logits"] = s["draft_logits"].copy_(s["logits"][[0, 1, 2, 4, 5, 7, 8, 9, 10]])  # p = q
    s["uniforms"].fill_(0.5)
    clean = sb.verify_drafts(**s, seed=5)
    assert clean["accepted"].tolist() == [3, 2, 4]
    for bad in (-1, V, 2 ** 31 - 1, -2 ** 31):
        t = dict(s, drafts=s["drafts"].clone())
        t["drafts"][5] = bad
        f = sb.verify_drafts(**t, seed=5)
        assert sb.device_status(f["workspace"]) == sb.SB_ERR_INVALID_ARG
        assert f["accepted"].tolist() == [3, 1, 4] and 0 <= f["token"][5] < V and f["token"][6] == -1
        keep = [0, 1, 2, 3, 4, 7, 8, 9, 10, 11]
        assert torch.equal(f["token"][keep], clean["token"][keep])
    for starts, accepted in (([0, 4, 2, 12], [3, -1, None]), ([0, 4, 7, 13], [-1, -1, -1]),
                             ([-3, 4, 7, 12], [-1, None, None]),
                             ([0, 4, 7, 2 ** 31 - 1], [-1, -1, -1]), ([5, -2 ** 31, 7, 12], [-1, -1, None])):
        f = sb.verify_drafts(**dict(s, starts=torch.tensor(starts, dtype=torch.int32, device="cuda")), seed=5)
        assert sb.device_status(f["workspace"]) == sb.SB_ERR_INVALID_ARG
        for got, want in zip(f["accepted"].tolist(), accepted):
            assert want is None or got == want, (starts, f["accepted"].tolist())
    # fewer draft rows than drafts
    f = sb.verify_drafts(**dict(s, draft_logits=s["draft_logits"][:6].contiguous()), seed=5)
    assert f["accepted"].tolist() == [3, 2, -1]
    assert sb.device_status(f["workspace"]) == sb.SB_ERR_INVALID_ARG
    f = sb.verify_drafts(**dict(s, draft_logits=s["draft_logits"][:0]), seed=5)
    assert f["accepted"].tolist() == [-1, -1, -1]


@gpu
def test_repeats_streams_and_graphs_give_the_same_answers():
    s = _make([4, 1, 0, 7] * 8, 20011, seed=13)
    want = _check(s, seed=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    names = ("token", "accepted", "token_logprob")
    for stream in (None, side, side.cuda_stream):
        for _ in range(5):
            f = sb.verify_drafts(**s, seed=6, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(f[k], want[k]) for k in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = sb.verify_drafts(**s, seed=6)
    other = _make([0, 2, None, 5] * 8, 20011, seed=14)
    for k in ("logits", "draft_logits", "drafts", "uniforms"):
        n = min(len(s[k]), len(other[k]))
        s[k][:n].copy_(other[k][:n])
    s["starts"].copy_(other["starts"])  # fewer rows than before
    graph.replay()
    torch.cuda.synchronize()
    want = _check(s, seed=6)
    assert all(torch.equal(f[k], want[k]) for k in names)


@gpu
def test_offsets_past_32_bits():
    V, n = 151936, 20_000
    small = _make([1, 2], V, seed=15)
    z = torch.zeros(n, V, dtype=BF, device="cuda")
    z[-5:] = small["logits"]
    drafts = torch.zeros(n, dtype=torch.int32, device="cuda")
    drafts[-5:] = small["drafts"]
    u = torch.zeros(n, device="cuda")
    u[-5:] = small["uniforms"]
    # many rows of requests without drafts, and the small batch behind them
    starts = torch.cat([torch.arange(n - 5, device="cuda"), small["starts"] + n - 5]).int()
    f = sb.verify_drafts(z, drafts, starts, u, draft_logits=small["draft_logits"], seed=7)
    # the draws go by the row's number: the same stream, moved there
    moved = (7 + (n - 5) * V * 0x9E3779B97F4A7C15) % 2 ** 64
    want = sb.verify_drafts(**small, seed=moved)
    assert torch.equal(f["token"][-5:], want["token"]) and torch.equal(f["accepted"][-2:], want["accepted"])
    assert (f["token"] >= -1).all() and (f["accepted"][:-2] == 0).all()


@gpu
def test_greedy():
    i32 = torch.int32
    target = torch.tensor([5, 6, 7, 8, 1, 2, 9, 4, 4], dtype=i32, device="cuda")
    drafts = torch.tensor([5, 6, 0, 8, 1, 2, 9, 3, 4], dtype=i32, device="cuda")
    starts = torch.tensor([0, 4, 4, 6, 8], dtype=i32, device="cuda")
    f = sb.verify_greedy(target, drafts, starts)
    assert f["token"].tolist() == [5, 6, 7, -1, 1, 2, 9, 4, -1] and f["accepted"].tolist() == [2, 0, 1, 1]
    g = torch.Generator(device="cuda").manual_seed(16)
    lengths = [1, 2, 33, 64, 65, 300, 1]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=i32, device="cuda")
    R = int(starts[-1])
    target = torch.randint(0, 100, (R,), generator=g, device="cuda", dtype=i32)
    for share in (0.0, 0.02, 1.0):
        drafts = torch.where(torch.rand(R, generator=g, device="cuda") < share, target + 1, target)
        f = sb.verify_greedy(target, drafts, starts)
        for b, n in enumerate(lengths):
            a = int(starts[b])
            t, d = target[a:a + n].tolist(), drafts[a:a + n].tolist()
            e = next((i for i in range(n - 1) if t[i] != d[i]), n - 1)
            assert f["accepted"][b] == e and f["token"][a:a + n].tolist() == t[:e + 1] + [-1] * (n - 1 - e)
    bad = torch.tensor([0, 5, 3, R + 1, 4, 5, 6, 7], dtype=i32, device="cuda")
    assert sb.verify_greedy(target, drafts, bad)["accepted"][1:3].tolist() == [-1, -1]
    none = sb.verify_greedy(target, drafts, bad[:1])
    assert (none["token"] == -1).all() and none["accepted"].shape == (0,)


@gpu
def test_refusals():
    s = _make([2], 40, seed=17)
    for bad in ({"logits": s["logits"].half()}, {"drafts": s["drafts"].long()}, {"starts": s["starts"].long()},
                {"uniforms": s["uniforms"].double()}, {"draft_logits": s["draft_logits"].float()},
                {"lse": torch.zeros(3, dtype=BF, device="cuda")}):
        with pytest.raises(TypeError):
            sb.verify_drafts(**{**s, **bad})
    for bad in ({"logits": s["logits"][0]}, {"logits": s["logits"].t()}, {"drafts": s["drafts"][:2]},
                {"starts": s["starts"][:0]}, {"uniforms": s["uniforms"].cpu()}, {"seed": 2 ** 64},
                {"draft_logits": s["draft_logits"][:, :39]}, {"lse": torch.zeros(2, device="cuda")},
                {"draft_lse": torch.zeros(3, device="cuda")},
                {"draft_logits": None, "draft_lse": torch.zeros(2, device="cuda")}):
        with pytest.raises(ValueError):
            sb.verify_drafts(**{**s, **bad})
    for T in (0.0, -1.0, float("inf"), float("nan"), 1e-42, 9e-31):
        with pytest.raises(sb.SbError):
            sb.verify_drafts(**s, temperature=T)
    with pytest.raises(sb.SbError):
        sb.verify_drafts(**s, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        sb.verify_greedy(s["drafts"].long(), s["drafts"], s["starts"])
    with pytest.raises(ValueError):
        sb.verify_greedy(s["drafts"], s["drafts"][:2], s["starts"])


def test_c_refusals():
    P = 1 << 20

    def call(z=P, q=P, drafts=P, starts=P, u=P, lse=P, qlse=P, R=4, D=3, B=1, V=100, kind=0, T=1.0, token=P,
             accepted=P, lp=P, ws=P, n=1 << 30):
        return sb.sb_verify_drafts(z, q, drafts, starts, u, lse, qlse, R, D, B, V, kind, T, 0, token, accepted,
                                   lp, ws, n, 0)

    for kw in ({"z": None}, {"q": None}, {"drafts": None}, {"starts": None}, {"u": None}, {"R": -1},
               {"R": 2 ** 24}, {"D": -2}, {"D": 2 ** 24}, {"B": -1}, {"B": 2 ** 25}, {"V": 0}, {"V": 2 ** 31},
               {"kind": 2}, {"T": 0.0}, {"T": float("nan")}, {"token": None}, {"accepted": None}, {"ws": None}):
        assert call(**kw) == sb.SB_ERR_INVALID_ARG, kw
    for kw in ({"z": P + 1}, {"z": P + 2, "kind": 1}, {"q": P + 1}, {"drafts": P + 2}, {"starts": P + 1},
               {"u": P + 2}, {"lse": P + 2}, {"qlse": P + 1}, {"token": P + 2}, {"accepted": P + 2},
               {"lp": P + 2}, {"ws": P + 64}):
        assert call(**kw) == sb.SB_ERR_ALIGNMENT, kw
    assert sb.sb_verify_workspace_bytes(-1, 0, 10) == 0 and sb.sb_verify_workspace_bytes(1, 0, 0) == 0
    assert sb.sb_verify_workspace_bytes(0, -1, 10) > 0
    for kw in ({"target": None}, {"drafts": None}, {"starts": None}, {"R": -1}, {"B": -1}, {"token": None},
               {"accepted": None}):
        a = {"target": P, "drafts": P, "starts": P, "R": 4, "B": 1, "token": P, "accepted": P, **kw}
        assert sb.sb_verify_greedy(*a.values(), 0) == sb.SB_ERR_INVALID_ARG, kw
    assert sb.sb_verify_greedy(P + 2, P, P, 4, 1, P, P, 0) == sb.SB_ERR_ALIGNMENT
