"""Preference loss and its gradient on the GPU against the float64 oracle.

Error of one exponential: the argument x = z - max (exact or half a float32
step) times log2 e, then the hardware's 1-ulp exponential: (2|x| + 3) 2^-24
relative.  A softmax sum adds one 2^-24 for each of the V / 256 + 24 additions
and rescalings on its longest path, so log sum is off by at most
E = (2 E|x| + 3 + 2 (V / 256 + 24)) 2^-24, E|x| <= the row's range; a token's
log probability by E and half its own step."""

import numpy as np
import pytest
import torch

from communication_avoiding_mixed_amd import binding as B
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def host(t):
    return t.double().cpu().numpy()


def make(tokens, vocab, pairs, dtype, seed, spread=2.5, extra=0, offset=0):
    rng = np.random.default_rng(seed)
    wide = torch.full((tokens, vocab + extra), float("nan"), dtype=T[dtype], device="cuda")
    z = wide[:, offset:offset + vocab]
    z.copy_(torch.from_numpy((rng.standard_normal((tokens, vocab)) * spread).astype(np.float32)))
    labels = rng.integers(0, vocab, tokens)
    labels[rng.random(tokens) < 0.3] = -100
    cuts = np.sort(rng.integers(0, tokens + 1, 2 * pairs - 1))
    offsets = np.concatenate([[0], cuts, [tokens]])
    ref = (rng.standard_normal(tokens) - np.log(vocab)).astype(np.float32)
    g = rng.standard_normal(pairs).astype(np.float32)
    return z, labels, offsets, ref, g


def gpu(a, dtype=None):
    return torch.from_numpy(np.asarray(a)).cuda()


def check(z, labels, offsets, ref, g, beta, kind, eps, average, dtype):
    zv = host(z)
    want = H.preference(zv, labels, offsets, ref, beta, kind, eps, average, g.astype(np.float64))
    fwd = B.pref_loss(z, gpu(labels), gpu(offsets), None if ref is None else gpu(ref), beta, kind, eps, average)
    vocab = zv.shape[1]
    span = float(np.max(zv.max(1) - zv.min(1))) if zv.size else 0.0
    err = (2 * span + 3 + 2 * (vocab / 256 + 24)) * U
    lp = host(fwd.logps)
    assert (np.abs(lp - want["logps"]) <= err + U * np.abs(want["logps"])).all()
    beta32, eps32 = float(np.float32(beta)), float(np.float32(eps))
    for p in range(len(g)):
        # each side's tokens are off by err each; beta and smoothing reach the kernel in float32
        off = 0.0
        for side in (0, 1):
            rows = [t for t in range(offsets[2 * p + side], offsets[2 * p + side + 1]) if labels[t] >= 0]
            off += err * (min(1, len(rows)) if average else len(rows))
        h, gh = want["margin"][p], float(host(fwd.margin)[p])
        assert abs(gh - h) <= off + U * abs(h)
        # the loss and slope are those of a margin within off of the oracle's, at the float32 beta and smoothing
        ls = [H.pair_loss(h + s * off, kind, beta32, eps32) for s in (-1, 0, 1)]
        lo, hi = min(l for l, _ in ls), max(l for l, _ in ls)
        if kind == "squared" and abs(h - 0.5 / beta32) <= off:
            lo = 0.0
        assert lo * (1 - 2 * U) - 1e-30 <= float(host(fwd.loss)[p]) <= hi * (1 + 2 * U)
        for side in (0, 1):
            share = want["slope"][2 * p + side] / H.pair_loss(h, kind, beta, eps)[1] if want["slope"][2 * p + side] else 1.0
            ends = sorted(d * share for _, d in ls)
            got = float(host(fwd.slope)[2 * p + side])
            assert ends[0] - 4 * U * abs(ends[0]) - 1e-30 <= got <= ends[-1] + 4 * U * abs(ends[-1]) + 1e-30
    # the gradient from the slopes the kernel kept, so that only its own error counts
    slope = host(fwd.slope)
    d = B.pref_grad(fwd, gpu(g))
    ref_d = np.zeros_like(zv)
    mag = np.zeros_like(zv)
    for s in range(2 * len(g)):
        for t in range(offsets[s], offsets[s + 1]):
            if labels[t] >= 0:
                q = np.exp(zv[t] - zv[t].max())
                q /= q.sum()
                coef = slope[s] * float(g[s // 2])
                ref_d[t] = -coef * q
                ref_d[t, labels[t]] += coef
                mag[t] = np.abs(coef) * q
                mag[t, labels[t]] += abs(coef)
    eps_out = torch.finfo(T[dtype]).eps / 2
    rel = err + (2 * span + 8) * U
    tol = rel * mag + eps_out * (np.abs(ref_d) + rel * mag) + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    got = host(d)
    assert (np.abs(got - ref_d) <= tol).all(), np.max(np.abs(got - ref_d) / tol)
    seq = np.full(len(zv), -1)
    for s in range(2 * len(g)):
        seq[offsets[s]:offsets[s + 1]] = s
    assert not got[(labels < 0) | (seq < 0)].any()
    return fwd, d


SHAPES = [(1, 1, 1), (2, 2, 1), (7, 33, 1), (40, 255, 3), (33, 2000, 4), (64, 257, 20), (10, 50001, 2), (300, 64, 2), (5, 8192, 2)]


@pytest.mark.parametrize("dtype", list(T))
@pytest.mark.parametrize("tokens,vocab,pairs", SHAPES)
def test_loss_and_gradient(tokens, vocab, pairs, dtype):
    for i, (kind, eps, average, beta, extra, offset) in enumerate([
            ("logistic", 0.0, False, 0.1, 0, 0), ("logistic", 0.2, True, 0.5, 8, 0), ("squared", 0.0, True, 0.3, 5, 3)]):
        z, labels, offsets, ref, g = make(tokens, vocab, pairs, dtype, i, 2.5, extra, offset)
        fwd, d = check(z, labels, offsets, ref, g, beta, kind, eps, average, dtype)
        again = B.pref_loss(z, gpu(labels), gpu(offsets), gpu(ref), beta, kind, eps, average)
        assert torch.equal(fwd.loss, again.loss) and torch.equal(fwd.stats, again.stats)
        assert torch.equal(fwd.logps, B.token_logps(z, gpu(labels)))
        wide = torch.zeros((tokens, vocab + 3), dtype=T[dtype], device="cuda")
        assert torch.equal(B.pref_grad(fwd, gpu(g), out=wide[:, 1:1 + vocab]), d)
        assert not wide[:, 0].any() and not wide[:, 1 + vocab:].any()
        assert torch.equal(B.pref_grad(fwd, gpu(g), out=z), d)  # in place


def test_without_reference_and_offsets_inside():
    z, labels, offsets, ref, g = make(30, 100, 2, "fp32", 5)
    offsets = np.array([3, 9, 9, 20, 25])
    check(z, labels, offsets, None, g, 0.2, "logistic", 0.0, False, "fp32")


def test_masked_vocabulary_and_rows_that_are_not_read():
    z, labels, offsets, ref, g = make(12, 70, 2, "fp32", 6)
    offsets = np.array([0, 3, 6, 9, 12])
    labels[:] = np.arange(12)
    labels[[0, 4]] = -1
    z[0], z[4] = float("nan"), float("inf")  # masked rows
    z[1:, 20:60] = float("-inf")             # words that cannot occur
    z[2, :] = torch.finfo(torch.float32).min  # a mask of the type's lowest value
    z[2, 2] = 0.0
    fwd = B.pref_loss(z, gpu(labels), gpu(offsets), gpu(ref))
    d = B.pref_grad(fwd, gpu(g))
    assert torch.isfinite(fwd.loss).all() and torch.isfinite(d).all()
    zv = host(z)
    zv[[0, 4]] = 0
    want = H.preference(zv, labels, offsets, ref, 0.1, grad_loss=g.astype(np.float64))
    np.testing.assert_allclose(host(fwd.logps), want["logps"], rtol=2e-6, atol=1e-5)
    assert not d[[0, 4]].any() and not d[1:, 20:60].any()
    assert float(fwd.logps[2]) == 0.0 and not d[2].any()


def test_impossible_labels():
    z, labels, offsets, ref, g = make(8, 50, 2, "fp32", 7)
    offsets = np.array([0, 2, 4, 6, 8])
    labels[:] = 1
    z[0, 1] = float("-inf")   # a label of probability zero: infinite loss, a finite gradient
    labels[5] = 50            # a label past the vocabulary: NaN, nothing read
    fwd = B.pref_loss(z, gpu(labels), gpu(offsets), gpu(ref))
    d = host(B.pref_grad(fwd, gpu(g)))
    assert np.isinf(host(fwd.loss)[0]) and np.isinf(host(fwd.logps)[0]) and np.isfinite(d[:4]).all()
    assert np.isnan(host(fwd.loss)[1]) and np.isnan(host(fwd.logps)[5]) and np.isnan(d[5]).all()
    z[2] = float("-inf")      # nothing can occur: NaN
    assert np.isnan(host(B.token_logps(z, gpu(labels)))[2])


def test_all_masked_and_empty():
    z, labels, offsets, ref, g = make(6, 40, 1, "bf16", 8)
    labels[:] = -5
    fwd = B.pref_loss(z, gpu(labels), gpu(np.array([0, 6, 6])), gpu(ref), average=True)
    assert abs(float(fwd.loss) - np.log(2)) < 1e-7 and not B.pref_grad(fwd, gpu(g)).any()
    none = torch.empty((0, 40), device="cuda")
    fwd = B.pref_loss(none, torch.empty(0, dtype=torch.int64, device="cuda"), gpu(np.zeros(3, np.int64)))
    assert abs(float(fwd.loss) - np.log(2)) < 1e-7 and B.pref_grad(fwd, gpu(g)).shape == (0, 40)


def test_long_gradient():
    # over 128 MiB: streamed stores; rows against torch's float64 on a sample
    tokens, vocab = 1100, 65543
    z, labels, offsets, ref, g = make(tokens, vocab, 2, "bf16", 14)
    fwd = B.pref_loss(z, gpu(labels), gpu(offsets), gpu(ref))
    d = B.pref_grad(fwd, gpu(g))
    slope = host(fwd.slope)
    for t in (0, 1, 500, 1099, int(offsets[1]), int(offsets[2])):
        t = min(t, tokens - 1)
        row, got = host(z[t]), host(d[t])
        s = max(i for i in range(4) if offsets[i] <= t)
        want = np.zeros(vocab)
        if labels[t] >= 0:
            q = np.exp(row - row.max())
            want = -slope[s] * float(g[s // 2]) * q / q.sum()
            want[labels[t]] += slope[s] * float(g[s // 2])
        # the exponential's and the sum's errors (2 * 30 + 2 * 280) 2^-24, then half a bf16 step
        assert (np.abs(got - want) <= (2.0 ** -8 + 700 * U) * np.abs(want) + 700 * U * np.abs(want).max()).all()


def test_bad_offsets_stay_inside():
    # not decreasing is the caller's part; values past the ends are clamped
    z, labels, offsets, ref, g = make(6, 40, 1, "fp32", 9)
    labels[:] = 1
    a = B.pref_loss(z, gpu(labels), gpu(np.array([-4, 3, 99])), gpu(ref))
    b = B.pref_loss(z, gpu(labels), gpu(np.array([0, 3, 6])), gpu(ref))
    assert torch.equal(a.loss, b.loss)
    assert torch.equal(B.pref_grad(a, gpu(g)), B.pref_grad(b, gpu(g)))


def test_large_margins():
    z, labels, offsets, ref, g = make(4, 9, 1, "fp32", 10)
    labels[:] = 2
    for shift in (1e4, -1e4):
        r = np.array([-shift, 0, 0, 0], np.float32)
        fwd = B.pref_loss(z, gpu(labels), gpu(np.array([0, 2, 4])), gpu(r), beta=1.0)
        lp = H.token_logps(host(z), labels)
        want = H.pair_loss(lp[:2].sum() - lp[2:].sum() + shift, "logistic", 1.0, 0.0)
        np.testing.assert_allclose(float(fwd.loss), want[0], rtol=1e-6, atol=1e-38)
        assert np.isfinite(float(fwd.slope[0]))


def test_gradient_against_differences_of_the_loss():
    z, labels, offsets, ref, g = make(6, 12, 1, "fp32", 11, 1.0)
    offsets, labels[:] = np.array([0, 3, 6]), [1, 5, -1, 3, 0, 11]
    fwd = B.pref_loss(z, gpu(labels), gpu(offsets), gpu(ref), 0.4)
    d = host(B.pref_grad(fwd, gpu(g)))
    for t, v in ((0, 1), (1, 2), (3, 3), (5, 0), (4, 11)):
        step = 2.0 ** -6
        up, down = z.clone(), z.clone()
        up[t, v] += step
        down[t, v] -= step
        a = float(B.pref_loss(up, gpu(labels), gpu(offsets), gpu(ref), 0.4).loss)
        b = float(B.pref_loss(down, gpu(labels), gpu(offsets), gpu(ref), 0.4).loss)
        # float32 losses of order one: 2^-24 * 8 / step; third derivative term step^2 / 6 * beta
        assert abs((a - b) / (2 * step) * g[0] - d[t, v]) <= abs(g[0]) * (8 * U * 4 / step + step ** 2 / 6 * 0.4)


def test_side_stream_and_graph_replays():
    z, labels, offsets, ref, g = make(50, 300, 3, "bf16", 12)
    lab, off, rf, gr = gpu(labels), gpu(offsets), gpu(ref), gpu(g)

    def step():
        fwd = B.pref_loss(z, lab, off, rf)
        return fwd.loss, fwd.margin, fwd.logps, B.pref_grad(fwd, gr)

    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        z.copy_(torch.randn(50, 300, device="cuda").bfloat16())
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)


def test_binding_refusals():
    z, labels, offsets, ref, g = make(6, 40, 1, "fp32", 13)
    lab, off = gpu(labels), gpu(offsets)
    for bad in (lab[:5], lab.to(torch.int32), lab.cpu()):
        with pytest.raises(ValueError, match="labels"):
            B.pref_loss(z, bad, off)
    for bad in (off[:2], off.cpu(), off.to(torch.int32)):
        with pytest.raises(ValueError, match="offsets"):
            B.pref_loss(z, lab, bad)
    with pytest.raises(ValueError, match="ref_logps"):
        B.pref_loss(z, lab, off, gpu(ref).double())
    with pytest.raises(B.CasgdError, match="beta"):
        B.pref_loss(z, lab, off, beta=-1.0)
    with pytest.raises(B.CasgdError, match="smoothing"):
        B.pref_loss(z, lab, off, smoothing=0.1, loss="squared")
    fwd = B.pref_loss(z, lab, off)
    with pytest.raises(ValueError, match="grad_loss"):
        B.pref_grad(fwd, torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="out must"):
        B.pref_grad(fwd, gpu(g), out=torch.zeros(6, 41, device="cuda"))
    with pytest.raises(ValueError, match="out must"):
        B.pref_grad(fwd, gpu(g), out=torch.zeros(6, 40, device="cuda", dtype=torch.float16))


def test_offsets_past_32_bits():
    # 8.7 GB of bf16 logits; only the last rows are labelled, the others are not read
    tokens, vocab = 66001, 65536
    z = torch.empty((tokens, vocab), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(4, vocab, device="cuda").bfloat16()
    z[-4:] = tail
    labels = torch.full((tokens,), -1, dtype=torch.int64)
    labels[-4:] = torch.tensor([vocab - 1, 5, 77, vocab - 2])
    offsets = torch.tensor([0, tokens - 2, tokens])
    fwd = B.pref_loss(z, labels.cuda(), offsets.cuda())
    lp = H.token_logps(host(tail), labels[-4:].numpy())
    np.testing.assert_allclose(host(fwd.logps[-4:]), lp, rtol=3e-6)
    d = B.pref_grad(fwd, torch.ones(1, device="cuda"))
    small = B.pref_loss(tail, labels[-4:].cuda(), torch.tensor([0, 2, 4]).cuda())
    assert abs(float(fwd.loss) - float(small.loss)) <= 1e-5
    ref = host(B.pref_grad(small, torch.ones(1, device="cuda")))
    # the two calls' sums run in another order: slopes and softmax differ by a few float32 steps, then bf16's
    assert (np.abs(host(d[-4:]) - ref) <= 2.0 ** -7 * np.abs(ref) + 1e-12).all()
    assert not d[:-4].any()
