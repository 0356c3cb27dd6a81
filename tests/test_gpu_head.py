"""A preference-trained head: one step of every operator together against the
float64 oracle, and a short run whose loss falls."""

import numpy as np
import pytest
import torch

from communication_avoiding_mixed_amd import binding as B
from communication_avoiding_mixed_amd import head as HD
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu


def host(t):
    return t.double().cpu().numpy()


def test_one_step_against_the_oracle():
    pairs, length, features, vocab, eta = 3, 9, 200, 300, 0.3
    h, labels, offsets = HD.synthetic_pairs(pairs, length, features, vocab, 3)
    gen = torch.Generator().manual_seed(4)
    w0 = torch.randn(vocab, features, generator=gen) / features ** 0.5
    head = HD.PreferenceHead(w0.clone().cuda(), beta=0.2)
    ref = head.reference_logps(h, labels) * 0.9
    fwd, dh = head.step(h, labels, offsets, ref, eta, need_dfeatures=True)

    hv, w4 = host(h), H.rounded(w0.numpy(), "mx4")
    z = torch.from_numpy(H.rounded(hv, "mx4") @ w4.T).bfloat16().double().numpy()
    want = H.preference(z, labels.cpu().numpy(), offsets.cpu().tolist(), host(ref), 0.2, grad_loss=np.full(pairs, 1 / pairs))
    # logits that round to the neighbouring bf16 value move a token's log
    # probability by up to 2^-8 |z|; few do, and 7 tokens a sequence sum up
    np.testing.assert_allclose(host(fwd.margin), want["margin"], atol=14 * 2.0 ** -8 * 4)
    dz = want["dlogits"]
    slack = 3 * 2.0 ** -8  # dlogits are rounded to bf16, from logits that were
    x8 = H.rounded(hv, "mx8")
    assert np.linalg.norm(host(dh) - dz @ w4) <= slack * np.linalg.norm(dz @ w4)
    step = w0.double().numpy() - host(head.weight)
    assert np.linalg.norm(step - eta * dz.T @ x8) <= slack * np.linalg.norm(eta * dz.T @ x8)
    q = H.quantize(host(head.weight), "mx4")
    np.testing.assert_array_equal(head.w4.codes.cpu().numpy(), q[0])
    np.testing.assert_array_equal(head.w4.scales.cpu().numpy(), q[1])


def test_single_token_equals_its_row_of_the_batch():
    # the forms for few and many rows differ in the order of their float32 sums only
    gen = torch.Generator().manual_seed(5)
    head = HD.PreferenceHead(torch.randn(700, 512, generator=gen).cuda())
    h = torch.randn(300, 512, generator=gen).cuda()
    batch = host(head.logits(h))
    bound = 512 * 2.0 ** -22 * np.abs(H.rounded(host(h), "mx4")) @ np.abs(H.rounded(host(head.weight), "mx4")).T
    for rows in (1, 16, 32, 64):
        assert (np.abs(host(head.logits(h[:rows])) - batch[:rows]) <= bound[:rows]).all()


def test_loss_falls():
    h, labels, offsets = HD.synthetic_pairs(8, 16, 256, 512)
    gen = torch.Generator().manual_seed(1)
    head = HD.PreferenceHead((torch.randn(512, 256, generator=gen) / 16).cuda())
    ref = head.reference_logps(h, labels)
    losses = []
    for _ in range(12):
        fwd, _ = head.step(h, labels, offsets, ref, 0.2)
        losses.append(float(fwd.loss.mean()))
    assert abs(losses[0] - np.log(2)) < 1e-6  # the policy starts as the reference
    assert losses[-1] < 0.5 * losses[0] and float((fwd.margin > 0).float().mean()) == 1.0


def test_weights_must_be_float32():
    with pytest.raises(ValueError, match="float32"):
        HD.PreferenceHead(torch.zeros(4, 64, device="cuda").half())
