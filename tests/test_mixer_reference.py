"""Pins of the 64-bit reference of the gated delta rule and the group norm:
properties and independent forms, and gradients against differences."""

import numpy as np
import pytest
import torch

from tests import mixer_reference as ref


def test_beta_zero_is_pure_decay():
    w = ref.make_gdr(1, 9, 2, 3, 1, 4, torch.float64, 1)
    w["beta"] = torch.zeros_like(w["beta"])
    y, h = ref.gdr_of(w, True)
    d = torch.nn.functional.softplus(w["dt"].double() + w["bias"].double())
    total = torch.exp((d * w["A"].double()).sum(1))
    torch.testing.assert_close(h, w["h0"].double() * total[..., None, None])


def test_full_write_recalls_the_value():
    """beta = 1 and a unit key: the state then answers exactly v for that key."""
    w = ref.make_gdr(1, 5, 1, 3, 1, 4, torch.float64, 2)
    w["beta"] = torch.ones_like(w["beta"])
    _, h = ref.gdr_of(w, True)
    k = w["k"][0, -1, 0].double()
    k = k / k.norm()
    # the norm's epsilon leaves |k|^2 = 1 - O(1e-6)
    torch.testing.assert_close(h[0, 0] @ k, w["v"][0, -1, 0].double(), rtol=1e-5, atol=1e-5)


def test_matrix_form():
    """S_t = a S_{t-1} (I - beta k k^T) + beta v k^T, by dense products."""
    w = ref.make_gdr(1, 6, 2, 3, 1, 4, torch.float64, 3, qk_norm=False, bias=False)
    y, h = ref.gdr_of(w, False, scale=0.7)
    for hd in range(2):
        S = w["h0"][0, hd].double()
        for t in range(6):
            k, q, v = (w[n][0, t, 0 if n != "v" else hd].double() for n in ("k", "q", "v"))
            a, be = torch.exp(w["dt"][0, t, hd] * w["A"][hd]), w["beta"][0, t, hd]
            S = a * S @ (torch.eye(4, dtype=torch.float64) - be * torch.outer(k, k)) + be * torch.outer(v, k)
            torch.testing.assert_close(y[0, t, hd], 0.7 * S @ q)
        torch.testing.assert_close(h[0, hd], S)


@pytest.mark.parametrize("qk_norm", [False, True])
def test_gdr_gradients_against_differences(qk_norm):
    w = ref.make_gdr(1, 4, 2, 2, 1, 3, torch.float64, 4, qk_norm=qk_norm)
    w = {n: t.double() for n, t in w.items()}
    grads = ref.gdr_grads_of(w, qk_norm)

    def loss():
        y, h = ref.gdr_of(w, qk_norm)
        return ((y * w["dy"]).sum() + (h * w["dh"]).sum()).item()

    for n in ref.NAMES:
        flat = w[n].view(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 6)):
            old = flat[i].item()
            flat[i] = old + 1e-5
            up = loss()
            flat[i] = old - 1e-5
            down = loss()
            flat[i] = old
            assert abs((up - down) / 2e-5 - grads[n].view(-1)[i].item()) < 1e-7, n


def test_norm_is_torch_group_norm():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 7, 12, generator=g, dtype=torch.float64)
    w, b = torch.randn(12, generator=g, dtype=torch.float64), torch.randn(12, generator=g, dtype=torch.float64)
    want = torch.nn.functional.group_norm(x.movedim(2, 1), 3, w, b, 1e-5).movedim(1, 2)
    torch.testing.assert_close(ref.norm(x, 3, w, b, per_token=False), want)
    want = torch.nn.functional.group_norm(x.reshape(14, 12), 3, w, b, 1e-5).reshape(2, 7, 12)
    torch.testing.assert_close(ref.norm(x, 3, w, b), want)


def test_norm_gates():
    g = torch.Generator().manual_seed(6)
    x, z = (torch.randn(1, 2, 4, generator=g, dtype=torch.float64) for _ in range(2))
    s = z.numpy() / (1 + np.exp(-z.numpy()))
    u = x.numpy() * s
    want = u / np.sqrt((u ** 2).mean(-1, keepdims=True) + 1e-5)
    np.testing.assert_allclose(ref.norm(x, 1, z=z, center=False, gate="before").numpy(), want)
    n = x.numpy() / np.sqrt((x.numpy() ** 2).mean(-1, keepdims=True) + 1e-5)
    np.testing.assert_allclose(ref.norm(x, 1, z=z, center=False, gate="after").numpy(), n * s)
