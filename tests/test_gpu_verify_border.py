"""Verification of drafted tokens where decisions stand on the border: sides that differ by a rounding of an input and no
more.  Sums in fp32 get part of them wrong, which every test shows for its own inputs; the kernel's answers have to be
those of 64 bits, whose own error (1e-15) is far below the smallest distance there is here."""
import numpy as np
import pytest

from batch_ref import verify

torch = pytest.importorskip("torch")

from decoder_only_transformer_gb300 import tfm  # noqa: E402

INF = float("inf")


def _call(target, dl, draft, u, noise, V, temperature):
    B, K = draft.shape
    ws = torch.full((tfm.verify_draft_workspace_bytes(B, K, V),), 255, dtype=torch.uint8, device="cuda")
    tokens = torch.full((B, K + 1), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    a = [t.cuda() for t in (target, dl, draft)], [t.cuda() for t in (u, noise)]
    tfm.verify_draft(*a[0], None, *a[1], V, tokens, acc, ws, temperature=temperature)
    tfm.device_status()
    return tokens.cpu().numpy(), acc.cpu().numpy()


def _same(target, dl, draft, u, noise, V, temperature):
    B, K = draft.shape
    want = verify(target, dl if K else None, draft, [K] * B, u, noise, V, float(np.float32(temperature)))
    got = _call(target, dl, draft, u, noise, V, temperature)
    assert np.array_equal(got[1], want[1]), np.flatnonzero(got[1] != want[1])
    assert np.array_equal(got[0], want[0]), np.flatnonzero((got[0] != want[0]).any(1))


def _logits(seed, B, K, V, off):
    g = torch.Generator().manual_seed(seed)
    ld = (V + 3) // 4 * 4
    target = torch.randn(B * (K + 1), ld, generator=g) * 2
    dl = target.view(B, K + 1, ld)[:, :K].reshape(B * K, ld) + off * torch.randn(B * K, ld, generator=g)
    return g, target, dl


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [1.0, 0.7, 1.3])
def test_races_of_weights_far_below_the_largest(temperature):
    """The largest weight against one e^-83 of it with as much less noise, 1e-6 apart."""
    B, V = 64, 5000
    g = torch.Generator().manual_seed(1)
    t = float(np.float32(temperature))
    target = torch.full((B, V), -INF)
    noise = torch.empty(B, V).exponential_(generator=g).clamp_(min=1e-30)
    deep = torch.randint(1, V, (B,), generator=g)
    z = -(80 + 3 * torch.rand(B, generator=g)) * temperature
    rows = torch.arange(B)
    target[:, 0], noise[:, 0] = 0.0, 0.5
    target[rows, deep] = z
    side = (torch.randint(0, 2, (B,), generator=g) * 2 - 1).double()
    noise[rows, deep] = (0.5 * torch.exp(z.double() / t) * (1 + 1e-6 * side)).float()
    assert (noise[rows, deep] > 1.2e-38).all()
    K0 = torch.empty(B, 0, dtype=torch.int32)
    want = verify(target, None, K0, [0] * B, None, noise, V, t)[0][:, 0]
    assert np.array_equal(want == 0, side.numpy() > 0)
    _same(target, torch.empty(0, V), K0, torch.empty(B, 0), noise, V, temperature)
